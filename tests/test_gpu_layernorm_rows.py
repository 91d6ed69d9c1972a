"""Layer norm and its gradient where every block takes more than one row: the
long-row kernels' accumulated column sums and reused buffers, the second rows
of the register kernels."""
from __future__ import annotations

import pytest

from tests.test_gpu_layernorm import DT, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("M,N", [(600, 16391), (257, 20001), (513, 16400), (8200, 1000), (2100, 1500), (2100, 4096),
                                 (2049, 4099), (1030, 7000), (16384, 512)])
def test_second_rows(M, N, dtype):
    check(M, N, DT[dtype], seed=M + 2 * N)


@pytest.mark.parametrize("N", [16391, 4096])
def test_second_rows_strided(N):
    for dtype in DT.values():
        check(2100 if N == 4096 else 600, N, dtype, pad=5, shift=3, affine=False, seed=N)
