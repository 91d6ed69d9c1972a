"""Layer norm and its gradient where every block takes more than one row: the
long-row kernels' accumulated column sums and reused buffers, the second rows
of the register kernels."""
from __future__ import annotations

import pytest
import torch

import packed_xor_popcount_amd as bnn
from tests.test_gpu_layernorm import DEV, DT, check, gam

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


def test_rows_past_2_27_columns():
    """More columns than one launch of 16 threads each covers with 2^32
    threads.  Sums over two rows: gamma(M + 20) sum|dy xh| as for any M."""
    M, N = 2, 2 ** 27 + 13
    print("layernorm", M, N, flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(27)
    x = torch.randn(M, N, generator=g, device=DEV).to(torch.bfloat16)
    dy = torch.randn(M, N, generator=g, device=DEV).to(torch.bfloat16)
    mean, rstd = torch.tensor([0.1, -0.2], device=DEV), torch.tensor([0.9, 1.1], device=DEV)
    dx, dg, db = bnn.layernorm_bwd(dy, x, mean, rstd)
    for lo in range(0, N, 2 ** 24):
        part = slice(lo, min(N, lo + 2 ** 24))
        d = dy[:, part].double()
        xh = (x[:, part].double() - mean.double()[:, None]) * rstd.double()[:, None]
        assert ((dg[part].double() - (d * xh).sum(0)).abs() <= gam(M + 20) * (d * xh).abs().sum(0)).all()
        assert ((db[part].double() - d.sum(0)).abs() <= gam(M + 16) * d.abs().sum(0)).all()
        assert dx[:, part].isfinite().all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N", [70, 4096, 20001])
def test_past_the_range_of_fp32(N, dtype):
    """A row whose squares overflow gives r = 0 and y = beta, one whose sum
    overflows an infinite mean and y = NaN; the rows beside them are as they are alone."""
    g = torch.Generator(device=DEV)
    g.manual_seed(N)
    x = torch.randn(5, N, generator=g, device=DEV).to(DT[dtype])
    beta = torch.randn(N, generator=g, device=DEV)
    ref, _, r = bnn.layernorm_fwd(x, None, beta)
    low = torch.finfo(torch.bfloat16).min
    x[1, N // 2] = low
    x[3, 1] = x[3, N - 1] = low
    y, mu2, r2 = bnn.layernorm_fwd(x, None, beta)
    keep = [0, 2, 4]
    assert torch.equal(y[keep], ref[keep]) and torch.equal(r2[keep], r[keep])
    assert r2[1] == 0 and torch.equal(y[1], beta.to(DT[dtype]))
    assert mu2[3].isinf() and y[3].isnan().all()
