"""Scales near the ends of fp32 in the grouped sign-weight product: the output
is row_scale * (alpha * sum) with each product rounded once, so nothing but
those products may overflow or vanish."""
from __future__ import annotations

import pytest
import torch

import packed_xor_popcount_amd as bnn
from tests.test_gpu_signw_grouped import ALGOS, DEV, DT, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("algo", list(ALGOS))
@pytest.mark.parametrize("counts,N,K", [([3, 0, 40, 1], 70, 130), ([140, 300, 17, 190], 600, 200),
                                        ([9000, 0, 4100], 1100, 70), ([20, 9, 0, 30] * 20, 300, 64)])
def test_scales_at_the_ends_of_fp32(counts, N, K, algo):
    """Activations 0 and +-1 at a few places, so sums are small integers, many
    of them 0; alpha up to the largest fp32 value, where sums of 0 stay 0 and
    sums of 1 the scale itself, and down to the smallest normal one."""
    c = Case(21, counts, N, K, integers=True, row_scale=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(N)
    few = torch.rand(c.x.shape, generator=g, device=DEV) < 1.0 / K
    c.x.copy_(torch.where(few, c.x.sign(), torch.zeros_like(c.x)))
    c.alpha.copy_(torch.tensor([3.4e38, -2.0e38, 1.0, 1.2e-38], device=DEV)[
        torch.randint(0, 4, c.alpha.shape, generator=g, device=DEV)])
    c.row_scale.copy_(torch.tensor([1.0, 2.0 ** -100, -0.5], device=DEV)[torch.arange(c.R, device=DEV) % 3])
    s, _ = c.sums()
    a, r = c.factors()
    ref = (s.float() * a) * r
    use = c.inside()
    assert (s == 0).any() and (s.abs() == 1).any() and ref.isfinite().any()
    for dtype in DT.values():
        y = c.run(ALGOS[algo], dtype)
        assert torch.equal(y[use], ref.to(dtype)[use])
