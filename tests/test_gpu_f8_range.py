"""Block-scaled 8-bit product on the GPU where operands differ much in size:
products that cancel.

Inputs are built so that every partial sum that matters is exact in fp32 (the
bound is stated with each test), so the results are compared bit for bit.
"""
from __future__ import annotations

import pytest
import torch

import packed_xor_popcount_amd as bnn
from tests.test_gpu_f8 import DEV, DT, decode

pytestmark = pytest.mark.gpu

# Row counts and widths that reach each kernel: few rows (16 and 32 at a
# time), small tiles, large tiles.
PLACES = [(1, 70), (16, 33), (17, 70), (32, 65), (33, 70), (300, 129), (2900, 2999)]


def cancelling(g, rows, k, weight):
    """Groups of eight consecutive k: two ones (in a weight of opposite signs,
    so that their products cancel), then 2^-8 or 0 (a weight: +-2^-8)."""
    nb = -(-k // 128)
    at = torch.arange(nb * 128, device=DEV) % 8
    s = 1.0 - 2.0 * torch.randint(0, 2, (rows, nb * 16), generator=g, device=DEV).repeat_interleave(8, 1)
    r = torch.randint(0, 2, (rows, nb * 128), generator=g, device=DEV).float()
    if weight:
        v = torch.where(at == 0, s, torch.where(at == 1, -s, (1 - 2 * r) * 2.0 ** -8))
    else:
        v = torch.where(at < 2, torch.ones_like(r), r * 2.0 ** -8)
    v[:, k - k % 8:] = 0
    q = v.to(torch.float8_e4m3fn).view(torch.uint8)
    sc = torch.zeros(rows, bnn.f8_scale_bytes(k), dtype=torch.uint8, device=DEV)
    sc[:, :nb] = 127
    return q, sc


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("M,N", PLACES)
def test_small_products_beside_cancelling_ones(M, N, dtype):
    """Products of +-1 cancel exactly; what is left are at most 228 products of
    +-2^-16, a sum of eight significant bits.  Partial sums are multiples of
    2^-16 below 2^6: exact in fp32 in any order."""
    print("cancelling", M, N, dtype, flush=True)
    K = 300
    g = torch.Generator(device=DEV)
    g.manual_seed(M + N)
    x, w = cancelling(g, M, K, False), cancelling(g, N, K, True)
    ref = decode(*x, K) @ decode(*w, K).t()
    assert (ref != 0).any()
    y = bnn.gemm_f8(*x, *w, K, dtype=DT[dtype])
    assert torch.equal(y.double(), ref)
