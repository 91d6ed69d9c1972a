"""Block-scaled 8-bit product on the GPU where operands differ much in size:
products that cancel, operands that decode to 2^128, scale bytes of 0.

Inputs are built so that every partial sum that matters is exact in fp32 (the
bound is stated with each test), so the results are compared bit for bit, or
within the fp32 bound of a sum of K terms (gamma(K + 8) sum|x w|, u = 2^-23)
and one rounding to bf16 (2^-8 |y|).
"""
from __future__ import annotations

import pytest
import torch

import packed_xor_popcount_amd as bnn
from tests.test_gpu_f8 import DEV, DT, U, decode, test_nan_reaches_its_row_and_column_only as check_nan
from tests.test_gpu_f8 import test_product_exact as check_exact, test_product_rounding as check_rounding

pytestmark = pytest.mark.gpu

# Row counts and widths that reach each kernel: few rows (16 and 32 at a
# time), small tiles, large tiles.
PLACES = [(1, 70), (16, 33), (17, 70), (32, 65), (33, 70), (300, 129), (2900, 2999), (3300, 3301)]


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


def check_sizes(x, w, K, kind, least=-1.0):
    """Outputs whose products' magnitudes sum to more than `least` and fit
    fp32.  kind "fast": bf16 by the 8-bit instructions, which also drop up to
    7 2^-13 of the largest product of each eight consecutive k."""
    a, b = decode(*x, K), decode(*w, K)
    ref, size = a @ b.t(), a.abs() @ b.abs().t()
    y = bnn.gemm_f8(*x, *w, K, dtype=DT[kind] if kind in DT else DT["bf16"], fast=kind == "fast").double()
    n = K + 8
    tol = n * U / (1 - n * U) * size
    if kind == "fast":
        tol = tol + 7 * 2.0 ** -13 * (a.abs().view(len(a), -1, 8).amax(2) @ b.abs().view(len(b), -1, 8).amax(2).t())
    if kind != "fp32":
        tol = tol * 1.01 + ref.abs() * 2.0 ** -8
    fits = (size < 3.0e38) & (size > least)
    bad = ~((y - ref).abs() <= tol) & fits
    assert fits.any() and not bad.any(), (int(bad.sum()), y[bad][:4], ref[bad][:4])


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fast"])
@pytest.mark.parametrize("where", ["x", "w", "both"])
@pytest.mark.parametrize("M,N", PLACES)
def test_largest_finite_values(M, N, where, dtype):
    """The largest finite bf16 value is rounded to 256 * 2^120 = 2^128, past
    the range of bf16: against small weights the product is finite, and
    against zeros it is zero."""
    print("largest", M, N, where, dtype, flush=True)
    K = 200
    g = torch.Generator(device=DEV)
    g.manual_seed(M * 3 + N)
    big = torch.finfo(torch.bfloat16).max

    def operand(rows, has):
        v = torch.randint(-2, 3, (rows, K), generator=g, device=DEV).float() * 2.0 ** -30
        if has:
            r = torch.arange(0, rows, 3, device=DEV)
            v[r, r * 7 % K] = big
            v[r, r * 5 % K] = -big
        return bnn.quant_f8(v)

    x, w = operand(M, where != "w"), operand(N, where != "x")
    check_sizes(x, w, K, dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fast"])
@pytest.mark.parametrize("where", ["x", "w"])
@pytest.mark.parametrize("M,N", PLACES)
def test_smallest_scale(M, N, where, dtype):
    """Blocks of scale byte 0 (2^-127), their values 2 .. 8 times that and so
    normal numbers, beside rows of ordinary values and of 2^128."""
    print("smallest", M, N, where, dtype, flush=True)
    K = 200
    g = torch.Generator(device=DEV)
    g.manual_seed(M * 5 + N)

    def ints(rows):
        s = 1 - 2 * torch.randint(0, 2, (rows, K), generator=g, device=DEV).double()
        return torch.randint(2, 9, (rows, K), generator=g, device=DEV).double() * s

    def tiny(rows):
        v = ints(rows)
        v *= torch.exp2(torch.tensor([-127.0, 0.0, -127.0], dtype=torch.float64, device=DEV))[
            torch.arange(rows, device=DEV) % 3][:, None]
        v = v.float()
        v[2::3, 0] = torch.finfo(torch.bfloat16).max
        v[2::3, 1:128] = 0
        q, s = bnn.quant_f8(v)
        assert (s[0::3, :2] == 0).all() and (s[2::3, 1] == 0).all()
        return q, s

    def plain(rows):  # in one half of the columns large, so that tiny products are normal numbers
        v = ints(rows)
        v[::2] *= 2.0 ** 60
        v[1::2] *= 2.0 ** -20
        return bnn.quant_f8(v.float())

    if where == "x":
        x, w = tiny(M), plain(N)
    else:
        x, w = plain(M), tiny(N)
    check_sizes(x, w, K, dtype, 2.0 ** -90)  # above it no product is near the subnormals


@pytest.mark.parametrize("M,N,K", [(3300, 3301, 300), (2600, 4300, 1024), (10700, 1000, 129), (4096, 2600, 0)])
def test_large_tiles(M, N, K):
    """Products of enough outputs for the large tiles, whole and partial."""
    if K == 0:
        z = torch.empty(max(M, N), 0, dtype=torch.uint8, device=DEV)
        for dtype in DT.values():
            assert not bnn.gemm_f8(z[:M], z[:M], z[:N], z[:N], 0, out=torch.full((M, N), 9.0, device=DEV, dtype=dtype)).any()
        return
    check_exact(M, N, K)
    check_rounding(M, N, K)


def test_nan_in_large_tiles():
    check_nan(160000)  # by 70 columns: as many outputs as 170 large tiles
