"""Layer norm and its gradient on the GPU against float64.

Tolerances, from the arithmetic (u = 2^-24, gamma(n) = n u / (1 - n u)): a row
is summed by at least 64 lanes and a tree, so a row sum passes at most
D = ceil(N / 64) + 16 additions; the column sums over M rows pass at most M + 16.
  mean      gamma(D) mean|x|
  variance  relative: 2 e_mean mean|d| / v + (e_mean^2) / v + gamma(D + 4)
  rstd      relative: half of that + 4 u
  y         |gamma r| e_mean + |gamma xh| e_rstd + 4 u (|gamma xh| + |beta|)
  dx        r (gamma(D + 4) mean|g| + |xh| gamma(D + 8) mean|g xh|
               + 8 u (|g| + |c1| + |xh c2|))
  dgamma    gamma(M + 20) sum|dy xh|     dbeta  gamma(M + 16) sum|dy|
and bf16 outputs add half a unit in the last place: 2^-8 |value| + 2^-134 (8 significant bits).
"""
from __future__ import annotations

import pytest
import torch

import packed_xor_popcount_amd as bnn

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def gam(n):
    return n * U / (1 - n * U)


def rounding(ref, dtype):
    return ref.abs() * 2.0 ** -8 + 2.0 ** -134 if dtype == torch.bfloat16 else 0.0


def fwd64(x, gamma, beta, eps):
    x = x.double()
    mean = x.mean(1)
    d = x - mean[:, None]
    v = d.square().mean(1)
    rstd = 1.0 / torch.sqrt(v + eps)
    g = torch.ones(x.shape[1], dtype=torch.float64, device=x.device) if gamma is None else gamma.double()
    b = torch.zeros_like(g) if beta is None else beta.double()
    xh = d * rstd[:, None]
    depth = -(-x.shape[1] // 64) + 16
    e_mean = gam(depth) * x.abs().mean(1)
    e_var = (2 * e_mean * d.abs().mean(1) + e_mean ** 2 + gam(depth + 4) * v) / (v + eps)
    e_rstd = 0.5 * e_var + 4 * U
    gx = (xh * g).abs()
    tol = (g.abs() * (rstd * e_mean)[:, None] + gx * e_rstd[:, None] + 4 * U * (gx + b.abs())) * 1.01
    return xh * g + b, mean, rstd, tol, e_mean * 1.01, rstd * e_rstd * 1.01


def bwd64(dy, x, mean, rstd, gamma):
    x, dy, mean, rstd = x.double(), dy.double(), mean.double(), rstd.double()
    M, N = x.shape
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy if gamma is None else dy * gamma.double()
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = rstd[:, None] * (g - c1 - xh * c2)
    depth = -(-N // 64) + 16
    tol = rstd[:, None] * (gam(depth + 4) * g.abs().mean(1, keepdim=True)
                           + xh.abs() * gam(depth + 8) * (g * xh).abs().mean(1, keepdim=True)
                           + 8 * U * (g.abs() + c1.abs() + (xh * c2).abs())) * 1.01
    return (dx, (dy * xh).sum(0), dy.sum(0), tol, gam(M + 20) * (dy * xh).abs().sum(0),
            gam(M + 16) * dy.abs().sum(0))


def rows_of(g, M, N, dtype, pad, shift=0, scale=1.0, mean=0.0):
    """M x N view of a wider buffer whose other places hold NaN; `shift`
    elements in front of the first row."""
    ld = N + pad
    buf = torch.full((shift + M * ld,), float("nan"), dtype=dtype, device=DEV)
    v = buf[shift:].view(M, ld)[:, :N]
    v.copy_((torch.randn(M, N, generator=g, device=DEV) * scale + mean).to(dtype))
    return v


def inside(got, ref, tol, what):
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((got.double() - ref).abs().max()))


def check(M, N, dtype, pad=0, shift=0, affine=True, scale=1.0, mean=0.0, eps=1e-5, seed=0):
    print("layernorm", M, N, dtype, pad, shift, affine, flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(1000 + seed)
    x = rows_of(g, M, N, dtype, pad, shift, scale, mean)
    dy = rows_of(g, M, N, dtype, pad, shift)
    gamma = 1 + 0.5 * torch.randn(N, generator=g, device=DEV) if affine else None
    beta = torch.randn(N, generator=g, device=DEV) if affine else None
    y, mu, r = bnn.layernorm_fwd(x, gamma, beta, eps)
    ref, mu64, r64, tol, tmu, tr = fwd64(x, gamma, beta, eps)
    assert y.dtype == dtype and tuple(y.shape) == (M, N)
    inside(mu, mu64, tmu, "mean")
    inside(r, r64, tr, "rstd")
    inside(y, ref, tol + rounding(ref, dtype), "y")
    y2, none1, none2 = bnn.layernorm_fwd(x, gamma, beta, eps, stats=False)
    assert torch.equal(y, y2) and none1 is None and none2 is None
    dx, dg, db = bnn.layernorm_bwd(dy, x, mu, r, gamma)
    rx, rg, rb, tx, tg, tb = bwd64(dy, x, mu, r, gamma)
    inside(dx, rx, tx + rounding(rx, dtype), "dx")
    inside(dg, rg, tg, "dgamma")
    inside(db, rb, tb, "dbeta")
    again = bnn.layernorm_bwd(dy, x, mu, r, gamma)
    assert all(torch.equal(a, b) for a, b in zip((dx, dg, db), again)), "not the same bits twice"
    only, none1, none2 = bnn.layernorm_bwd(dy, x, mu, r, gamma, params=False)
    assert torch.equal(only, dx) and none1 is None and none2 is None


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 2), (3, 7), (2, 63), (5, 64), (1, 65), (4, 255), (7, 256),
                                 (3, 511), (64, 512), (33, 513), (301, 1000), (17, 1024), (130, 2047),
                                 (9, 2049), (1, 4096), (4, 4096), (520, 4096), (3, 5000), (2, 8192),
                                 (3, 11008), (5, 16384), (2, 16391), (1, 65536), (2, 70001)])
def test_sizes(M, N, dtype):
    check(M, N, DT[dtype], seed=M * 7 + N)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (5, 3), (1, 8), (4, 4)])
@pytest.mark.parametrize("N", [64, 100, 1000, 4096, 4099])
def test_strides_and_alignment(N, pad, shift, dtype):
    check(19, N, DT[dtype], pad, shift, seed=pad * 31 + shift + N)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("M", [1, 2, 255, 256, 257, 1025, 5000, 16385])
def test_row_counts(M, dtype):
    check(M, 96, DT[dtype], seed=M)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_without_affine(dtype):
    check(37, 1000, DT[dtype], affine=False)


@pytest.mark.parametrize("N", [500, 4096])
def test_large_mean_small_spread(N):
    """A mean 1000 times the spread: the centred second pass keeps the variance."""
    check(21, N, torch.float32, scale=1.0, mean=1000.0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_constant_rows(dtype):
    x = torch.full((3, 260), 2.5, dtype=DT[dtype], device=DEV)
    y, mu, r = bnn.layernorm_fwd(x, None, torch.full((260,), 0.25, device=DEV), 1e-5)
    assert torch.equal(y.float(), torch.full_like(y.float(), 0.25))
    assert torch.equal(mu, torch.full_like(mu, 2.5))
    assert torch.allclose(r.double(), torch.full((3,), 1e-5 ** -0.5, dtype=torch.float64, device=DEV), rtol=1e-6)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("N", [70, 4096])
def test_a_bad_row_stays_alone(N, bad):
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    x = torch.randn(9, N, generator=g, device=DEV)
    ref, mu, r = bnn.layernorm_fwd(x)
    x2 = x.clone()
    x2[4, N - 1] = bad
    y, mu2, r2 = bnn.layernorm_fwd(x2)
    keep = [i for i in range(9) if i != 4]
    assert torch.equal(y[keep], ref[keep]) and torch.equal(mu2[keep], mu[keep])
    assert y[4].isnan().all() and r2[4].isnan()


def test_output_rows_of_a_wider_tensor():
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    for dtype in DT.values():
        for N, pad in ((100, 3), (128, 8), (1000, 1)):
            x = torch.randn(11, N, generator=g, device=DEV).to(dtype)
            wide = torch.full((11, N + pad), 7.0, dtype=dtype, device=DEV)
            y, _, _ = bnn.layernorm_fwd(x, out=wide[:, :N])
            assert torch.equal(y, bnn.layernorm_fwd(x)[0])
            assert (wide[:, N:] == 7.0).all()


def test_no_rows():
    x = torch.empty(0, 33, device=DEV)
    y, mu, r = bnn.layernorm_fwd(x)
    assert y.shape == (0, 33) and mu.shape == (0,)
    dx, dg, db = bnn.layernorm_bwd(x, x, mu, r)
    assert dx.shape == (0, 33) and not dg.any() and not db.any() and dg.shape == (33,)


def test_gradient_against_differences():
    """Central differences of the float64 forward pass, step 1e-4: their
    truncation is below step^2 |third derivative| / 6, which for rows of unit
    spread and N = 12 stays below 1e-6 (derivatives of y are of the order of
    r^3 <= 30 and the weights below 3)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    M, N, eps, h = 3, 12, 1e-5, 1e-4
    x = torch.randn(M, N, generator=g, device=DEV)
    gamma = 1 + 0.3 * torch.randn(N, generator=g, device=DEV)
    beta = torch.randn(N, generator=g, device=DEV)
    w = torch.randn(M, N, generator=g, device=DEV).clamp(-3, 3)
    y, mu, r = bnn.layernorm_fwd(x, gamma, beta, eps)
    dx, dg, db = bnn.layernorm_bwd(w, x, mu, r, gamma)

    def loss(x, gamma, beta):
        return (fwd64(x, gamma, beta, eps)[0] * w.double()).sum()

    def slopes(v, f):
        out = torch.zeros_like(v)
        for i in range(v.numel()):
            a, b = v.clone(), v.clone()
            a.view(-1)[i] += h
            b.view(-1)[i] -= h
            out.view(-1)[i] = (f(a) - f(b)) / (2 * h)
        return out

    x6, g6, b6 = x.double(), gamma.double(), beta.double()
    for got, num in ((dx, slopes(x6, lambda v: loss(v, g6, b6))), (dg, slopes(g6, lambda v: loss(x6, v, b6))),
                     (db, slopes(b6, lambda v: loss(x6, g6, v)))):
        assert (got.double() - num).abs().max() < 1e-6 + 64 * U * num.abs().max() + 64 * U


def test_rows_past_32_bit_offsets():
    """Rows whose element offsets pass 2^31 (and byte offsets 2^32)."""
    N, ld, M = 200, (1 << 20) + 8, 2100
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    big = torch.empty(M * ld, dtype=torch.bfloat16, device=DEV)
    x = big.view(M, ld)[:, :N]
    x.copy_(torch.randn(M, N, generator=g, device=DEV))
    y, mu, r = bnn.layernorm_fwd(x)
    ref = bnn.layernorm_fwd(x.contiguous())
    assert torch.equal(y, ref[0]) and torch.equal(mu, ref[1])
    dy = torch.randn(M, N, generator=g, device=DEV).to(torch.bfloat16)
    a = bnn.layernorm_bwd(dy, x, mu, r)
    b = bnn.layernorm_bwd(dy, x.contiguous(), mu, r)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_side_stream():
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    x = torch.randn(300, 777, generator=g, device=DEV)
    ref = bnn.layernorm_fwd(x)
    refb = bnn.layernorm_bwd(ref[0], x, ref[1], ref[2])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = bnn.layernorm_fwd(x)
        gotb = bnn.layernorm_bwd(got[0], x, got[1], got[2])
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(ref + refb, got + gotb))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("M,N", [(600, 1500), (600, 7000), (1100, 12001), (257, 3000), (1025, 16384), (513, 8192)])
def test_partial_rows(M, N, dtype):
    """Enough rows that the column sums pass through partial rows."""
    check(M, N, DT[dtype], seed=M + N)
