"""Low-rank adapters and their gradient on the GPU against float64.

Small whole numbers keep every sum exact (x and the factors of up to 3, ranks
and lengths so small that no sum reaches 2^24): results are equal.  Otherwise
products are exact and sums fp32, in units that may not round to nearest
(u = 2^-23, gamma(n) = n u / (1 - n u)):
  u, v     gamma(K + 8) sum|x a|
  out      gamma(3 r + 8) (|base| + |s| sum|u b|), u as the kernel made it
  dx       the same, plus |s| sum_j err(v_j) |a_j|
  da       gamma(3 T + 40) |s| sum|v x| + |s| sum err(v) |x|;  db the same without err
bf16 outputs add half a step, 2^-8 of the value.
"""
from __future__ import annotations

import pytest
import torch

import packed_xor_popcount_amd as bnn

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -23
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def gam(n):
    return n * U / (1 - n * U)


class Case:
    def __init__(self, seed, T, K, N, r, L, ids="mixed", pad=0, shift=0, integers=True, dtype=torch.float32):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)
        self.T, self.K, self.N, self.r, self.L, self.integers, self.dtype = T, K, N, r, L, integers, dtype
        i = torch.randint(-1, L, (T,), generator=self.g, device=DEV)
        if ids == "sorted":
            i = torch.sort(i).values
        elif ids == "one":
            i = torch.full((T,), L - 1, device=DEV)
        elif ids == "none":
            i = torch.where(torch.arange(T, device=DEV) % 2 == 0, -2 ** 31, L + 5)
        elif ids == "runs":
            i = i[torch.sort(torch.randint(0, T, (T,), generator=self.g, device=DEV)).values // 7 * 7 % T]
        self.ids = i.to(torch.int32)
        self.a, self.b = self.values(L, r, K), self.values(L, r, N)
        self.scale = torch.randint(1, 3, (L,), generator=self.g, device=DEV).float() if integers else \
            torch.randn(L, generator=self.g, device=DEV)
        self.x = self.rows(T, K, torch.bfloat16, pad, shift)
        self.dy = self.rows(T, N, torch.bfloat16, pad, shift)
        self.base = self.rows(T, N, dtype, pad, shift)
        self.dbase = self.rows(T, K, dtype, pad, shift)

    def values(self, *shape):
        v = torch.randint(-3, 4, shape, generator=self.g, device=DEV) if self.integers else \
            torch.randn(*shape, generator=self.g, device=DEV)
        return v.to(torch.bfloat16)

    def rows(self, M, N, dtype, pad, shift):
        """M x N view of a wider buffer whose other places hold NaN."""
        ld = N + pad
        buf = torch.full((shift + M * ld,), float("nan"), dtype=dtype, device=DEV)
        v = buf[shift:].view(M, ld)[:, :N]
        v.copy_(self.values(M, N))
        return v

    def each(self):
        for l in range(self.L):
            at = torch.nonzero(self.ids == l).flatten()
            if len(at):
                yield l, at


def rounding(ref, dtype):
    return ref.abs() * 2.0 ** -8 + 2.0 ** -133 if dtype == torch.bfloat16 else 0.0


def inside(got, ref, tol, what, integers):
    if integers and got.dtype == torch.float32:
        assert torch.equal(got.double(), ref), f"{what}: {(got.double() - ref).abs().max()}"
        return
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), f"{what}: {err.max()}"


def check_fwd(c, scale=True, base=True):
    sc, bs = (c.scale if scale else None), (c.base if base else None)
    out, u = bnn.adapter_fwd(c.x, c.ids, c.a, c.b, scale=sc, base=bs, dtype=c.dtype)
    ref_u = torch.zeros(c.T, c.r, dtype=torch.float64, device=DEV)
    tol_u = torch.zeros_like(ref_u)
    ref = c.base.double().clone() if base else torch.zeros(c.T, c.N, dtype=torch.float64, device=DEV)
    size = ref.abs()
    for l, at in c.each():
        x, a, b = c.x[at].double(), c.a[l].double(), c.b[l].double()
        s = float(c.scale[l]) if scale else 1.0
        ref_u[at] = x @ a.t()
        tol_u[at] = gam(c.K + 8) * (x.abs() @ a.abs().t())
        ref[at] += s * (u[at].double() @ b)
        size[at] += abs(s) * (u[at].double().abs() @ b.abs())
    inside(u, ref_u, tol_u, "u", c.integers)
    inside(out, ref, gam(3 * c.r + 8) * size + rounding(ref, out.dtype), "out", c.integers)
    none = (c.ids < 0) | (c.ids >= c.L)
    assert not u[none].any()
    assert torch.equal(out[none], c.base[none] if base else torch.zeros_like(out[none]))
    return out, u


SIZES = [(1, 1, 1, 1, 1), (1, 4096, 4096, 16, 3), (2, 7, 9, 5, 2), (15, 64, 130, 8, 4), (16, 127, 128, 16, 1), (17, 128, 127, 17, 5),
         (33, 129, 1000, 33, 40), (40, 1000, 70, 64, 7), (64, 520, 300, 100, 3), (100, 256, 513, 128, 20), (300, 140, 90, 4, 300),
         (513, 136, 700, 12, 6), (1100, 72, 40, 32, 2), (5000, 40, 24, 16, 9)]


@pytest.mark.parametrize("ids", ["mixed", "sorted", "one", "none", "runs"])
@pytest.mark.parametrize("T,K,N,r,L", SIZES)
def test_fwd(T, K, N, r, L, ids):
    for pad, shift, scale, base, integers, dt in ((0, 0, True, True, True, "fp32"), (3, 1, True, True, False, "bf16"),
                                                  (8, 0, False, False, False, "fp32")):
        check_fwd(Case(T + K, T, K, N, r, L, ids, pad, shift, integers, DT[dt]), scale, base)


def kept_in_8_bits(x):
    q, s = bnn.quant_f8(x)
    nb = q.shape[1] // 128
    v = q.view(torch.float8_e4m3fn).double().view(len(q), nb, 128) * torch.exp2(s[:, :nb].double() - 127)[:, :, None]
    return (q, s), v.view(len(q), -1)[:, :x.shape[1]]


def check_bwd(c, kept, scale=True, base=True):
    sc, bs = (c.scale if scale else None), (c.dbase if base else None)
    _, u = bnn.adapter_fwd(c.x, c.ids, c.a, c.b, scale=sc)
    arg, x6 = kept_in_8_bits(c.x) if kept == "f8" else (c.x, c.x.double())
    dx, da, db = bnn.adapter_bwd(c.dy, arg, u, c.ids, c.a, c.b, scale=sc, base=bs, dtype=c.dtype)
    ref = c.dbase.double().clone() if base else torch.zeros(c.T, c.K, dtype=torch.float64, device=DEV)
    tol = gam(3 * c.r + 8) * ref.abs()
    ref_a, ref_b = torch.zeros(c.L, c.r, c.K, dtype=torch.float64, device=DEV), torch.zeros(c.L, c.r, c.N,
                                                                                            dtype=torch.float64, device=DEV)
    tol_a, tol_b = torch.zeros_like(ref_a), torch.zeros_like(ref_b)
    for l, at in c.each():
        d, a, b, s = c.dy[at].double(), c.a[l].double(), c.b[l].double(), float(c.scale[l]) if scale else 1.0
        v, ev = d @ b.t(), gam(c.N + 8) * (d.abs() @ b.abs().t())
        ref[at] += s * (v @ a)
        tol[at] += abs(s) * (gam(3 * c.r + 8) * (v.abs() @ a.abs()) + ev @ a.abs()) * 1.01
        g = gam(3 * len(at) + 40)
        ref_a[l], ref_b[l] = s * (v.t() @ x6[at]), s * (u[at].double().t() @ d)
        tol_a[l] = abs(s) * (g * (v.abs().t() @ x6[at].abs()) + ev.t() @ x6[at].abs()) * 1.01
        tol_b[l] = abs(s) * g * (u[at].double().abs().t() @ d.abs()) * 1.01
    inside(dx, ref, tol + rounding(ref, dx.dtype), "dx", c.integers)
    inside(da, ref_a, tol_a, "da", c.integers)
    inside(db, ref_b, tol_b, "db", c.integers)
    only, none_a, none_b = bnn.adapter_bwd(c.dy, None, None, c.ids, c.a, c.b, scale=sc, base=bs, dtype=c.dtype, params=False)
    assert none_a is None and none_b is None and torch.equal(only, dx)
    no_dx, da2, db2 = bnn.adapter_bwd(c.dy, arg, u, c.ids, c.a, c.b, scale=sc, dx=False)
    assert no_dx is None and torch.equal(db2, db)
    inside(da2, ref_a, tol_a, "da without dx", c.integers)


@pytest.mark.parametrize("ids", ["mixed", "sorted", "one", "none", "runs"])
@pytest.mark.parametrize("T,K,N,r,L", SIZES)
def test_bwd(T, K, N, r, L, ids):
    for pad, shift, scale, base, integers, dt, kept in ((0, 0, True, True, True, "fp32", "bf16"),
                                                        (3, 1, True, True, False, "bf16", "f8"),
                                                        (0, 0, False, True, True, "fp32", "f8"),
                                                        (8, 0, False, False, False, "fp32", "bf16")):
        check_bwd(Case(T + K, T, K, N, r, L, ids, pad, shift, integers, DT[dt]), kept, scale, base)


@pytest.mark.parametrize("T,L,ids", [(3000, 3, "sorted"), (3000, 1, "one"), (2600, 600, "mixed"), (9000, 5, "runs"),
                                     (20000, 2, "mixed"), (300, 1010, "mixed"), (9000, 700, "mixed"), (8192, 1000, "runs"),
                                     (8193, 1, "one")])
def test_bwd_of_many_rows(T, L, ids):
    """Adapters whose rows are cut into several tiles, and many adapters."""
    for kept in ("bf16", "f8"):
        check_bwd(Case(T, T, 200, 136, 20, L, ids), kept)


@pytest.mark.parametrize("r", [3, 16, 17, 64, 65])
@pytest.mark.parametrize("T,K,N", [(300, 5, 300), (300, 300, 5), (90, 3, 2), (700, 8, 1024), (700, 1500, 7)])
def test_bwd_of_narrow_sides(T, K, N, r):
    """The input's gradient and the parameters' in one launch (ranks up to 64) and in two, at uneven widths."""
    for kept, dt in (("bf16", "fp32"), ("f8", "bf16")):
        check_bwd(Case(K + r, T, K, N, r, 6, "runs", pad=1, integers=False, dtype=DT[dt]), kept)


def test_bwd_of_many_adapters_and_columns():
    """More blocks than one launch takes for both gradients; whole numbers below 2^24, so every sum is exact."""
    T, K, N, L = 1030, 266000, 271003, 1024
    c = Case(5, T, K, N, 1, L, "mixed")
    at = (c.ids >= 0).nonzero().flatten()
    l = c.ids[at].long()
    _, u = bnn.adapter_fwd(c.x, c.ids, c.a, c.b, scale=c.scale)
    dx, da, db = bnn.adapter_bwd(c.dy, c.x, u, c.ids, c.a, c.b, scale=c.scale, base=c.dbase)
    ref = c.dbase.clone()
    sums = [torch.zeros(L, K, device=DEV), torch.zeros(L, N, device=DEV)]
    most = 0.0
    for i in range(0, len(at), 64):
        t, m = at[i:i + 64], l[i:i + 64]
        s = c.scale[m][:, None]
        v = (c.dy[t].float() * c.b[m, 0].float()).sum(1, keepdim=True)
        ref[t] += s * v * c.a[m, 0].float()
        for d, w, y in ((sums[0], v, c.x), (sums[1], u[t], c.dy)):
            p = s * w * y[t].float()
            most = max(most, float(p.abs().max()))
            d.index_add_(0, m, p)
    assert most * int(torch.bincount(l).max()) < 2 ** 24
    assert torch.equal(dx, ref) and torch.equal(da[:, 0], sums[0]) and torch.equal(db[:, 0], sums[1])


@pytest.mark.parametrize("T", [255, 256, 257, 512])
@pytest.mark.parametrize("N,r,L", [(300, 16, 40), (1030, 32, 2), (2100, 33, 3), (9000, 16, 250)])
def test_chunk_ends_and_the_choice_of_kernels(T, N, r, L):
    for ids in ("mixed", "sorted"):
        check_fwd(Case(T + N, T, 260, N, r, L, ids))


def test_order_of_rows_does_not_matter_to_a_row():
    c = Case(4, 200, 300, 260, 16, 6, integers=False)
    out, u = bnn.adapter_fwd(c.x, c.ids, c.a, c.b, scale=c.scale, base=c.base)
    p = torch.randperm(200, generator=c.g, device=DEV)
    out2, u2 = bnn.adapter_fwd(c.x[p], c.ids[p].contiguous(), c.a, c.b, scale=c.scale, base=c.base[p])
    assert torch.equal(out[p], out2) and torch.equal(u[p], u2)


@pytest.mark.parametrize("T", [40, 700])
def test_in_place(T):
    c = Case(5, T, 100, 90, 8, 3, pad=6)
    ref, _ = bnn.adapter_fwd(c.x, c.ids, c.a, c.b, scale=c.scale, base=c.base)
    before = c.base.clone()
    out, _ = bnn.adapter_fwd(c.x, c.ids, c.a, c.b, scale=c.scale, base=c.base, out=c.base)
    assert out.data_ptr() == c.base.data_ptr() and torch.equal(out, ref)
    assert torch.equal(out[c.ids < 0], before[c.ids < 0])


def test_nan_and_infinities_stay_in_their_rows():
    c = Case(6, 100, 200, 150, 12, 4, integers=False)
    clean, u0 = bnn.adapter_fwd(c.x, c.ids, c.a, c.b, scale=c.scale, base=c.base)
    dx0, da0, db0 = bnn.adapter_bwd(c.dy, c.x, u0, c.ids, c.a, c.b, scale=c.scale)
    at = int(torch.nonzero(c.ids == 2)[0])
    none = int(torch.nonzero(c.ids < 0)[0])
    other = c.ids != 2
    for bad in (float("nan"), float("inf")):
        x, dy = c.x.clone(), c.dy.clone()
        x[at, 3], x[none] = bad, bad
        dy[at, 5], dy[none] = bad, bad
        out, u = bnn.adapter_fwd(x, c.ids, c.a, c.b, scale=c.scale, base=c.base)
        rest = torch.arange(100, device=DEV) != at
        assert torch.equal(out[rest], clean[rest]) and torch.equal(u[rest], u0[rest])
        assert not torch.isfinite(u[at]).all() and not torch.isfinite(out[at]).any()
        dx, da, db = bnn.adapter_bwd(dy, x, u, c.ids, c.a, c.b, scale=c.scale)
        assert torch.equal(dx[rest], dx0[rest])
        keep = torch.tensor([0, 1, 3], device=DEV)
        assert torch.equal(da[keep], da0[keep]) and torch.equal(db[keep], db0[keep])
    # an adapter with infinities in its factors reaches its own rows only
    a = c.a.clone()
    a[2, :, 0] = float("inf")
    out, u = bnn.adapter_fwd(c.x, c.ids, a, c.b, scale=c.scale, base=c.base)
    assert torch.equal(out[other], clean[other]) and torch.equal(u[other], u0[other])


def test_values_past_bf16s_range_of_parts():
    """u up to fp32's largest values and below bf16's smallest: the parts add up to it."""
    x = torch.zeros(3, 2, dtype=torch.bfloat16, device=DEV)
    x[0, 0], x[1, 0], x[2, 0] = 3.3e38, 2.0 ** -100, -3.3e38
    a = torch.ones(1, 1, 2, dtype=torch.bfloat16, device=DEV)
    b = torch.full((1, 1, 4), 0.5, dtype=torch.bfloat16, device=DEV)
    out, u = bnn.adapter_fwd(x, torch.zeros(3, dtype=torch.int32, device=DEV), a, b)
    assert torch.equal(u[:, 0], x[:, 0].float()) and torch.equal(out, (u * 0.5).expand(3, 4))


def test_8_bit_input_at_the_ends_of_its_range():
    """Blocks of the largest and smallest scales: finite sums stay finite, zeros stay zeros."""
    x = torch.zeros(4, 256, device=DEV)
    x[0, 0], x[1, 1], x[2, 130], x[3, 131] = 3.3e38, 2.0 ** -126, 1.0, 2.0 ** -120
    q = bnn.quant_f8(x)
    ids = torch.zeros(4, dtype=torch.int32, device=DEV)
    a = torch.ones(1, 1, 256, dtype=torch.bfloat16, device=DEV)
    b = torch.ones(1, 1, 8, dtype=torch.bfloat16, device=DEV)
    dy = torch.zeros(4, 8, dtype=torch.bfloat16, device=DEV)
    dy[:, 0] = torch.tensor([2.0 ** -60, 2.0 ** 30, 3.0, 2.0 ** 20], device=DEV)
    u = torch.zeros(4, 1, device=DEV)
    _, da, _ = bnn.adapter_bwd(dy, q, u, ids, a, b)
    want = torch.zeros(256, device=DEV)
    want[0], want[1], want[130], want[131] = 2.0 ** 68, 2.0 ** -96, 3.0, 2.0 ** -100
    assert torch.equal(da[0, 0], want)


def test_against_differences():
    """The bilinear form <dy, out>: central differences are exact but for rounding."""
    c = Case(8, 6, 11, 9, 3, 2, integers=False)
    _, u = bnn.adapter_fwd(c.x, c.ids, c.a, c.b, scale=c.scale)
    dx, da, db = bnn.adapter_bwd(c.dy, c.x, u, c.ids, c.a, c.b, scale=c.scale)

    def value(x, a, b):
        total = 0.0
        for l, at in c.each():
            total = total + float(c.scale[l]) * (((x[at] @ a[l].t()) @ b[l]) * c.dy[at].double()).sum()
        return total

    args = [c.x.double(), c.a.double(), c.b.double()]
    h = 2.0 ** -10
    for i, grad in enumerate((dx, da, db)):
        flat = grad.double().flatten()
        for n in range(0, flat.numel(), 5):
            up, down = [v.clone() for v in args], [v.clone() for v in args]
            up[i].view(-1)[n] += h
            down[i].view(-1)[n] -= h
            # sums of at most 6 * 9 * 11 products of normal values in fp32: 1e-4 is 40 of their roundings
            assert abs((value(*up) - value(*down)) / (2 * h) - flat[n]) <= 1e-4, (i, n)


def test_empty():
    c = Case(2, 5, 8, 6, 2, 3)
    out, u = bnn.adapter_fwd(c.x[:0], c.ids[:0], c.a, c.b)
    assert out.shape == (0, 6) and u.shape == (0, 2)
    dx, da, db = bnn.adapter_bwd(c.dy[:0], c.x[:0], u, c.ids[:0], c.a, c.b)
    assert dx.shape == (0, 8) and not da.any() and not db.any() and da.shape == (3, 2, 8)
    none = torch.zeros(0, 2, 8, dtype=torch.bfloat16, device=DEV)
    out, u = bnn.adapter_fwd(c.x, c.ids, none, none[:, :, :6], base=c.base)
    assert torch.equal(out, c.base) and not u.any()
    dx, da, db = bnn.adapter_bwd(c.dy, c.x, u, c.ids, none, none[:, :, :6], base=c.dbase)
    assert torch.equal(dx, c.dbase) and da.shape == (0, 2, 8)
    nok = torch.zeros(5, 0, dtype=torch.bfloat16, device=DEV)
    out, u = bnn.adapter_fwd(nok, c.ids, c.a[:, :, :0].contiguous(), c.b, base=c.base)
    assert torch.equal(out, c.base) and not u.any()
    out, u = bnn.adapter_fwd(c.x, c.ids, c.a, c.b[:, :, :0].contiguous())
    assert out.shape == (5, 0) and torch.equal(u, check_fwd(c)[1])


def test_activations_past_32_bit_offsets():
    ld, T, K, N = (1 << 20) + 8, 2100, 136, 200
    c = Case(3, T, K, N, 8, 3, "runs")
    x = torch.empty(T * ld, dtype=torch.bfloat16, device=DEV).view(T, ld)[:, :K]
    x.copy_(c.x)
    base = torch.empty(T * ld, dtype=torch.bfloat16, device=DEV).view(T, ld)[:, :N]
    base.copy_(c.base)
    a, u = bnn.adapter_fwd(x, c.ids, c.a, c.b, base=base, out=base)
    b, u2 = bnn.adapter_fwd(c.x, c.ids, c.a, c.b, base=c.base.to(torch.bfloat16))
    assert torch.equal(a, b) and torch.equal(u, u2)


def test_factors_past_32_bit_offsets():
    L, r, K = 70, 128, 1 << 18
    c = Case(3, 40, K, 16, r, 1, "one")
    a = c.a.expand(L, r, K).clone()
    a[L - 1] *= -1
    assert a.numel() * 2 > 2 ** 32
    b = c.b.expand(L, r, 16).contiguous()
    for l, sign in ((L - 1, -1), (L - 2, 1)):
        ids = torch.full((40,), l, dtype=torch.int32, device=DEV)
        _, u = bnn.adapter_fwd(c.x, ids, a, b)
        _, u1 = bnn.adapter_fwd(c.x, torch.zeros_like(ids), c.a, c.b)
        assert torch.equal(u, sign * u1)


def test_side_stream_and_equal_bits():
    c = Case(9, 700, 300, 260, 16, 6, "runs", integers=False)

    def both():
        out, u = bnn.adapter_fwd(c.x, c.ids, c.a, c.b, scale=c.scale, base=c.base)
        return out, u, *bnn.adapter_bwd(c.dy, c.x, u, c.ids, c.a, c.b, scale=c.scale, base=c.dbase)

    ref = both()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        runs = [both() for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(a, b) for got in runs for a, b in zip(ref, got))


def test_bindings_refuse():
    c = Case(1, 4, 8, 6, 2, 3)
    with pytest.raises(TypeError):
        bnn.adapter_fwd(c.x.float(), c.ids, c.a, c.b)
    with pytest.raises(ValueError):
        bnn.adapter_fwd(c.x, c.ids.long(), c.a, c.b)
    with pytest.raises(ValueError):
        bnn.adapter_fwd(c.x, c.ids, c.a, c.b[:2])
    with pytest.raises(ValueError):
        bnn.adapter_fwd(c.x, c.ids, c.a.transpose(1, 2), c.b)
    with pytest.raises(ValueError):
        bnn.adapter_fwd(c.x, c.ids, c.a, c.b, base=c.base[:, :5])
    with pytest.raises(ValueError):
        bnn.adapter_fwd(c.x, c.ids, c.a, c.b, base=c.base, dtype=torch.bfloat16)
    big = torch.zeros(1, 129, 8, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(bnn.BnnError):
        bnn.adapter_fwd(c.x, c.ids, big, big[:, :, :6].contiguous())
    u = torch.zeros(4, 2, device=DEV)
    with pytest.raises(ValueError):
        bnn.adapter_bwd(c.dy, c.x[:3], u, c.ids, c.a, c.b)
    with pytest.raises(ValueError):
        bnn.adapter_bwd(c.dy, c.x, u[:, :1], c.ids, c.a, c.b)
    many = torch.zeros(1025, 2, 8, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(bnn.BnnError):
        bnn.adapter_bwd(c.dy, c.x, u, c.ids, many, many[:, :, :6].contiguous())
