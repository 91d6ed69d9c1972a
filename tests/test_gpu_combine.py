"""The sum of the experts' outputs and its gradient on the GPU against float64.

Tolerances (u = 2^-24): out is a sum of k + 1 terms, one fused multiply and add
each: (k + 1) u sum|terms|.  dy is one product: u |dy|.  dweights sums N exact
terms' products, each thread at most N / 64 + 8, then 9 joins: (N / 64 + 20) u
sum|dout y|.  bf16 outputs add half a step, 2^-8 of the value.  Small whole
numbers are exact throughout.
"""
from __future__ import annotations

import pytest
import torch

import packed_xor_popcount_amd as bnn

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


class Case:
    def __init__(self, seed, T, N, k, ydt, dt, masked=False, pad=0, shift=0, integers=False):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)
        self.T, self.N, self.k, self.integers = T, N, k, integers
        R = T * k
        order = torch.randperm(R, generator=self.g, device=DEV)
        keep = torch.rand(R, generator=self.g, device=DEV) > (0.3 if masked else -1.0)
        self.place = torch.where(keep, order, -2 - order).to(torch.int32).view(T, k)
        self.y = self.rows(R, N, ydt, pad, shift)
        self.dout = self.rows(T, N, dt, pad, shift)
        self.residual = self.rows(T, N, dt, pad, shift)
        w = torch.randint(-3, 4, (T, k), generator=self.g, device=DEV).float() if integers else \
            torch.rand(T, k, generator=self.g, device=DEV)
        self.weights = w

    def rows(self, M, N, dtype, pad, shift):
        """M x N view of a wider buffer whose other places hold NaN."""
        ld = N + pad
        buf = torch.full((shift + M * ld,), float("nan"), dtype=dtype, device=DEV)
        v = buf[shift:].view(M, ld)[:, :N]
        x = torch.randint(-4, 5, (M, N), generator=self.g, device=DEV) if self.integers else \
            torch.randn(M, N, generator=self.g, device=DEV)
        v.copy_(x.to(dtype))
        return v

    def gathered(self, y):
        place = self.place.long()
        has = place >= 0
        rows = y.double()[torch.where(has, place, torch.zeros_like(place))]
        return torch.where(has[:, :, None], rows, torch.zeros_like(rows)), has


def rounding(ref, dtype):
    return ref.abs() * 2.0 ** -8 + 2.0 ** -133 if dtype == torch.bfloat16 else 0.0


def check_fwd(c, weights=True, residual=True, dtype=None):
    w = c.weights if weights else None
    res = c.residual if residual else None
    out = bnn.combine_fwd(c.y, c.place, weights=w, residual=res, dtype=dtype)
    rows, has = c.gathered(c.y)
    terms = rows * (c.weights.double() if weights else has.double())[:, :, None]
    ref, size = terms.sum(1), terms.abs().sum(1)
    if residual:
        ref, size = ref + res.double(), size + res.double().abs()
    err = (out.double() - ref).abs()
    tol = 0.0 if c.integers else (c.k + 1) * U * size * 1.01 + rounding(ref, out.dtype)
    assert (err <= tol).all(), f"{err.max()}"
    return out


SIZES = [(1, 1, 1), (1, 4096, 8), (3, 7, 2), (5, 8, 3), (16, 9, 4), (33, 513, 5), (70, 1000, 6), (130, 2056, 9), (9, 300, 20),
         (2000, 520, 2), (5000, 70, 3), (4, 20000, 2)]


@pytest.mark.parametrize("ydt", list(DT))
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("T,N,k", SIZES)
def test_fwd(T, N, k, ydt, dt):
    for masked, pad, shift, weights, residual in ((False, 0, 0, True, True), (True, 5, 1, True, False),
                                                  (True, 8, 0, False, True), (False, 3, 3, False, False)):
        c = Case(T + N, T, N, k, DT[ydt], DT[dt], masked, pad, shift)
        out = check_fwd(c, weights, residual, DT[dt])
        assert out.dtype == DT[dt]
        check_fwd(Case(T + k, T, N, k, DT[ydt], torch.float32, masked, pad, shift, integers=True), weights, residual,
                  torch.float32)


def check_bwd(c, kept, weights=True):
    y, dyt = c.y, c.y.dtype
    if kept == "f8":
        q, s = bnn.quant_f8(c.y)
        nb = q.shape[1] // 128
        v = q.view(torch.float8_e4m3fn).double().view(len(q), nb, 128)
        y = (v * torch.exp2(s[:, :nb].double() - 127)[:, :, None]).view(len(q), -1)[:, :c.N]
        arg, dyt = (q, s), c.dout.dtype
    else:
        arg = c.y
    w = c.weights if weights else None
    dy, dw = bnn.combine_bwd(c.dout, c.place, weights=w, y=arg)
    assert dy.dtype == dyt
    rows, has = c.gathered(y)
    d = c.dout.double()
    terms = rows * d[:, None, :]
    ref_w = terms.sum(2)
    scale = torch.where(has, c.weights.double() if weights else torch.ones_like(c.weights, dtype=torch.float64),
                        torch.zeros_like(c.weights, dtype=torch.float64))
    ref = torch.empty(c.T * c.k, c.N, dtype=torch.float64, device=DEV)
    at = torch.where(has, c.place, -2 - c.place).long()
    ref[at.reshape(-1)] = (scale[:, :, None] * d[:, None, :]).reshape(-1, c.N)
    if c.integers:
        assert torch.equal(dw.double(), ref_w) and torch.equal(dy.double(), ref)
        return
    tol = (c.N / 64 + 20) * U * terms.abs().sum(2) * 1.01 + 2.0 ** -140
    assert ((dw.double() - ref_w).abs() <= tol).all()
    assert ((dy.double() - ref).abs() <= U * ref.abs() * 1.01 + rounding(ref, dyt)).all()
    assert not dw[~has].any()
    only, none = bnn.combine_bwd(c.dout, c.place, weights=w, rows=c.T * c.k, dtype=dyt)
    assert none is None and torch.equal(only, dy)


@pytest.mark.parametrize("kept", ["fp32", "bf16", "f8"])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("T,N,k", SIZES)
def test_bwd(T, N, k, dt, kept):
    ydt = DT.get(kept, torch.bfloat16)
    for masked, pad, shift, weights in ((False, 0, 0, True), (True, 5, 1, True), (True, 8, 0, False)):
        check_bwd(Case(T + N, T, N, k, ydt, DT[dt], masked, pad, shift), kept, weights)
        check_bwd(Case(T + k, T, N, k, ydt, DT[dt], masked, pad, shift, integers=True), kept, weights)


def test_bwd_against_differences():
    c = Case(3, 4, 13, 2, torch.float32, torch.float32, masked=True)
    dy, dw = bnn.combine_bwd(c.dout, c.place, weights=c.weights, y=c.y)
    d, w6, y6 = c.dout.double(), c.weights.double(), c.y.double()

    def value(y, w):
        rows, has = c.gathered(y)
        return ((rows * torch.where(has, w, torch.zeros_like(w))[:, :, None]).sum(1) * d).sum()

    h = 2.0 ** -10  # the sum is linear in each: no truncation, rounding 2^-52 * 2^8 / h
    for t in range(4):
        for j in range(2):
            e = torch.zeros_like(w6)
            e[t, j] = h
            assert abs((value(y6, w6 + e) - value(y6, w6 - e)) / (2 * h) - dw[t, j]) <= 1e-5
    for r in range(8):
        for n in (0, 7, 12):
            e = torch.zeros_like(y6)
            e[r, n] = h
            assert abs((value(y6 + e, w6) - value(y6 - e, w6)) / (2 * h) - dy[r, n]) <= 1e-5


def test_places_outside_are_skipped():
    """Negative, absent and too large places: nothing is read or written for them."""
    y = torch.full((4, 20), 2.0, device=DEV)
    place = torch.tensor([[0, -1, 4], [3, -7, 2 ** 30], [-1, -2 ** 31, 1]], dtype=torch.int32, device=DEV)
    out = bnn.combine_fwd(y, place)
    assert torch.equal(out, torch.full((3, 20), 2.0, device=DEV))
    dout = torch.ones(3, 20, device=DEV)
    dy, dw = bnn.combine_bwd(dout, place, y=y)
    assert torch.equal(dw, torch.tensor([[40.0, 0, 0], [40.0, 0, 0], [0, 0, 40.0]], device=DEV))
    assert (dy[[0, 1, 3]] == 1).all()
    y[2] = float("nan")  # not named: its values reach nothing
    assert torch.equal(bnn.combine_fwd(y, place), out)


def test_masked_rows_hold_nan():
    c = Case(5, 50, 130, 3, torch.bfloat16, torch.bfloat16, masked=True)
    has = c.place >= 0
    c.y[(-2 - c.place[~has]).long()] = float("nan")
    c.weights[~has] = float("nan")
    assert torch.isfinite(bnn.combine_fwd(c.y, c.place, c.weights)).all()
    dy, dw = bnn.combine_bwd(c.dout, c.place, c.weights, c.y)
    assert torch.isfinite(dy).all() and torch.isfinite(dw).all()


def test_residual_in_place():
    c = Case(6, 40, 100, 2, torch.float32, torch.bfloat16, pad=4)
    ref = bnn.combine_fwd(c.y, c.place, c.weights, c.residual)
    out = bnn.combine_fwd(c.y, c.place, c.weights, c.residual, out=c.residual)
    assert out.data_ptr() == c.residual.data_ptr() and torch.equal(out, ref)


def test_empty():
    y, place = torch.ones(4, 6, device=DEV), torch.zeros(0, 2, dtype=torch.int32, device=DEV)
    assert bnn.combine_fwd(y, place).shape == (0, 6)
    dy, dw = bnn.combine_bwd(torch.zeros(0, 6, device=DEV), place, y=y)
    assert dy.shape == (4, 6) and dw.shape == (0, 2)
    none = torch.zeros(3, 0, device=DEV)
    place = torch.zeros(3, 1, dtype=torch.int32, device=DEV)
    assert bnn.combine_fwd(none, place).shape == (3, 0)
    dy, dw = bnn.combine_bwd(none, place, y=none)
    assert torch.equal(dw, torch.zeros(3, 1, device=DEV))


def test_largest_8_bit_values():
    """Magnitudes that the 8-bit form takes to 2^128: products that fit stay finite, zeros stay zeros."""
    y = torch.zeros(2, 256, device=DEV)
    y[0, 0], y[0, 1], y[1, 130] = 3.3e38, -1e38, 2.0
    q, s = bnn.quant_f8(y)
    dout = torch.zeros(2, 256, device=DEV)
    dout[0, 0], dout[1, 130] = 2.0 ** -20, 4.0
    place = torch.tensor([[0], [1]], dtype=torch.int32, device=DEV)
    _, dw = bnn.combine_bwd(dout, place, y=(q, s))
    assert dw[0, 0].item() == 2.0 ** 108 and dw[1, 0].item() == 8.0


def test_past_32_bit_offsets():
    ld, T, N = (1 << 20) + 8, 2100, 200
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    y = torch.empty(T * ld, dtype=torch.bfloat16, device=DEV).view(T, ld)[:, :N]
    y.copy_(torch.randint(-8, 9, (T, N), generator=g, device=DEV))
    place = torch.randperm(T, generator=g, device=DEV).to(torch.int32).view(T, 1)
    assert torch.equal(bnn.combine_fwd(y, place), y[place.flatten().long()])
    dy, dw = bnn.combine_bwd(y, place, y=y)
    dy2, dw2 = bnn.combine_bwd(y.contiguous(), place, y=y.contiguous())
    assert torch.equal(dy, dy2) and torch.equal(dw, dw2)


def test_side_stream():
    c = Case(9, 3000, 520, 2, torch.bfloat16, torch.bfloat16)
    ref = bnn.combine_fwd(c.y, c.place, c.weights), *bnn.combine_bwd(c.dout, c.place, c.weights, c.y)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = bnn.combine_fwd(c.y, c.place, c.weights), *bnn.combine_bwd(c.dout, c.place, c.weights, c.y)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_bindings_refuse():
    c = Case(1, 4, 8, 2, torch.float32, torch.float32)
    with pytest.raises(ValueError):
        bnn.combine_fwd(c.y, c.place.long())
    with pytest.raises(ValueError):
        bnn.combine_fwd(c.y, c.place, weights=c.weights[:3])
    with pytest.raises(ValueError):
        bnn.combine_fwd(c.y, c.place, residual=c.residual, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bnn.combine_bwd(c.dout, c.place, y=c.y[:, :7])
    with pytest.raises(TypeError):
        bnn.combine_bwd(c.dout, c.place, y=(c.y, c.y))
    with pytest.raises(TypeError):
        bnn.combine_fwd(c.y, c.place, dtype=torch.float16)
