"""The router and its gradient on the GPU against float64.

Tolerances, from the arithmetic (u = 2^-24): z - m is one subtraction (|z - m| u
of the exponent), expf is good to 2 u relative (2 ulp), a row's sum passes at most
E / 64 + 7 additions:
  rel(e)   u (|z - m| + 4)                       of exp(z - m)
  rel(S)   sum_e p rel(e) + u (E / 64 + 8)       of the sum; 1 / S and the product: 2 u
  p        p (rel(e) + rel(S) + 3 u) + 2^-125    weights: the same, S over the choices
  P        sums over T tokens and at most 300 partial sums: (T + 320) u of their value
  loss     E more terms
  dz       p (|g| + |s|) (rel(p) + 4 u) + p (sum_i p |g| (max rel(p) + (E / 64 + 12) u) + inner)
           inner: sum_j |w dw| (k + 8) u, and at the choices w (|dw| + |sum|) 4 u
bf16 outputs add half a step, 2^-8 of the value.  Choices, rows, counts are equal.
"""
from __future__ import annotations

import pytest
import torch

import packed_xor_popcount_amd as bnn

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
TINY = 2.0 ** -125
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def logits(seed, T, E, dtype, pad=0, shift=0, scale=2.0, ties=False):
    """T x E view of a wider buffer whose other places hold NaN."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    ld = E + pad
    buf = torch.full((shift + T * ld,), float("nan"), dtype=dtype, device=DEV)
    v = buf[shift:].view(T, ld)[:, :E]
    z = torch.randn(T, E, generator=g, device=DEV) * scale
    v.copy_((z.round() if ties else z).to(dtype))
    return v


def reference(z, k, valid, normalise):
    z = z.double().cpu()
    T, E = z.shape
    ok = z > -float("inf")
    if valid is not None:
        ok &= valid.cpu().bool()[:, None]
    zz = z.masked_fill(~ok, -float("inf"))
    top, idx = torch.sort(zz, dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    has = top > -float("inf")
    routed = has[:, 0]
    m = torch.where(routed, top[:, 0], torch.zeros(T, dtype=torch.float64))
    ex = torch.exp(zz - m[:, None])
    s = ex.sum(1)
    p = torch.where(routed[:, None], ex / s.clamp(min=1e-300)[:, None], torch.zeros_like(ex))
    et = torch.where(has, torch.exp(top - m[:, None]), torch.zeros_like(top))
    w = et / (et.sum(1, keepdim=True).clamp(min=1e-300) if normalise else s.clamp(min=1e-300)[:, None])
    expert = torch.where(has, idx, torch.full_like(idx, -1))
    key = torch.where(has, idx, torch.full_like(idx, E)).reshape(-1)
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k)
    place = torch.where(key < E, place, -2 - place).view(T, k)
    rows = torch.where(key[order] < E, order // k, torch.full_like(order, -1))
    counts = torch.bincount(key, minlength=E + 1)[:E]
    tv = int(routed.sum())
    slope = counts.double() * E / (k * max(tv, 1) ** 2)
    loss = (slope * p.sum(0)).sum()
    rel_e = U * ((zz - m[:, None]).abs().masked_fill(~ok, 0.0) + 4)
    rel_s = (p * rel_e).sum(1, keepdim=True) + U * (E // 64 + 9)
    rel_p = rel_e + rel_s + 3 * U
    return dict(expert=expert, w=w, place=place, rows=rows, counts=counts, m=m, rs=torch.where(routed, 1 / s, 0 * s),
                slope=slope, loss=loss, p=p, rel_p=rel_p, rel_s=rel_s[:, 0], routed=routed, has=has, tv=tv, ok=ok)


def close(got, ref, tol, what):
    err = (got.double().cpu() - ref).abs()
    assert (err <= tol).all(), f"{what}: {err.max()} at {(err - tol).argmax()}"


def check_fwd(z, k, valid=None, normalise=True, loss=True):
    r = bnn.route_fwd(z, k, valid=valid, normalise=normalise, loss=loss)
    ref = reference(z, k, valid, normalise)
    T, E = z.shape
    for name, want in (("experts", ref["expert"]), ("place", ref["place"]), ("rows", ref["rows"]),
                       ("counts", ref["counts"])):
        assert torch.equal(getattr(r, name).cpu().long(), want), name
    off = torch.cat([torch.zeros(1, dtype=torch.long), torch.cumsum(ref["counts"], 0)])
    assert torch.equal(r.offsets.cpu().long(), off)
    rel = torch.gather(ref["rel_p"], 1, ref["expert"].clamp(min=0))
    if normalise:  # the denominator is a sum over the choices
        rel = 2 * rel.amax(dim=1, keepdim=True) + (k + 8) * U
    close(r.weights, ref["w"], ref["w"] * rel + TINY, "weights")
    close(r.stats[:, 0], ref["m"], 0.0, "maximum")
    close(r.stats[:, 1], ref["rs"], ref["rs"] * (ref["rel_s"] + 2 * U), "1 / sum")
    if loss:
        close(r.slope, ref["slope"], ref["slope"] * 2 * U + TINY, "slope")
        worst = float(ref["rel_p"].masked_fill(~ref["ok"], 0.0).max()) if T else 0.0
        close(r.loss[0], ref["loss"], ref["loss"] * ((T + 320 + E) * U + worst) + TINY, "loss")
    else:
        assert r.slope is None and r.loss is None
    return r, ref


SIZES = [(1, 1, 1), (1, 4, 4), (2, 3, 2), (7, 64, 8), (63, 65, 5), (64, 100, 1), (65, 128, 8), (129, 129, 32), (200, 256, 6),
         (300, 300, 7), (1000, 513, 4), (90, 1024, 8), (1025, 60, 3), (5000, 16, 2), (20000, 33, 2), (40001, 4, 1)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,E,k", SIZES)
def test_fwd(T, E, k, dtype):
    for normalise, pad, shift in ((True, 0, 0), (False, 5, 3)):
        check_fwd(logits(T + E, T, E, DT[dtype], pad, shift), k, normalise=normalise)


@pytest.mark.parametrize("T,E,k", [(5, 8, 3), (100, 64, 8), (700, 130, 6), (3000, 1000, 5)])
def test_ties_go_to_the_lowest_index(T, E, k):
    for scale in (1.0, 0.01):  # 0.01: every logit of a row is 0
        check_fwd(logits(3, T, E, torch.float32, scale=scale, ties=True), k)


@pytest.mark.parametrize("T,E,k", [(1, 5, 2), (130, 64, 8), (2500, 70, 4)])
@pytest.mark.parametrize("which", ["some", "all", "logits", "both"])
def test_masks(T, E, k, which):
    z = logits(8, T, E, torch.float32, pad=2)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    valid = None
    if which in ("some", "both"):
        valid = torch.rand(T, generator=g, device=DEV) > 0.4
    if which == "all":
        valid = torch.zeros(T, dtype=torch.uint8, device=DEV)
    if which in ("logits", "both"):
        few = torch.rand(T, 1, generator=g, device=DEV)
        z.masked_fill_((few < 0.6) & (torch.rand(T, E, generator=g, device=DEV) < 0.97), -float("inf"))
        z[T // 2] = -float("inf")
        z[-1, 0] = torch.finfo(torch.float32).min  # the type's lowest value is a logit like others
    r, ref = check_fwd(z, k, valid)
    if which == "all":
        assert r.loss.item() == 0 and not r.weights.any() and (r.rows == -1).all()
    dw = torch.randn(T, k, generator=g, device=DEV)
    dz = bnn.route_bwd(z, r.experts, r.weights, r.stats, r.slope, dw, torch.ones(1, device=DEV))
    assert torch.isfinite(dz).all() and not dz[~ref["ok"].to(DEV)].any() and not dz[~ref["routed"].to(DEV)].any()


def test_no_tokens():
    z = torch.empty(0, 6, device=DEV)
    r = bnn.route_fwd(z, 2)
    assert not r.offsets.any() and not r.counts.any() and r.loss.item() == 0 and not r.slope.any()
    assert r.experts.shape == (0, 2) and r.rows.shape == (0,)
    assert bnn.route_bwd(z, r.experts, r.weights, r.stats).shape == (0, 6)


def test_nan_and_infinities():
    for T in (40, 3000):
        z = logits(4, T, 20, torch.float32)
        clean = bnn.route_fwd(z, 3)
        z[5, 7] = float("nan")
        z[6, 2] = float("inf")
        z[7] = float("nan")
        valid = torch.ones(T, dtype=torch.bool, device=DEV)
        z[9], valid[9] = float("nan"), False
        r = bnn.route_fwd(z, 3, valid=valid)
        assert not (r.experts[5] == 7).any() and r.experts[6, 0] == 2
        assert (r.experts[7] == -1).all() and (r.experts[9] == -1).all() and not r.weights[9].any()
        assert r.weights[5].isnan().all() and r.weights[6].isnan().all() and r.loss.isnan().all()
        rest = torch.ones(T, dtype=torch.bool, device=DEV)
        rest[[5, 6, 7, 9]] = False
        assert torch.equal(r.experts[rest], clean.experts[rest]) and torch.equal(r.weights[rest], clean.weights[rest])
        where = torch.nonzero(r.place[rest] >= 0)
        assert len(where) == int(rest.sum()) * 3
        assert torch.equal(r.rows[r.place[rest].reshape(-1).long()],
                           torch.nonzero(rest).flatten().to(torch.int32).repeat_interleave(3))
        # a masked token's NaN reaches nothing
        z[5, 7], z[6, 2], z[7] = 0.0, 0.0, 0.0
        assert torch.isfinite(bnn.route_fwd(z, 3, valid=valid).loss).all()


def bwd64(z, r, ref, dw, dl, normalise):
    k = r.experts.shape[1]
    p, has = ref["p"], ref["has"]
    w = r.weights.double().cpu()
    d = torch.where(has, dw.double().cpu(), torch.zeros_like(w)) if dw is not None else torch.zeros_like(w)
    gl = (r.slope.double().cpu() * dl if dl is not None else torch.zeros(z.shape[1], dtype=torch.float64)).expand_as(p)
    at = ref["expert"].clamp(min=0)
    inner = (w * d).sum(1, keepdim=True)
    s = (p * gl).sum(1, keepdim=True) + (0 if normalise else inner)
    add = w * (d - inner if normalise else d)
    dz = (p * (gl - s)).scatter_add(1, at, add)
    size = (w * d).abs().sum(1, keepdim=True)
    rel = ref["rel_p"].masked_fill(~ref["ok"], 0.0)
    tol = p * ((gl.abs() + s.abs()) * (rel + 4 * U)
               + (p * gl).abs().sum(1, keepdim=True) * (rel.amax(1, keepdim=True) + (z.shape[1] // 64 + 12) * U)
               + size * (k + 8) * U)
    tol = tol.scatter_add(1, at, torch.where(has, w * ((d.abs() + inner.abs()) * 4 * U + size * (k + 8) * U), 0 * w))
    return dz, tol + 8 * U * dz.abs() + TINY * (1 + d.abs().amax(1, keepdim=True))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,E,k", SIZES)
def test_bwd(T, E, k, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    for normalise, pad in ((True, 0), (False, 3)):
        z = logits(T * 3 + E, T, E, DT[dtype], pad)
        r = bnn.route_fwd(z, k, normalise=normalise)
        ref = reference(z, k, None, normalise)
        dw = torch.randn(T, k, generator=g, device=DEV)
        for use_w, dl in ((True, 30.0), (True, None), (False, 1.5)):
            got = bnn.route_bwd(z, r.experts, r.weights, r.stats, r.slope if dl else None, dw if use_w else None,
                                torch.tensor([dl], device=DEV) if dl else None, normalise)
            want, tol = bwd64(z, r, ref, dw if use_w else None, dl, normalise)
            assert got.dtype == z.dtype and got.shape == z.shape
            close(got, want, tol + (2.0 ** -8 * want.abs() + 2.0 ** -133 if dtype == "bf16" else 0.0), (normalise, use_w, dl))


@pytest.mark.parametrize("normalise", [True, False])
def test_bwd_against_differences(normalise):
    """d/dz of <dw, weights> + dl loss by central differences in 64 bits, choices and counts held."""
    T, E, k, dl, h = 6, 9, 3, 4.0, 2.0 ** -12
    z = logits(21, T, E, torch.float32)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    dw = torch.randn(T, k, generator=g, device=DEV)
    r = bnn.route_fwd(z, k, normalise=normalise)
    got = bnn.route_bwd(z, r.experts, r.weights, r.stats, r.slope, dw, torch.tensor([dl], device=DEV), normalise).double().cpu()
    at, slope, d = r.experts.long().cpu(), r.slope.double().cpu(), dw.double().cpu()

    def value(x):
        p = torch.softmax(x, 1)
        w = p.gather(1, at)
        if normalise:
            w = w / w.sum(1, keepdim=True)
        return (w * d).sum() + dl * (p * slope).sum()

    z6 = z.double().cpu()
    for t in range(T):
        for e in range(E):
            up, down = z6.clone(), z6.clone()
            up[t, e] += h
            down[t, e] -= h
            diff = (value(up) - value(down)) / (2 * h)
            # third derivatives of a softmax of values below 6: at most 6 * 6 / 6 h^2; rounding 2^-52 * 64 / h
            assert abs(diff - got[t, e]) <= 36 * h * h + 1e-5, (t, e)


def test_equal_bits_on_every_run_and_stream():
    z = logits(5, 9000, 96, torch.bfloat16)
    a = bnn.route_fwd(z, 4)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        runs = [bnn.route_fwd(z, 4) for _ in range(3)]
    s.synchronize()
    for b in runs:
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_bindings_refuse():
    z = torch.zeros(4, 6, device=DEV)
    with pytest.raises(bnn.BnnError):
        bnn.route_fwd(z, 7)
    with pytest.raises(bnn.BnnError):
        bnn.route_fwd(torch.zeros(2, 1025, device=DEV), 2)
    with pytest.raises(ValueError):
        bnn.route_fwd(z, 2, valid=torch.zeros(3, dtype=torch.bool, device=DEV))
    with pytest.raises(ValueError):
        bnn.route_fwd(z.t(), 2)
    with pytest.raises(TypeError):
        bnn.route_fwd(z.half(), 2)
    r = bnn.route_fwd(z, 2)
    with pytest.raises(ValueError):
        bnn.route_bwd(z, r.experts, r.weights[:, :1], r.stats)
    with pytest.raises(TypeError):
        bnn.route_bwd(z, r.experts, r.weights, r.stats, dloss=torch.ones(1, device=DEV))  # no slope
    with pytest.raises(ValueError):
        bnn.route_bwd(z, r.experts, r.weights, r.stats, r.slope, dloss=torch.ones(2, device=DEV))
