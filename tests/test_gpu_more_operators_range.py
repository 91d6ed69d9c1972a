"""Router, sum of the experts' outputs and adapters at the ends of fp32's range:
magnitudes that overflow on the way only, infinities and NaN.

Every value below is a power of two (or a short sum of them), so that products
and sums are exact and results are equal."""
from __future__ import annotations

import math

import pytest
import torch

import packed_xor_popcount_amd as bnn

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
INF = math.inf


# 1, 8 and 9 columns of a row, the last of a block, three blocks; few tokens (four waves
# each) and many (one wave each)
@pytest.mark.parametrize("T", [3, 4100])
@pytest.mark.parametrize("N", [1, 8, 9, 128, 300])
def test_sum_of_experts_from_8_bits_takes_large_gradients(T, N):
    y = torch.zeros(T, N, device=DEV)
    y[:, N - 1], y[:, N // 2] = 2.0 ** -20, -2.0 ** -19
    dout = torch.full((T, N), 2.0 ** 120, device=DEV)
    place = torch.arange(T, dtype=torch.int32, device=DEV).flip(0).view(T, 1).contiguous()
    _, want = bnn.combine_bwd(dout, place, y=y)
    dy, dw = bnn.combine_bwd(dout, place, y=bnn.quant_f8(y))
    assert torch.isfinite(want).all()
    assert torch.equal(dw, want) and torch.equal(dy, dout)


@pytest.mark.parametrize("byte", [0, 1, 60, 127, 200, 245, 246, 247, 250, 255])
def test_sum_of_experts_from_8_bits_at_every_scale(byte):
    """448, its negative and the smallest value under a scale of 2^(byte - 127), each times the power
    of two that takes the product to about 1 (or as near as fp32's range lets it)."""
    q = torch.zeros(3, 128, dtype=torch.float8_e4m3fn, device=DEV)
    q[0, 5], q[1, 127], q[2, 64] = 448.0, -448.0, 2.0 ** -9
    s = torch.zeros(3, 4, dtype=torch.uint8, device=DEV)
    s[:, 0] = byte
    up = max(-126, min(127, 127 - byte - 8))
    dout = torch.zeros(3, 128, device=DEV)
    dout[:2] = 2.0 ** up
    up2 = max(-126, min(127, 127 - byte + 9))
    dout[2] = 2.0 ** up2
    place = torch.arange(3, dtype=torch.int32, device=DEV).view(3, 1)
    _, dw = bnn.combine_bwd(dout, place, y=(q.view(torch.uint8), s))
    want = [448 * 2.0 ** (byte - 127 + up), -448 * 2.0 ** (byte - 127 + up), 2.0 ** (byte - 127 - 9 + up2)]
    assert dw.flatten().tolist() == want


@pytest.mark.parametrize("big", [2.0 ** 126, 2.0 ** 127, -2.0 ** 127, 3.38e38])
@pytest.mark.parametrize("T", [2, 300])
def test_gradient_from_8_bits_leaves_zeros_beside_large_factors(big, T):
    """A block of the largest scale byte: its zeros give zeros whatever finite value they meet."""
    x = torch.zeros(T, 130, device=DEV)
    x[0, 3], x[1, 3], x[1, 128] = 3.3e38, -3.3e38, 2.0 ** -100
    q = bnn.quant_f8(x)
    assert int(q[1][0, 0]) == 247
    ids = torch.zeros(T, dtype=torch.int32, device=DEV)
    ids[1] = 1
    a = torch.ones(2, 2, 130, dtype=torch.bfloat16, device=DEV)
    b = torch.ones(2, 2, 8, dtype=torch.bfloat16, device=DEV)
    b[:, 1] = 0
    dy = torch.zeros(T, 8, dtype=torch.bfloat16, device=DEV)
    dy[:2, 0] = big
    v = dy[0, 0].item()
    for dx in (True, False):
        _, da, _ = bnn.adapter_bwd(dy, q, torch.zeros(T, 2, device=DEV), ids, a, b, dx=dx)
        want = torch.zeros(2, 2, 130, device=DEV)
        want[0, 0, 3], want[1, 0, 3] = math.copysign(INF, v), -math.copysign(INF, v)
        want[1, 0, 128] = v * 2.0 ** -100
        assert torch.equal(da, want)


@pytest.mark.parametrize("T", [40, 3000])
@pytest.mark.parametrize("E", [5, 20, 600])
@pytest.mark.parametrize("normalise", [True, False])
def test_router_tokens_of_nan_have_no_expert(T, E, normalise):
    """NaN alone, or beside -inf: no expert is left, so zeros everywhere but in the loss."""
    g = torch.Generator(device=DEV)
    g.manual_seed(T + E)
    z = torch.randn(T, E, generator=g, device=DEV)
    z[3], z[17] = math.nan, -INF
    z[17, 2] = math.nan
    r = bnn.route_fwd(z, 3, normalise=normalise)
    dw = torch.randn(T, 3, generator=g, device=DEV)
    dz = bnn.route_bwd(z, r.experts, r.weights, r.stats, r.slope, dw, torch.ones(1, device=DEV), normalise)
    for t in (3, 17):
        assert (r.experts[t] == -1).all() and not r.weights[t].any() and (r.place[t] < -1).all()
        assert torch.equal(r.stats[t], torch.zeros(2, device=DEV))
        assert torch.equal(dz[t], torch.zeros(E, device=DEV))
    rest = torch.ones(T, dtype=torch.bool, device=DEV)
    rest[[3, 17]] = False
    assert torch.isfinite(dz[rest]).all() and r.loss.isnan().all()


@pytest.mark.parametrize("dl", [math.nan, INF])
def test_router_gradient_is_zero_without_an_expert(dl):
    z = torch.randn(50, 12, device=DEV)
    z[4] = -INF
    valid = torch.ones(50, dtype=torch.bool, device=DEV)
    valid[9] = False
    r = bnn.route_fwd(z, 2, valid=valid)
    dz = bnn.route_bwd(z, r.experts, r.weights, r.stats, r.slope, None, torch.full((1,), dl, device=DEV))
    assert not dz[[4, 9]].any() and not torch.isfinite(dz[0]).all()


# one launch (few rows), two launches, ranks of one operand, of two and of four
ADAPTERS = [(1, 16), (40, 5), (40, 20), (300, 16), (300, 30), (300, 40), (300, 70)]


@pytest.mark.parametrize("T,r", ADAPTERS)
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_adapters_scale_the_sum(T, r, out):
    """scale * u leaves fp32's range, scale * sum u b does not."""
    K, N = 136, 260
    x = torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)
    x[:, 3] = 2.0 ** 120
    a = torch.zeros(2, r, K, dtype=torch.bfloat16, device=DEV)
    a[0, :, 3] = 1.0
    a[1, :, 3] = 2.0 ** -126
    b = torch.zeros(2, r, N, dtype=torch.bfloat16, device=DEV)
    b[0, r - 1], b[1, r - 1] = 2.0 ** -60, 2.0 ** 120
    x[1::2, 3] = 2.0 ** 20
    scale = torch.tensor([2.0 ** 30, 2.0 ** -40], device=DEV)
    ids = (torch.arange(T, device=DEV) % 2).to(torch.int32)
    base = torch.full((T, N), 2.0 ** 80, dtype=out, device=DEV)
    base[1::2] = 2.0 ** -30
    got, u = bnn.adapter_fwd(x, ids, a, b, scale=scale, base=base)
    assert u[0, 0].item() == 2.0 ** 120 and (T == 1 or u[1, 0].item() == 2.0 ** -106)
    want = torch.full((T, N), 2.0 ** 90 + 2.0 ** 80, device=DEV).to(out)
    want[1::2] = 2.0 ** -26 + 2.0 ** -30
    assert torch.equal(got, want.to(out))
    got, _ = bnn.adapter_fwd(x, ids, a, b, scale=scale, dtype=out)
    assert got[0, 0].item() == 2.0 ** 90 and (T == 1 or got[1, 0].item() == 2.0 ** -26)
    # the gradient by x is the same product: dy in x's place, b and a in a's and b's
    got, _, _ = bnn.adapter_bwd(x, None, None, ids, b, a, scale=scale, base=base, params=False)
    assert torch.equal(got, want.to(out))
    q, u0 = torch.zeros(T, N, dtype=torch.bfloat16, device=DEV), torch.zeros(T, r, device=DEV)
    got, _, _ = bnn.adapter_bwd(x, q, u0, ids, b, a, scale=scale, base=base)
    assert torch.equal(got, want.to(out))


@pytest.mark.parametrize("T,r", ADAPTERS)
def test_infinite_factors_give_infinities(T, r):
    """An infinity times a number is an infinity, times zero NaN; columns without one are as before."""
    K, N = 140, 261
    g = torch.Generator(device=DEV)
    g.manual_seed(r)
    x = torch.randint(1, 3, (T, K), generator=g, device=DEV).to(torch.bfloat16)
    a = torch.randint(1, 3, (2, r, K), generator=g, device=DEV).to(torch.bfloat16)
    b = torch.randint(1, 3, (2, r, N), generator=g, device=DEV).to(torch.bfloat16)
    ids = (torch.arange(T, device=DEV) // 20 % 2).to(torch.int32)
    base = torch.randint(-4, 5, (T, N), generator=g, device=DEV).float()
    clean, u = bnn.adapter_fwd(x, ids, a, b, base=base)
    assert (u > 0).all()
    bad = b.clone()
    bad[0, r - 1, 0], bad[0, 0, 7], bad[0, r // 2, 260] = INF, -INF, INF
    bad[1, r - 1, 130], bad[1, 0, 255] = -INF, math.nan
    want = clean.clone()
    one, two = ids == 0, ids == 1
    want[one, 0], want[one, 7], want[one, 260] = INF, -INF, INF
    want[two, 130], want[two, 255] = -INF, math.nan
    got, u2 = bnn.adapter_fwd(x, ids, a, bad, base=base)
    assert torch.equal(u, u2)
    assert torch.equal(got.nan_to_num(7.5, 1e30, -1e30), want.nan_to_num(7.5, 1e30, -1e30))
    # u = 0 meets the infinity: NaN
    zero = x.clone()
    zero[0] = 0
    got, _ = bnn.adapter_fwd(zero, ids, a, bad, base=base)
    assert got[0, [0, 7, 260]].isnan().all() and torch.equal(got[0, 8:260], base[0, 8:260])
    # an infinite u: infinities in every column
    x2 = x.clone()
    x2[0, 5] = INF
    got, u2 = bnn.adapter_fwd(x2, ids, a, b, base=base)
    assert (u2[0] == INF).all() and (got[0] == INF).all() and torch.equal(got[1:], clean[1:])


@pytest.mark.parametrize("kept", ["bf16", "f8"])
@pytest.mark.parametrize("T,r", ADAPTERS + [(1500, 12)])
def test_infinite_gradients_give_infinities(T, r, kept):
    """Infinities in the output's gradient and in the kept input: no NaN where the sum has none."""
    K, N = 261, 140
    g = torch.Generator(device=DEV)
    g.manual_seed(r)
    x = torch.randint(1, 3, (T, K), generator=g, device=DEV).to(torch.bfloat16)
    dy = torch.randint(1, 3, (T, N), generator=g, device=DEV).to(torch.bfloat16)
    a = torch.randint(1, 3, (2, r, K), generator=g, device=DEV).to(torch.bfloat16)
    b = torch.randint(1, 3, (2, r, N), generator=g, device=DEV).to(torch.bfloat16)
    u = torch.randint(1, 3, (T, r), generator=g, device=DEV).float()
    ids = (torch.arange(T, device=DEV) // 20 % 2).to(torch.int32)

    def call(x, dy, a=a, base=None):
        return bnn.adapter_bwd(dy, bnn.quant_f8(x) if kept == "f8" else x, u, ids, a, b)

    dx0, da0, db0 = call(x, dy)
    last = int(torch.nonzero(ids == ids[-1])[-1])
    l = int(ids[last])
    bad = dy.clone()
    bad[last, 3] = INF
    dx, da, db = call(x, bad)  # v is infinite, so dx and da of the row's adapter are
    want = db0.clone()
    want[l, :, 3] = INF
    assert torch.equal(db, want)
    rest = torch.arange(T, device=DEV) != last
    assert (dx[last] == INF).all() and torch.equal(dx[rest], dx0[rest])
    want = da0.clone()
    want[l] = INF
    assert torch.equal(da, want)
    if kept == "bf16":
        bad = x.clone()
        bad[last, 0], bad[last, 260] = INF, -INF
        dx, da, db = call(bad, dy)
        want = da0.clone()
        want[l, :, 0], want[l, :, 260] = INF, -INF
        assert torch.equal(da, want) and torch.equal(dx, dx0) and torch.equal(db, db0)
    bad = a.clone()
    bad[l, r - 1, 9], bad[l, 0, 260] = INF, -INF
    dx, da, db = call(x, dy, a=bad)
    want = dx0.clone()
    want[ids == l, 9], want[ids == l, 260] = INF, -INF
    assert torch.equal(dx, want) and torch.equal(da, da0) and torch.equal(db, db0)


@pytest.mark.parametrize("T", [3, 400])
@pytest.mark.parametrize("K,N", [(0, 9), (9, 0), (0, 0)])
def test_gradient_of_empty_sides(T, K, N):
    """No columns on one side: its gradients are empty, the other's as for any width."""
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    dy = torch.randint(-2, 3, (T, N), generator=g, device=DEV).to(torch.bfloat16)
    x = torch.randint(-2, 3, (T, K), generator=g, device=DEV).to(torch.bfloat16)
    u = torch.randint(-2, 3, (T, 2), generator=g, device=DEV).float()
    base = torch.randint(-2, 3, (T, K), generator=g, device=DEV).float()
    ids = (torch.arange(T, device=DEV) % 3 - 1).to(torch.int32)
    a, b = (torch.ones(2, 2, n, dtype=torch.bfloat16, device=DEV) for n in (K, N))
    dx, da, db = bnn.adapter_bwd(dy, x, u, ids, a, b, base=base)
    assert torch.equal(dx, base) and da.shape == (2, 2, K) and db.shape == (2, 2, N) and not da.any()
    for l in range(2):
        mine = ids == l
        assert torch.equal(db[l], u[mine].t() @ dy[mine].float())


def test_most_adapters():
    """The largest number of adapters: an id and a row's place in its chunk share a word."""
    L, T = 2 ** 20 - 1, 1000
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    ids = torch.randint(-1, L, (T,), generator=g, device=DEV).to(torch.int32)
    ids[::7], ids[3::7] = L - 1, 0
    a, b = (torch.randint(-3, 4, (L, 1, n), generator=g, device=DEV).to(torch.bfloat16) for n in (2, 3))
    x = torch.randint(-3, 4, (T, 2), generator=g, device=DEV).to(torch.bfloat16)
    for rows in (T, 30):
        out, u = bnn.adapter_fwd(x[:rows], ids[:rows], a, b)
        l, has = ids[:rows].long().clamp(min=0), (ids[:rows] >= 0).float()[:, None]
        want = (a[l, 0].float() * x[:rows].float()).sum(1, keepdim=True) * has
        assert torch.equal(u, want) and torch.equal(out, want * b[l, 0].float())


def test_sum_in_place_with_another_stride_is_refused():
    buf = torch.zeros(200, device=DEV)
    residual, out = buf.as_strided((8, 10), (12, 1)), buf.as_strided((8, 10), (20, 1))
    y, place = torch.ones(8, 10, device=DEV), torch.arange(8, dtype=torch.int32, device=DEV).view(8, 1)
    with pytest.raises(bnn.BnnError):
        bnn.combine_fwd(y, place, residual=residual, out=out)
    assert not buf.any()
