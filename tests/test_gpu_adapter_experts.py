"""Router, grouped products, the sum behind them and the adapters as they are used
together: the example's block against float64, its gradients against the
formulas, and the whole run captured in a graph.

Tolerances: an e4m3 value is rounded by at most 2^-4 of itself above its block's
smallest steps and by at most 2^-17 of the block's largest below them; bf16 by
2^-8.  Stages downstream of a rounding are compared on the rounded values that
they were given, so each bound is one stage's own: 2^-7 of the sum of
magnitudes for the bf16 hidden values; fp32 sums of n terms n 2^-24 of it.
"""
from __future__ import annotations

import os
import sys

import pytest
import torch

import packed_xor_popcount_amd as bnn

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import adapter_experts  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def signs(wp, k):
    at = torch.arange(k, device=wp.device)
    return (1 - 2 * ((wp[..., at // 64] >> (at % 64)) & 1)).double()


def decoded(q, s, k):
    nb = q.shape[1] // 128
    v = q.view(torch.float8_e4m3fn).double().view(len(q), nb, 128) * torch.exp2(s[:, :nb].double() - 127)[:, :, None]
    return v.view(len(q), -1)[:, :k]


def inputs(tokens, width, adapters, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(tokens, width, generator=g, device=DEV).to(torch.bfloat16)
    ids = torch.randint(-1, adapters, (tokens,), generator=g, device=DEV).to(torch.int32)
    dout = torch.randn(tokens, width, generator=g, device=DEV).to(torch.bfloat16).float()
    return x, ids, dout


@pytest.mark.parametrize("tokens", [1, 5, 130, 700])
def test_block_and_gradients(tokens):
    W, H, E, K, L, R = 200, 330, 7, 2, 4, 5
    block = adapter_experts.AdapterExperts(W, H, E, K, L, R, seed=3)
    x, ids, dout = inputs(tokens, W, L, tokens)
    out, kept = block.forward(x, ids, keep=True)
    served, none = block.forward(x, ids)
    assert none is None and torch.equal(served, out)

    h = bnn.layernorm_fwd(x, block.gamma, block.beta, stats=False)[0]
    h6 = h.double()
    r = kept.routing
    ref = bnn.gemm_f8(*kept.h, *block.shared_q, W).double()
    size = ref.abs()
    for t in range(tokens):
        l = int(ids[t])
        if l >= 0:
            u = block.a[l].double() @ h6[t]
            ref[t] += block.scale[l].double() * (u @ block.b[l].double())
            size[t] += (block.scale[l].double() * (u.abs() @ block.b[l].double().abs()))
        p = torch.softmax(kept.logits[t].double(), 0)
        top, best = torch.sort(kept.logits[t], descending=True, stable=True)
        assert best[:K].tolist() == r.experts[t].tolist()
        w = p[best[:K]] / p[best[:K]].sum()
        for j in range(K):
            e = int(best[j])
            v = (signs(block.up[e], W) @ h6[t]) * block.up_scale[e].double()
            v = v * torch.sigmoid(v)
            ref[t] += w[j] * (signs(block.down[e], H) @ v) * block.down_scale[e].double()
            size[t] += w[j] * v.abs().sum() * block.down_scale[e].double()
    assert ((out.double() - ref).abs() <= 2.0 ** -7 * size).all()

    dl = 0.5
    drouter, da, db, dh = block.gradients(dout, ids, kept, torch.full((1,), dl, device=DEV))
    # the formulas in 64 bits on the kept values
    d6, hq6, y6 = dout.double(), decoded(*kept.h, W), decoded(*kept.d, W)
    rows = y6[r.place.long()]
    dw = (rows * d6[:, None, :]).sum(2)
    dw_size = (rows * d6[:, None, :]).abs().sum(2)
    p = torch.softmax(kept.logits.double(), 1)
    w, at = r.weights.double(), r.experts.long()
    gl = dl * r.slope.double()
    dz = p * (gl - (p * gl).sum(1, keepdim=True))
    dz = dz.scatter_add(1, at, w * (dw - (w * dw).sum(1, keepdim=True)))
    tol = 1e-5 * (gl.abs().max() + dw_size.sum(1, keepdim=True))  # fp32 sums of at most 200 terms: 200 2^-24
    drouter6, dh6 = dz.t() @ hq6, dz @ block.router.double()
    assert ((drouter.double() - drouter6).abs() <= 2 * tol.expand_as(dz).t() @ hq6.abs() + 1e-5).all()
    for l in range(L):
        mine = ids == l
        s, a, b = block.scale[l].double(), block.a[l].double(), block.b[l].double()
        v, u = d6[mine] @ b.t(), kept.u[mine].double()
        assert ((da[l].double() - s * v.t() @ hq6[mine]).abs()
                <= 2e-4 * s * ((d6[mine].abs() @ b.abs().t()).t() @ hq6[mine].abs())).all()
        assert ((db[l].double() - s * u.t() @ d6[mine]).abs() <= 2e-4 * s * (u.abs().t() @ d6[mine].abs())).all()
        dh6[mine] += s * v @ a
    bound = 2 * tol * block.router.double().abs().sum(0) + 1e-4 * dh6.abs().max()
    assert ((dh.double() - dh6).abs() <= bound).all()

    # the experts' outputs in 8 bits: each within 2^-4 of itself, or 2^-17 of its block's largest
    d = bnn.gemm_signw_grouped(torch.nn.functional.silu(bnn.gemm_signw_grouped(
        h, block.up, r.offsets, alpha=block.up_scale, rows=r.rows)).to(torch.bfloat16), block.down, r.offsets,
        alpha=block.down_scale).double()
    assert ((y6 - d).abs() <= 2.0 ** -4 * d.abs() + 2.0 ** -17 * d.abs().amax(1, keepdim=True)).all()


def test_padded_tokens_stay_out():
    """Tokens that are not valid reach no expert and no gradient but the adapters' own."""
    block = adapter_experts.AdapterExperts(128, 192, 6, 3, 3, 4, seed=5)
    x, ids, dout = inputs(90, 128, 3, 8)
    valid = torch.arange(90, device=DEV) % 4 != 1
    x[~valid] = 0
    h = bnn.layernorm_fwd(x, block.gamma, block.beta, stats=False)[0]
    logits = h.float() @ block.router.t()
    r = bnn.route_fwd(logits, 3, valid=valid)
    used = int(r.offsets[-1])
    assert used == 3 * int(valid.sum()) and (r.rows[used:] == -1).all()
    d = torch.full((270, 128), float("nan"), device=DEV)
    t = bnn.gemm_signw_grouped(h, block.up, r.offsets, alpha=block.up_scale, rows=r.rows, dtype=torch.bfloat16)
    bnn.gemm_signw_grouped(t, block.down, r.offsets, alpha=block.down_scale, out=d)
    assert d[used:].isnan().all()
    out = bnn.combine_fwd(d, r.place, weights=r.weights)
    assert torch.isfinite(out).all() and not out[~valid].any()
    dy, dw = bnn.combine_bwd(dout, r.place, weights=r.weights, y=d)
    assert torch.isfinite(dy).all() and not dy[used:].any() and not dw[~valid].any()
    dz = bnn.route_bwd(logits, r.experts, r.weights, r.stats, r.slope, dw, torch.ones(1, device=DEV))
    assert torch.isfinite(dz).all() and not dz[~valid].any()


@pytest.mark.parametrize("tokens", [3, 600])
def test_captured_and_replayed(tokens):
    """The whole forward and backward run in one graph, replayed on new inputs with
    other work in between; two graphs alternate."""
    W, E, K, L, R = 256, 20, 4, 5, 8
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    a = (torch.randn(L, R, W, generator=g, device=DEV) * 0.1).to(torch.bfloat16)
    b = (torch.randn(L, R, W, generator=g, device=DEV) * 0.1).to(torch.bfloat16)
    wp = torch.randint(-2 ** 62, 2 ** 62, (E, W, W // 64), generator=g, device=DEV)

    def run(x, ids, z, dout, dl):
        r = bnn.route_fwd(z, K)
        base, u = bnn.adapter_fwd(x, ids, a, b)
        d = bnn.gemm_signw_grouped(x, wp, r.offsets, rows=r.rows, dtype=torch.bfloat16)
        out = bnn.combine_fwd(d, r.place, r.weights, residual=base)
        q = bnn.quant_f8(d)
        dy, dw = bnn.combine_bwd(dout, r.place, r.weights, q)
        dz = bnn.route_bwd(z, r.experts, r.weights, r.stats, r.slope, dw, dl)
        xq = bnn.quant_f8(x)
        return [*r, base, u, out, dy, dw, dz, *bnn.adapter_bwd(dout, xq, u, ids, a, b)]

    def fresh():
        return (torch.randn(tokens, W, generator=g, device=DEV).to(torch.bfloat16),
                torch.randint(-1, L, (tokens,), generator=g, device=DEV).to(torch.int32),
                torch.randn(tokens, E, generator=g, device=DEV), torch.randn(tokens, W, generator=g, device=DEV)
                .to(torch.bfloat16), torch.rand(1, generator=g, device=DEV))

    graphs = []
    for _ in range(2):
        held = fresh()
        run(*held)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            with torch.cuda.graph(graph, stream=s):
                outs = run(*held)
        torch.cuda.synchronize()
        graphs.append((graph, held, outs))
    for i in range(6):
        graph, held, outs = graphs[i % 2]
        new = fresh()
        want = run(*new)
        for x, y in zip(held, new):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(outs, want):
            assert torch.equal(x, y)


def test_two_streams_at_once():
    block = adapter_experts.AdapterExperts(256, 320, 9, 2, 6, 16, seed=7)
    cases = [inputs(900, 256, 6, 20 + i) for i in range(4)]

    def both(x, ids, dout):
        out, kept = block.forward(x, ids, keep=True)
        return out, *block.gradients(dout, ids, kept, torch.ones(1, device=DEV))

    want = [both(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for s, c in zip(streams, cases):
        with torch.cuda.stream(s):
            got.append(both(*c))
    torch.cuda.synchronize()
    for x, y in zip(want, got):
        # what torch's own products make (router, its gradient) may differ by their kernels' choice
        assert torch.equal(x[0], y[0]) and torch.equal(x[2], y[2]) and torch.equal(x[3], y[3])


def test_example_runs(capsys):
    adapter_experts.main()
    assert "balance loss" in capsys.readouterr().out
