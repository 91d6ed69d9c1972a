"""The example block on the GPU against float64 (the operators together).

Tolerances: an e4m3 value is rounded by at most 2^-4 of itself above its
block's smallest steps, and by at most 2^-10 of the scale below them (the
block's largest value is at least 224 scales, so below 2^-17 of it); a product
of two rounded operands is then off by at most (2 2^-4 + 2^-8) sum|x w| plus
2^-16 max|x| max|w| K for the small values.  The experts' hidden values are
rounded to bf16 (2^-8), everything else is fp32: 2^-7 of the sum of magnitudes.
"""
from __future__ import annotations

import os
import sys

import pytest
import torch

import packed_xor_popcount_amd as bnn

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import expert_block  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def signs(wp, k):
    at = torch.arange(k, device=wp.device)
    return (1 - 2 * ((wp[..., at // 64] >> (at % 64)) & 1)).double()


def f8_tolerance(x, w):
    k = x.shape[1]
    return ((2 * 2.0 ** -4 + 2.0 ** -8) * (x.abs() @ w.abs().t()) * 1.01
            + 2.0 ** -16 * k * x.abs().amax(1, keepdim=True) * w.abs().amax(1))


@pytest.mark.parametrize("tokens", [1, 5, 130])
def test_block(tokens):
    block = expert_block.ExpertBlock(width=200, hidden=330, experts=7, topk=2, seed=3)
    g = torch.Generator(device=DEV)
    g.manual_seed(tokens)
    x = torch.randn(tokens, 200, generator=g, device=DEV).to(torch.bfloat16)
    h = block.norm(x)
    h6 = h.double()
    ref = h6 @ block.shared_weight.double().t()
    assert ((block.shared(h).double() - ref).abs() <= f8_tolerance(h6, block.shared_weight.double())).all()

    weight, chosen = torch.softmax(h.float() @ block.router.t(), dim=1).topk(2, dim=1)
    ref = torch.zeros(tokens, 200, dtype=torch.float64, device=DEV)
    size = torch.zeros(tokens, 200, dtype=torch.float64, device=DEV)
    for t in range(tokens):
        for p, e in zip(weight[t].double(), chosen[t].tolist()):
            u = (signs(block.up[e], 200) @ h6[t]) * block.up_scale[e].double()
            u = u * torch.sigmoid(u)
            ref[t] += p * (signs(block.down[e], 330) @ u) * block.down_scale[e].double()
            size[t] += p * u.abs().sum() * block.down_scale[e].double()
    got = block.experts(h).double()
    assert ((got - ref).abs() <= 2.0 ** -7 * size).all()
    out = block.forward(x).double()
    total = x.double() + block.shared(h).double() + got
    assert ((out - total).abs() <= 2.0 ** -8 * 1.01 * total.abs() + 1e-5).all()


def test_training_step():
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    T, N, K = 150, 260, 200
    x = torch.randn(T, K, generator=g, device=DEV)
    gamma, beta = 1 + 0.1 * torch.randn(K, generator=g, device=DEV), torch.randn(K, generator=g, device=DEV)
    w = torch.randn(N, K, generator=g, device=DEV) * K ** -0.5
    dy = torch.randn(T, N, generator=g, device=DEV)
    y, dx, dgamma, dbeta, dw = expert_block.norm_projection_step(x, gamma, beta, w, dy)
    h = bnn.layernorm_fwd(x, gamma, beta)[0].double()
    assert ((y.double() - h @ w.double().t()).abs() <= f8_tolerance(h, w.double())).all()
    assert ((dw.double() - dy.double().t() @ h).abs() <= f8_tolerance(dy.double().t(), h.t())).all()
    dh = dy.double() @ w.double()
    tol = f8_tolerance(dy.double(), w.double().t())
    assert ((dbeta.double() - dh.sum(0)).abs() <= tol.sum(0)).all()
    x6 = x.double()
    xh = (x6 - x6.mean(1, keepdim=True)) / torch.sqrt(x6.var(1, correction=0, keepdim=True) + 1e-5)
    assert ((dgamma.double() - (dh * xh).sum(0)).abs() <= (tol * xh.abs()).sum(0) * 1.01 + 1e-4).all()
    gr = dh * gamma.double()
    r = 1 / torch.sqrt(x6.var(1, correction=0, keepdim=True) + 1e-5)
    ref = r * (gr - gr.mean(1, keepdim=True) - xh * (gr * xh).mean(1, keepdim=True))
    tg = tol * gamma.double().abs()
    bound = r * (tg + tg.mean(1, keepdim=True) + xh.abs() * (tg * xh.abs()).mean(1, keepdim=True))
    assert ((dx.double() - ref).abs() <= bound * 1.01 + 1e-4).all()


def test_routing_is_a_permutation():
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    rows, offsets, weight, place = expert_block.route(torch.randn(50, 9, generator=g, device=DEV), 3)
    assert offsets[0] == 0 and offsets[-1] == 150 and (offsets.diff() >= 0).all()
    assert torch.equal(place.reshape(-1).sort().values, torch.arange(150, device=DEV))
    assert torch.equal(rows[place.reshape(-1)].view(50, 3), torch.arange(50, device=DEV, dtype=torch.int32)[:, None].expand(50, 3))
