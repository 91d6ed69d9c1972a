"""A feed-forward block with sign-weight experts, and a training step of the
norm and projection in front of it.

    python examples/expert_block.py

The block as it is served (ExpertBlock.forward, one token or a prompt):

    h   = layernorm(x)
    out = x + shared(h) + sum_j p_j expert_j(h)

``shared`` is a projection kept at eight bits (quant_f8 + gemm_f8); the experts
are two-layer networks whose weights are packed signs (gemm_signw_grouped),
each token going to its ``topk`` best ones.  Rows are sorted by expert on the
GPU; the sizes of the groups never travel to the host.

``norm_projection_step`` is the training side: loss gradients of y = layernorm(x) W^T
with 8-bit products in all three directions (quant_f8's transposed form makes
the operands of the two gradient products).
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import packed_xor_popcount_amd as bnn  # noqa: E402


def route(logits, topk):
    """(rows, offsets, weights, place): the tokens' rows in the experts' order,
    each expert's range of them, the router's weight of each row, and where
    each token's ``topk`` rows are."""
    experts = logits.shape[1]
    weight, chosen = torch.softmax(logits, dim=1).topk(topk, dim=1)
    expert, order = torch.sort(chosen.reshape(-1), stable=True)
    bounds = torch.arange(experts + 1, device=logits.device)
    offsets = torch.searchsorted(expert, bounds).to(torch.int32)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    rows = (order // topk).to(torch.int32)
    return rows, offsets, weight.reshape(-1)[order].contiguous(), place.view(-1, topk)


class ExpertBlock:
    def __init__(self, width, hidden, experts, topk, device="cuda", seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=g, device=device)

        def signs(n, k):  # packed signs and absmean scales of every expert
            packed, scale = [], []
            for _ in range(experts):
                w = randn(n, k) * k ** -0.5
                packed.append(bnn.pack_signs(w))
                scale.append(w.abs().mean(dim=1))
            return torch.stack(packed), torch.stack(scale)

        self.width, self.hidden, self.topk = width, hidden, topk
        self.gamma, self.beta = 1 + 0.1 * randn(width), 0.1 * randn(width)
        self.router = randn(experts, width) * width ** -0.5
        self.shared_weight = randn(width, width) * width ** -0.5
        self.shared_q = bnn.quant_f8(self.shared_weight)
        self.up, self.up_scale = signs(hidden, width)
        self.down, self.down_scale = signs(width, hidden)

    def norm(self, x):
        return bnn.layernorm_fwd(x, self.gamma, self.beta, stats=False)[0]

    def shared(self, h):
        return bnn.gemm_f8(*bnn.quant_f8(h), *self.shared_q, self.width)

    def experts(self, h):
        rows, offsets, weight, place = route(h.float() @ self.router.t(), self.topk)
        u = bnn.gemm_signw_grouped(h, self.up, offsets, alpha=self.up_scale, rows=rows)
        u = torch.nn.functional.silu(u).to(torch.bfloat16)
        d = bnn.gemm_signw_grouped(u, self.down, offsets, alpha=self.down_scale, row_scale=weight)
        return d[place].sum(dim=1)

    def forward(self, x):
        h = self.norm(x)
        return (x.float() + self.shared(h) + self.experts(h)).to(torch.bfloat16)


def norm_projection_step(x, gamma, beta, w, dy):
    """Output and gradients of y = layernorm(x) w^T for the output's gradient
    dy: (y, dx, dgamma, dbeta, dw)."""
    (n, k), tokens = w.shape, x.shape[0]
    h, mean, rstd = bnn.layernorm_fwd(x, gamma, beta)
    y = bnn.gemm_f8(*bnn.quant_f8(h), *bnn.quant_f8(w), k)
    dh = bnn.gemm_f8(*bnn.quant_f8(dy), *bnn.quant_f8(w, transpose=True), n, dtype=x.dtype)
    dw = bnn.gemm_f8(*bnn.quant_f8(dy, transpose=True), *bnn.quant_f8(h, transpose=True), tokens)
    dx, dgamma, dbeta = bnn.layernorm_bwd(dh, x, mean, rstd, gamma)
    return y, dx, dgamma, dbeta, dw


def main():
    block = ExpertBlock(width=1024, hidden=2048, experts=16, topk=2)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for tokens in (1, 7, 2048):
        x = torch.randn(tokens, 1024, generator=g, device="cuda").to(torch.bfloat16)
        for _ in range(3):
            out = block.forward(x)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(20):
            out = block.forward(x)
        b.record()
        b.synchronize()
        print(f"{tokens} tokens: {tuple(out.shape)}, {a.elapsed_time(b) / 20 * 1e3:.0f} us a pass")
    x = torch.randn(2048, 1024, generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn(2048, 1024, generator=g, device="cuda").to(torch.bfloat16)
    _, dx, dgamma, _, dw = norm_projection_step(x, block.gamma, block.beta, block.shared_weight, dy)
    print(f"gradients: dx {tuple(dx.shape)}, dgamma {tuple(dgamma.shape)}, dw {tuple(dw.shape)}")


if __name__ == "__main__":
    main()
