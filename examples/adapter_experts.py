"""A feed-forward block with routed sign-weight experts and low-rank adapters of
many requests, and the gradients of what is trained in it.

    python examples/adapter_experts.py

    h   = layernorm(x)
    s   = shared(h) + scale_id B_id' A_id h          each row with its request's adapter
    out = s + sum_j p_j expert_j(h)                  p, experts: the router's choices

The experts' packed signs and the shared projection's 8-bit weights are frozen;
trained are the router (with its balance loss) and the adapters.  ``forward``
keeps for ``gradients`` what those need, the large activations (h and the
experts' outputs) in block-scaled 8 bits.
"""
from __future__ import annotations

import os
import sys
from typing import NamedTuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import packed_xor_popcount_amd as bnn  # noqa: E402


class Kept(NamedTuple):
    h: tuple        # 8 bits
    d: tuple        # 8 bits: the experts' outputs
    u: torch.Tensor
    logits: torch.Tensor
    routing: bnn.Routing


class AdapterExperts:
    def __init__(self, width, hidden, experts, topk, adapters, rank, device="cuda", seed=0):
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

        self.width, self.topk = width, topk
        self.gamma, self.beta = 1 + 0.1 * randn(width), 0.1 * randn(width)
        self.router = randn(experts, width) * width ** -0.5
        self.shared_weight = randn(width, width) * width ** -0.5
        self.shared_q = bnn.quant_f8(self.shared_weight)
        self.up, self.up_scale = signs(hidden, width)
        self.down, self.down_scale = signs(width, hidden)
        self.a = (randn(adapters, rank, width) * width ** -0.5).to(torch.bfloat16)
        self.b = (randn(adapters, rank, width) * rank ** -0.5).to(torch.bfloat16)
        self.scale = 0.5 + torch.rand(adapters, generator=g, device=device)

    def forward(self, x, ids, valid=None, keep=False):
        """(out, what gradients takes or None); ``ids``: each row's adapter, -1 for none."""
        h = bnn.layernorm_fwd(x, self.gamma, self.beta, stats=False)[0]
        hq = bnn.quant_f8(h)
        s = bnn.gemm_f8(*hq, *self.shared_q, self.width)
        s, u = bnn.adapter_fwd(h, ids, self.a, self.b, scale=self.scale, base=s, out=s)
        logits = h.float() @ self.router.t()
        r = bnn.route_fwd(logits, self.topk, valid=valid, loss=keep)
        t = bnn.gemm_signw_grouped(h, self.up, r.offsets, alpha=self.up_scale, rows=r.rows)
        t = torch.nn.functional.silu(t).to(torch.bfloat16)
        d = bnn.gemm_signw_grouped(t, self.down, r.offsets, alpha=self.down_scale)
        out = bnn.combine_fwd(d, r.place, weights=r.weights, residual=s, out=s)
        return out, Kept(hq, bnn.quant_f8(d), u, logits, r) if keep else None

    def gradients(self, dout, ids, kept, dloss):
        """(drouter, da, db, dh): of the router's weights, of the adapters, and
        what reaches h through both; ``dloss`` is the balance loss's gradient."""
        dy = dout.to(torch.bfloat16)
        r = kept.routing
        _, dw = bnn.combine_bwd(dy, r.place, weights=r.weights, y=kept.d)
        dz = bnn.route_bwd(kept.logits, r.experts, r.weights, r.stats, r.slope, dw, dloss)
        q, s = kept.h
        blocks = q.shape[1] // 128
        h = q.view(torch.float8_e4m3fn).float().view(len(q), blocks, 128)
        h = torch.ldexp(h, s[:, :blocks].int().unsqueeze(2) - 127).view(len(q), -1)[:, :self.width]
        dh, da, db = bnn.adapter_bwd(dy, kept.h, kept.u, ids, self.a, self.b, scale=self.scale,
                                     base=dz @ self.router)
        return dz.t() @ h, da, db, dh


def main():
    block = AdapterExperts(width=1024, hidden=2048, experts=16, topk=2, adapters=8, rank=16)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for tokens in (1, 7, 2048):
        x = torch.randn(tokens, 1024, generator=g, device="cuda").to(torch.bfloat16)
        ids = torch.randint(-1, 8, (tokens,), generator=g, device="cuda").to(torch.int32)
        for _ in range(3):
            out, _ = block.forward(x, ids)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(20):
            out, _ = block.forward(x, ids)
        b.record()
        b.synchronize()
        print(f"{tokens} tokens: {tuple(out.shape)}, {a.elapsed_time(b) / 20 * 1e3:.0f} us a pass")
    out, kept = block.forward(x, ids, keep=True)
    drouter, da, db, _ = block.gradients(torch.randn(out.shape, generator=g, device="cuda"), ids, kept,
                                         torch.full((1,), 0.01, device="cuda"))
    print(f"balance loss {kept.routing.loss.item():.3f}; gradients: router {tuple(drouter.shape)}, "
          f"adapters {tuple(da.shape)} and {tuple(db.shape)}")


if __name__ == "__main__":
    main()
