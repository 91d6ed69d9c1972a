"""Timing cases of the operators beside the grouped sign-weight products: the
router with its balance loss, the sum of the experts' outputs and the low-rank
adapters of many requests, each with its gradient; the gradients read what the
forward pass kept in 16, 32 or block-scaled 8 bits.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, rounded once at the end) or, with ``own`` set, through the package's
entry points; ``exact`` computes it in 64 bits from the definition.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "bf16": 2, "f8": 1}
BLOCK = 128  # elements under one scale of the 8-bit form


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # four sequences that decode: latency; no loss is wanted
        {"name": "route_decode", "op": "route_fwd", "tokens": 4, "experts": 64, "k": 8, "dtype": "bf16", "pad": 0,
         "masked": False, "normalise": True, "loss": False},
        # a training batch whose sequences are padded
        {"name": "route_train", "op": "route_fwd", "tokens": 16384, "experts": 128, "k": 8, "dtype": "fp32", "pad": 0,
         "masked": True, "normalise": True, "loss": True},
        # gradient of an odd batch, logits cut out of a wider product, experts switched off for some tokens
        {"name": "route_bwd_odd", "op": "route_bwd", "tokens": 3001, "experts": 60, "k": 4, "dtype": "bf16", "pad": 5,
         "masked": True, "normalise": False, "loss": True},
        # gradient of the training batch
        {"name": "route_bwd_train", "op": "route_bwd", "tokens": 16384, "experts": 128, "k": 8, "dtype": "fp32", "pad": 0,
         "masked": True, "normalise": True, "loss": True},
        # eight experts' outputs of each decoding sequence onto its residual stream
        {"name": "combine_decode", "op": "combine_fwd", "tokens": 4, "n": 4096, "k": 8, "dtype": "fp32", "out": "bf16",
         "masked": False, "weights": True, "residual": True},
        # a prompt batch, two experts a token
        {"name": "combine_prompt", "op": "combine_fwd", "tokens": 8192, "n": 4096, "k": 2, "dtype": "bf16", "out": "bf16",
         "masked": False, "weights": True, "residual": True},
        # gradient of an odd batch at the edge layer's width
        {"name": "combine_bwd_odd", "op": "combine_bwd", "tokens": 301, "n": 1000, "k": 3, "dtype": "fp32", "out": "fp32",
         "masked": True},
        # gradient of a training batch that kept the experts' outputs in 8 bits
        {"name": "combine_bwd_train", "op": "combine_bwd", "tokens": 8192, "n": 4096, "k": 4, "dtype": "f8", "out": "bf16",
         "masked": True},
        # 32 decoding sequences, each with one of 24 adapters, beside a 4096 x 4096 projection
        {"name": "adapter_decode", "op": "adapter_fwd", "rows": 32, "k": 4096, "n": 4096, "rank": 16, "adapters": 24,
         "runs": 1, "out": "fp32", "pad": 0},
        # prompts of ragged lengths with eight adapters beside the feed-forward layer's projection
        {"name": "adapter_prompt", "op": "adapter_fwd", "rows": 4096, "k": 4096, "n": 11008, "rank": 16, "adapters": 8,
         "runs": 300, "out": "bf16", "pad": 0},
        # gradient of a small odd batch with an odd rank
        {"name": "adapter_bwd_odd", "op": "adapter_bwd", "rows": 777, "k": 1000, "n": 1501, "rank": 12, "adapters": 5,
         "runs": 60, "kept": "bf16", "out": "fp32", "pad": 3},
        # training step of four adapters at once, the input kept in 8 bits
        {"name": "adapter_bwd_train", "op": "adapter_bwd", "rows": 8192, "k": 4096, "n": 4096, "rank": 32, "adapters": 4,
         "runs": 1000, "kept": "f8", "out": "bf16", "pad": 0},
    ]


def _log(rng, lo, hi):
    """A whole number, its logarithm spread evenly over [lo, hi]; a third are rounded to a multiple of 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.34 and v >= 64:
        v -= v % 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["route_fwd", "route_bwd", "combine_fwd", "combine_bwd", "adapter_fwd", "adapter_fwd",
                     "adapter_bwd", "adapter_bwd"])
    if op.startswith("route"):
        experts = _log(rng, 4, 256)
        return {"op": op, "tokens": _log(rng, 1, min(16384, 16384 * 128 // experts)), "experts": experts,
                "k": rng.randint(1, min(8, experts)), "dtype": rng.choice(["bf16", "fp32"]),
                "pad": rng.choice([0, 0, 8, 5]), "masked": rng.random() < 0.5, "normalise": rng.random() < 0.5,
                "loss": op == "route_bwd" or rng.random() < 0.6}
    if op.startswith("combine"):
        n, k = _log(rng, 64, 8192), rng.choice([1, 2, 3, 4, 6, 8])
        case = {"op": op, "tokens": _log(rng, 1, min(8192, 36000000 // (n * k))), "n": n, "k": k,
                "dtype": rng.choice(["bf16", "fp32"]), "out": rng.choice(["bf16", "fp32"]), "masked": rng.random() < 0.4}
        if op == "combine_fwd":
            case["weights"], case["residual"] = rng.random() < 0.7, rng.random() < 0.5
        elif rng.random() < 0.4:
            case["dtype"] = "f8"
        return case
    k, n = _log(rng, 64, 11008), _log(rng, 64, 11008)
    case = {"op": op, "rows": _log(rng, 1, max(1, min(8192, 8192 * 4096 // (k + n)))), "k": k, "n": n,
            "rank": rng.choice([4, 8, 16, 16, 32, 32, 64, rng.randint(1, 64)]), "adapters": _log(rng, 1, 32),
            "runs": rng.choice([1, 1, 40, 500]), "out": rng.choice(["bf16", "fp32"]), "pad": rng.choice([0, 0, 8, 3])}
    if op == "adapter_bwd":
        case["kept"] = rng.choice(["bf16", "f8"])
        case["rows"] = max(1, case["rows"] // 2)
    return case


# ---------------------------------------------------------------------------
# inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _rows_of(g, rows, cols, dtype, pad):
    """(rows, cols) of a wider matrix: its rows are cols + pad apart."""
    return _randn(g, rows, cols + pad).to(dtype)[:, :cols]


def _quantised(v):
    """Block-scaled e4m3 form of real rows: bytes (rows, 128 * blocks), zeros
    past K, and scale bytes (rows, 4 * ceil(blocks / 4))."""
    v = v.float()
    rows, k = v.shape
    nb = -(-k // BLOCK)
    x = torch.nn.functional.pad(v, (0, nb * BLOCK - k)).reshape(rows, nb, BLOCK)
    mant, ex = torch.frexp(x.abs().amax(dim=2))
    e = torch.where(mant > 0.875, ex - 8, ex - 9)  # 448 = 0.875 * 2^9
    e = torch.where(mant == 0, torch.zeros_like(e), e.clamp(min=-127))
    q = torch.ldexp(x, -e.unsqueeze(2)).to(torch.float8_e4m3fn)
    s = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, -nb % 4))
    return q.reshape(rows, nb * BLOCK).view(torch.uint8), s


def _dequantised(q, s, k):
    rows, nb = q.shape[0], q.shape[1] // BLOCK
    v = q.view(torch.float8_e4m3fn).float().reshape(rows, nb, BLOCK)
    return torch.ldexp(v, s[:, :nb].to(torch.int32).unsqueeze(2) - 127).reshape(rows, nb * BLOCK)[:, :k]


def _logits(g, case):
    """Router logits, some experts popular; where the batch is masked: padded
    tokens, tokens for which most or all experts are switched off."""
    t, e = case["tokens"], case["experts"]
    z = _randn(g, t, e + case["pad"]) * 1.5 + _randn(g, 1, e + case["pad"])
    valid = None
    if case["masked"]:
        u = torch.rand(t, 1, generator=g, device=DEV)
        off = torch.rand(t, e + case["pad"], generator=g, device=DEV) < 0.9
        z = z.masked_fill((u < 0.05) & off, -math.inf).masked_fill(u > 0.99, -math.inf)
        valid = torch.rand(t, generator=g, device=DEV) > 0.1
    return z.to(DTYPES[case["dtype"]])[:, :e], valid


def _places(g, case, experts=32):
    """Where each token's k rows lie among the rows sorted by expert; rows of
    tokens that are left out come last (place = -2 - row)."""
    t, k = case["tokens"], case["k"]
    chosen = (_randn(g, t, experts) + _randn(g, 1, experts)).topk(k, dim=1).indices
    if case["masked"]:
        chosen = chosen.masked_fill(torch.rand(t, 1, generator=g, device=DEV) < 0.1, experts)
    expert, order = torch.sort(chosen.reshape(-1), stable=True)
    row = torch.arange(t * k, device=DEV)
    place = torch.empty_like(order)
    place[order] = torch.where(expert < experts, row, -2 - row)
    return place.view(t, k).to(torch.int32)


def _ids(g, case):
    """The adapter of each row: ``runs`` rows in a row belong to one request on
    average; a request in eight has none (-1)."""
    rows, n = case["rows"], case["adapters"]
    requests = max(1, round(rows / case["runs"]))
    bounds = torch.sort(torch.randint(0, rows, (requests,), generator=g, device=DEV)).values
    request = torch.searchsorted(bounds, torch.arange(rows, device=DEV), right=True) if case["runs"] > 1 else \
        torch.arange(rows, device=DEV)
    ids = torch.randint(0, n, (max(requests, rows) + 1,), generator=g, device=DEV)
    ids[torch.rand(ids.shape, generator=g, device=DEV) < 0.125] = -1
    return ids[request].to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    st = {"case": dict(case)}
    if op.startswith("route"):
        st["logits"], st["valid"] = _logits(g, case)
        if op == "route_bwd":
            (st["experts"], st["weights"], _, _, _, _, st["stats"], st["slope"], _) = _route_plain(
                st["logits"], st["valid"], case["k"], case["normalise"])
            st["dweights"] = _randn(g, case["tokens"], case["k"])
            st["dloss"] = torch.full((1,), 0.01 * case["tokens"], device=DEV)
    elif op.startswith("combine"):
        t, n, k = case["tokens"], case["n"], case["k"]
        st["place"] = _places(g, case)
        y = _randn(g, t * k, n) * torch.exp(0.5 * _randn(g, t * k, 1))
        st["y"] = _quantised(y) if case["dtype"] == "f8" else y.to(DTYPES[case["dtype"]])
        st["weights"] = torch.softmax(_randn(g, t, k), dim=1) if case.get("weights", True) else None
        if op == "combine_fwd":
            st["residual"] = _randn(g, t, n).to(DTYPES[case["out"]]) if case["residual"] else None
        else:
            st["dout"] = _randn(g, t, n).to(DTYPES[case["out"]])
    else:
        t, k, n, r, na = case["rows"], case["k"], case["n"], case["rank"], case["adapters"]
        st["ids"] = _ids(g, case)
        ids = st["ids"].tolist()
        st["present"] = [i for i in range(na) if i in set(ids)]
        st["a"] = (_randn(g, na, r, k) * k ** -0.5).to(torch.bfloat16)
        st["b"] = (_randn(g, na, r, n) * r ** -0.5).to(torch.bfloat16)
        st["scale"] = 0.5 + torch.rand(na, generator=g, device=DEV)
        st["x"] = _rows_of(g, t, k, torch.bfloat16, case["pad"])
        if op == "adapter_fwd":
            st["base"] = _rows_of(g, t, n, DTYPES[case["out"]], case["pad"])
        else:
            st["dy"] = _rows_of(g, t, n, torch.bfloat16, case["pad"])
            st["base"] = _rows_of(g, t, k, DTYPES[case["out"]], case["pad"])
            st["u"] = torch.zeros(t, r, device=DEV)
            for i in st["present"]:
                at = st["ids"] == i
                st["u"][at] = st["x"][at].float() @ st["a"][i].float().t()
            if case["kept"] == "f8":
                st["x"] = _quantised(st["x"])
    return st


# ---------------------------------------------------------------------------
# the operators

def _run_own(st):
    import packed_xor_popcount_amd as bnn
    case = st["case"]
    op = case["op"]
    if op == "route_fwd":
        r = bnn.route_fwd(st["logits"], case["k"], valid=st["valid"], normalise=case["normalise"], loss=case["loss"])
        return list(r) if case["loss"] else list(r[:7])
    if op == "route_bwd":
        return [bnn.route_bwd(st["logits"], st["experts"], st["weights"], st["stats"], slope=st["slope"],
                              dweights=st["dweights"], dloss=st["dloss"], normalise=case["normalise"])]
    if op == "combine_fwd":
        return [bnn.combine_fwd(st["y"], st["place"], weights=st["weights"], residual=st["residual"],
                                dtype=DTYPES[case["out"]])]
    if op == "combine_bwd":
        return list(bnn.combine_bwd(st["dout"], st["place"], weights=st["weights"], y=st["y"]))
    if op == "adapter_fwd":
        return list(bnn.adapter_fwd(st["x"], st["ids"], st["a"], st["b"], scale=st["scale"], base=st["base"]))
    return list(bnn.adapter_bwd(st["dy"], st["x"], st["u"], st["ids"], st["a"], st["b"], scale=st["scale"],
                                base=st["base"]))


def _route_plain(logits, valid, k, normalise):
    t, e = logits.shape
    z = logits.float()
    if valid is not None:
        z = torch.where(valid[:, None], z, torch.full_like(z, -math.inf))
    top, chosen = torch.sort(z, dim=1, descending=True, stable=True)
    top, chosen = top[:, :k], chosen[:, :k]
    has = top > -math.inf
    routed = has[:, 0]
    m = torch.where(routed, top[:, 0], torch.zeros_like(top[:, 0]))
    ez = torch.exp(z - m[:, None])
    rsum = torch.where(routed, 1.0 / ez.sum(dim=1), torch.zeros_like(m))
    p = ez * rsum[:, None]
    weights = torch.exp(top - m[:, None])
    if normalise:
        weights = weights / torch.where(routed, weights.sum(dim=1), torch.ones_like(m))[:, None]
    else:
        weights = weights * rsum[:, None]
    slot = torch.where(has, chosen, torch.full_like(chosen, e)).reshape(-1)
    expert, order = torch.sort(slot, stable=True)
    row = torch.arange(t * k, device=DEV)
    place = torch.empty_like(order)
    place[order] = torch.where(expert < e, row, -2 - row)
    rows = torch.where(expert < e, order // k, torch.full_like(order, -1))
    counts = torch.bincount(slot, minlength=e + 1)[:e]
    offsets = torch.nn.functional.pad(torch.cumsum(counts, 0), (1, 0))
    tokens = routed.sum()
    each = tokens.clamp(min=1).double()
    slope = (counts.double() * e / (k * each * each)).float()
    loss = (slope * p.sum(dim=0)).sum().reshape(1)
    i32 = torch.int32
    return [torch.where(has, chosen, torch.full_like(chosen, -1)).to(i32), weights, place.view(t, k).to(i32), rows.to(i32),
            offsets.to(i32), counts.to(i32), torch.stack([m, rsum], dim=1), slope, loss]


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "route_fwd":
        r = _route_plain(st["logits"], st["valid"], case["k"], case["normalise"])
        return r if case["loss"] else r[:7]
    if op == "route_bwd":
        z, m, rsum = st["logits"].float(), st["stats"][:, :1], st["stats"][:, 1:]
        p = torch.where(rsum > 0, torch.exp(z - m) * rsum, torch.zeros_like(z))
        grad = (st["dloss"] * st["slope"]).expand_as(p).clone()
        at, has = st["experts"].long().clamp(min=0), st["experts"] >= 0
        dw = torch.where(has, st["dweights"], torch.zeros_like(st["dweights"]))
        if not case["normalise"]:
            grad.scatter_add_(1, at, dw)
        dz = p * (grad - (p * grad).sum(dim=1, keepdim=True))
        if case["normalise"]:
            w = st["weights"]
            dz.scatter_add_(1, at, torch.where(has, w * (dw - (w * dw).sum(dim=1, keepdim=True)), torch.zeros_like(w)))
        return [dz.to(st["logits"].dtype)]
    if op.startswith("combine"):
        place, w = st["place"].long(), st["weights"]
        has = place >= 0
        row = torch.where(has, place, -2 - place)
        y = _dequantised(*st["y"], case["n"]) if case["dtype"] == "f8" else st["y"].float()
        if op == "combine_fwd":
            scale = has.float() if w is None else torch.where(has, w, torch.zeros_like(w))
            out = (y[row] * scale[:, :, None]).sum(dim=1)
            if st["residual"] is not None:
                out = out + st["residual"].float()
            return [out.to(DTYPES[case["out"]])]
        scale = torch.where(has, w, torch.zeros_like(w))
        dout = st["dout"].float()
        dy = torch.empty_like(y)
        dy[row.reshape(-1)] = (dout[:, None, :] * scale[:, :, None]).reshape(-1, case["n"])
        dweights = torch.where(has, (dout[:, None, :] * y[row]).sum(dim=2), torch.zeros_like(w))
        return [dy.to(st["dout"].dtype if case["dtype"] == "f8" else st["y"].dtype), dweights]
    ids, r = st["ids"].long(), case["rank"]
    out = st["base"].float()
    if op == "adapter_fwd":
        if case["runs"] == 1 and case["rows"] <= 256:  # every row's own factors, all rows at once
            at, has = ids.clamp(min=0), (ids >= 0).float()
            u = torch.bmm(st["a"][at].float(), st["x"].float().unsqueeze(2)).squeeze(2) * has[:, None]
            out = out + torch.bmm((u * st["scale"][at][:, None]).unsqueeze(1), st["b"][at].float()).squeeze(1)
            return [out.to(st["base"].dtype), u]
        u = torch.zeros(case["rows"], r, device=DEV)
        out = out.clone()
        for i in st["present"]:
            at = torch.nonzero(ids == i).flatten()
            u[at] = st["x"][at].float() @ st["a"][i].float().t()
            out[at] += (u[at] * st["scale"][i]) @ st["b"][i].float()
        return [out.to(st["base"].dtype), u]
    out = out.clone()
    x = _dequantised(*st["x"], case["k"]) if case["kept"] == "f8" else st["x"].float()
    da = torch.zeros(st["a"].shape, device=DEV)
    db = torch.zeros(st["b"].shape, device=DEV)
    for i in st["present"]:
        at = torch.nonzero(ids == i).flatten()
        dy = st["dy"][at].float()
        v = (dy @ st["b"][i].float().t()) * st["scale"][i]
        out[at] += v @ st["a"][i].float()
        da[i] = v.t() @ x[at]
        db[i] = (st["u"][at] * st["scale"][i]).t() @ dy
    return [out.to(st["base"].dtype), da, db]


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op = case["op"]
    if op.startswith("route"):
        t, e, k, s = case["tokens"], case["experts"], case["k"], SIZE[case["dtype"]]
        mask = t if case["masked"] and op == "route_fwd" else 0
        if op == "route_fwd":
            return {"bytes": t * e * s + mask + 16 * t * k + 8 * t + 12 * e, "flops": 4 * t * e}
        return {"bytes": 2 * t * e * s + 12 * t * k + 8 * t + 4 * e, "flops": 8 * t * e}
    if op.startswith("combine"):
        t, n, k, s, o = case["tokens"], case["n"], case["k"], SIZE[case["dtype"]], SIZE[case["out"]]
        if op == "combine_fwd":
            return {"bytes": t * k * n * s + t * n * o * (2 if case["residual"] else 1) + 8 * t * k, "flops": 2 * t * k * n}
        d = o if case["dtype"] == "f8" else s
        return {"bytes": t * n * o + t * k * n * (s + d) + 12 * t * k, "flops": 3 * t * k * n}
    t, k, n, r, o = case["rows"], case["k"], case["n"], case["rank"], SIZE[case["out"]]
    used = min(case["adapters"], t if case["runs"] == 1 else -(-t // case["runs"]))
    factors = used * r * (k + n)
    if op == "adapter_fwd":
        return {"bytes": 2 * t * k + 2 * o * t * n + 2 * factors + 4 * t * r, "flops": 2 * t * r * (k + n)}
    return {"bytes": 2 * t * n + SIZE[case["kept"]] * t * k + 2 * o * t * k + 2 * factors + 4 * t * r
            + 4 * case["adapters"] * r * (k + n), "flops": 4 * t * r * (k + n)}


# ---------------------------------------------------------------------------
# 64 bits, from the definitions

def _decoded(q, s, k):
    """The 8-bit form's values, block by block."""
    v = q.view(torch.float8_e4m3fn).double()
    for i in range(q.shape[1] // BLOCK):
        v[:, i * BLOCK:(i + 1) * BLOCK] *= torch.exp2(s[:, i].double() - 127)[:, None]
    return v[:, :k]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op.startswith("route"):
        z, k, e = st["logits"].double(), case["k"], case["experts"]
        on = z > -math.inf
        if st["valid"] is not None:
            on = on & st["valid"].unsqueeze(1)
        z = z.masked_fill(~on, -math.inf)
        routed = on.any(dim=1)
        p = torch.softmax(z, dim=1).nan_to_num(0.0)  # a token without an expert: zeros
        if op == "route_fwd":
            order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
            w = p.gather(1, order)
            if case["normalise"]:
                w = (w / w.sum(dim=1, keepdim=True)).nan_to_num(0.0)
            m = z.amax(dim=1).masked_fill(~routed, 0.0)
            rsum = torch.where(routed, torch.exp(m - torch.logsumexp(z, dim=1)), torch.zeros_like(m))
            out = [None, w, None, None, None, None, torch.stack([m, rsum], dim=1)]
            if not case["loss"]:
                return out
            taken = on.gather(1, order)
            count = torch.zeros(e, dtype=torch.float64, device=DEV)
            count.index_add_(0, order[taken], torch.ones_like(order[taken], dtype=torch.float64))
            tv = max(int(routed.sum()), 1)
            share, mean = count / (k * tv), p.sum(dim=0) / tv
            return out + [e * share / tv, (e * torch.dot(share, mean)).reshape(1)]
        # the gradient through the softmax's Jacobian, choice by choice
        grad = st["dloss"].double() * st["slope"].double().unsqueeze(0)
        dz = p * (grad - torch.mv(p, grad[0]).unsqueeze(1))
        has = st["experts"] >= 0
        dw = st["dweights"].double() * has
        w = st["weights"].double() if case["normalise"] else p.gather(1, st["experts"].long().clamp(min=0)) * has
        inner = (w * dw).sum(dim=1)
        for j in range(k):
            at = st["experts"][:, j].long().clamp(min=0)
            if case["normalise"]:
                dz[torch.arange(len(at), device=DEV), at] += (w[:, j] * (dw[:, j] - inner)) * has[:, j]
            else:
                dz[torch.arange(len(at), device=DEV), at] += w[:, j] * dw[:, j]
        if not case["normalise"]:
            dz -= p * inner.unsqueeze(1)
        return [dz]
    if op.startswith("combine"):
        t, n, k = case["tokens"], case["n"], case["k"]
        y = _decoded(*st["y"], n) if case["dtype"] == "f8" else st["y"].double()
        if op == "combine_fwd":
            out = torch.zeros(t, n, dtype=torch.float64, device=DEV)
            if st["residual"] is not None:
                out += st["residual"].double()
            for j in range(k):
                token = torch.nonzero(st["place"][:, j] >= 0).flatten()
                part = y[st["place"][token, j].long()]
                if st["weights"] is not None:
                    part = part * st["weights"][token, j].double().unsqueeze(1)
                out[token] += part
            return [out]
        dy = torch.zeros(t * k, n, dtype=torch.float64, device=DEV)
        dw = torch.zeros(t, k, dtype=torch.float64, device=DEV)
        for j in range(k):
            token = torch.nonzero(st["place"][:, j] >= 0).flatten()
            at = st["place"][token, j].long()
            d = st["dout"][token].double()
            dy[at] = d * st["weights"][token, j].double().unsqueeze(1)
            dw[token, j] = torch.linalg.vecdot(d, y[at])
        return [dy, dw]
    t, k, n = case["rows"], case["k"], case["n"]
    a, b = st["a"].double(), st["b"].double()
    out = st["base"].double().clone()
    if op == "adapter_fwd":
        u = torch.zeros(t, case["rank"], dtype=torch.float64, device=DEV)
        for i in range(case["adapters"]):
            at = st["ids"] == i
            u[at] = torch.mm(st["x"][at].double(), a[i].t())
            out[at] += st["scale"][i].double() * torch.mm(u[at], b[i])
        return [out, u]
    x = _decoded(*st["x"], k) if case["kept"] == "f8" else st["x"].double()
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    for i in range(case["adapters"]):
        at, s = st["ids"] == i, st["scale"][i].double()
        d = st["dy"][at].double()
        v = torch.mm(d, b[i].t())
        out[at] += s * torch.mm(v, a[i])
        da[i] = s * torch.mm(v.t(), x[at])
        db[i] = s * torch.mm(st["u"][at].double().t(), d)
    return [out, da, db]
