"""Timing cases of the operators around the binarised layers: layer norm with
its gradient, the block-scaled 8-bit quantiser and product, and the
sign-weight product grouped by expert.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, rounded once at the end) or, with ``own`` set, through the package's
entry points; ``exact`` computes it in 64 bits from the definition.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
BLOCK = 128  # elements of K under one scale


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # the norm ahead of a sub-layer while decoding four sequences: latency
        {"name": "ln_fwd_decode", "op": "ln_fwd", "rows": 4, "n": 4096, "dtype": "bf16", "pad": 0, "stats": False},
        # the same norm over a training batch, statistics kept for the backward pass
        {"name": "ln_fwd_train", "op": "ln_fwd", "rows": 16384, "n": 4096, "dtype": "bf16", "pad": 0, "stats": True},
        # gradient over an odd batch of fp32 rows of the edge layer's width, cut out of wider rows
        {"name": "ln_bwd_odd", "op": "ln_bwd", "rows": 3001, "n": 1000, "dtype": "fp32", "pad": 3},
        # gradient of the training batch
        {"name": "ln_bwd_train", "op": "ln_bwd", "rows": 16384, "n": 4096, "dtype": "bf16", "pad": 0},
        # activations of the feed-forward layer's input, quantised along K before a projection
        {"name": "quant_rows", "op": "quant", "rows": 4096, "k": 4096, "dtype": "bf16", "pad": 0, "transpose": False},
        # a weight quantised along its output channels, the operand of the input's gradient
        {"name": "quant_cols", "op": "quant", "rows": 11008, "k": 4096, "dtype": "fp32", "pad": 0, "transpose": True},
        # one token through a projection: the weights' bytes bound it
        {"name": "f8_decode", "op": "f8", "m": 1, "n": 4096, "k": 4096, "out": "bf16"},
        # an odd middle-sized product with fp32 sums (the edge layer's K)
        {"name": "f8_odd", "op": "f8", "m": 201, "n": 1501, "k": 1000, "out": "fp32"},
        # the feed-forward shape of the packed product, in 8 bits
        {"name": "f8_large", "op": "f8", "m": 4096, "n": 11008, "k": 4096, "out": "bf16"},
        # one token sent to eight of 64 experts: their packed weights' bytes bound it
        {"name": "grouped_decode", "op": "grouped", "tokens": 1, "topk": 8, "experts": 64, "n": 1024, "k": 4096,
         "gather": True, "row_scale": False, "out": "bf16"},
        # a few hundred tokens on ten experts at the edge layer's K, weighted by the router (a down projection)
        {"name": "grouped_odd", "op": "grouped", "tokens": 301, "topk": 2, "experts": 10, "n": 700, "k": 1000,
         "gather": False, "row_scale": True, "out": "fp32"},
        # a prompt batch through 32 experts, rows gathered from the tokens (an up projection)
        {"name": "grouped_prompt", "op": "grouped", "tokens": 8192, "topk": 2, "experts": 32, "n": 4096, "k": 4096,
         "gather": True, "row_scale": False, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number, its logarithm spread evenly over [lo, hi]; a third are rounded to a multiple of 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.34 and v >= 64:
        v -= v % 64
    v = max(lo, min(hi, v))
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "quant", "f8", "f8", "grouped", "grouped"])
    if op in ("ln_fwd", "ln_bwd"):
        n = _log(rng, 32, 16384)
        case = {"op": op, "rows": _log(rng, 1, min(16384, (16384 * 4096) // n)), "n": n,
                "dtype": rng.choice(["bf16", "fp32"]), "pad": rng.choice([0, 0, 8, 3])}
        if case["dtype"] == "fp32":
            case["rows"] = max(1, case["rows"] // 2)
        if op == "ln_fwd":
            case["stats"] = rng.random() < 0.5
        return case
    if op == "quant":
        k = _log(rng, 64, 11008)
        return {"op": op, "rows": _log(rng, 1, min(11008, (11008 * 4096) // k)), "k": k,
                "dtype": rng.choice(["bf16", "fp32"]), "pad": rng.choice([0, 0, 8, 3]),
                "transpose": rng.random() < 0.5}
    if op == "f8":
        k, n = _log(rng, 64, 8192), _log(rng, 16, 11008)
        most = 4096 * 4096 * 11008
        return {"op": op, "m": _log(rng, 1, max(1, min(4096, most // (n * k)))), "n": n, "k": k,
                "out": rng.choice(["bf16", "fp32"])}
    topk = rng.choice([1, 2, 4, 8])
    experts = max(topk, _log(rng, 4, 128))
    k, n = _log(rng, 64, 4096), _log(rng, 64, 4096)
    while experts * n * k > 32 * 4096 * 4096:
        n = max(64, n // 2)
    tokens = _log(rng, 1, max(1, 16384 // topk))
    return {"op": op, "tokens": tokens, "topk": topk, "experts": experts, "n": n, "k": k,
            "gather": rng.random() < 0.5, "row_scale": rng.random() < 0.5, "out": rng.choice(["bf16", "fp32"])}


# ---------------------------------------------------------------------------
# inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _rows_of(g, rows, cols, dtype, pad, offset=0.0):
    """(rows, cols) of a wider matrix: its rows are cols + pad apart."""
    return (_randn(g, rows, cols + pad) + offset).to(dtype)[:, :cols]


def _quantised(v):
    """Block-scaled e4m3 form of fp32 rows: bytes (rows, 128 * blocks), zeros
    past K, and scale bytes (rows, 4 * ceil(blocks / 4))."""
    rows, k = v.shape
    nb = -(-k // BLOCK)
    x = torch.nn.functional.pad(v, (0, nb * BLOCK - k)).reshape(rows, nb, BLOCK)
    mant, ex = torch.frexp(x.abs().amax(dim=2))
    e = torch.where(mant > 0.875, ex - 8, ex - 9)  # 448 = 0.875 * 2^9
    e = torch.where(mant == 0, torch.zeros_like(e), e.clamp(min=-127))
    q = torch.ldexp(x, -e.unsqueeze(2)).to(torch.float8_e4m3fn)
    s = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, -nb % 4))
    return q.reshape(rows, nb * BLOCK).view(torch.uint8), s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    st = {"case": dict(case)}
    if op in ("ln_fwd", "ln_bwd"):
        dt, m, n = DTYPES[case["dtype"]], case["rows"], case["n"]
        # a residual stream: rows of different scale and mean
        x = _randn(g, m, n + case["pad"]) * (0.5 + 2.0 * torch.rand(m, 1, generator=g, device=DEV))
        x += _randn(g, m, 1)
        st["x"] = x.to(dt)[:, :n]
        st["gamma"] = 1.0 + 0.1 * _randn(g, n)
        st["beta"] = 0.1 * _randn(g, n)
        if op == "ln_bwd":
            st["dy"] = _rows_of(g, m, n, dt, case["pad"])
            xf = st["x"].float()
            st["mean"] = xf.mean(dim=1)
            st["rstd"] = torch.rsqrt((xf - st["mean"][:, None]).square().mean(dim=1) + 1e-5)
    elif op == "quant":
        dt = DTYPES[case["dtype"]]
        m, k = case["rows"], case["k"]
        st["x"] = (_randn(g, m, k + case["pad"]) * torch.exp(_randn(g, m, 1))).to(dt)[:, :k]
    elif op == "f8":
        m, n, k = case["m"], case["n"], case["k"]
        st["xq"], st["xs"] = _quantised(_randn(g, m, k) * torch.exp(0.5 * _randn(g, m, 1)))
        st["wq"], st["ws"] = _quantised(_randn(g, n, k) * 0.02)
    else:
        t, tk, ne, n, k = case["tokens"], case["topk"], case["experts"], case["n"], case["k"]
        kw = -(-k // 64)
        # a skewed router: some experts are popular, some get nothing
        logits = _randn(g, t, ne) + _randn(g, 1, ne)
        weight, chosen = torch.softmax(logits, dim=1).topk(tk, dim=1)
        order = torch.argsort(chosen.reshape(-1), stable=True)
        expert = chosen.reshape(-1)[order]
        token = (order // tk).to(torch.int32)
        counts = torch.bincount(expert, minlength=ne)
        x = _randn(g, t, k).to(torch.bfloat16)
        st["x"] = x if case["gather"] else x[token.long()].contiguous()
        st["rows"] = token if case["gather"] else None
        st["row_scale"] = weight.reshape(-1)[order].contiguous() if case["row_scale"] else None
        st["offsets"] = torch.nn.functional.pad(torch.cumsum(counts, 0), (1, 0)).to(torch.int32)
        st["expert"] = expert
        st["counts"] = counts.tolist()
        bits = torch.randint(0, 256, (ne, n, kw * 8), generator=g, device=DEV, dtype=torch.uint8)
        st["wp"] = bits.view(torch.int64)
        st["alpha"] = 0.02 * (0.5 + torch.rand(ne, n, generator=g, device=DEV))
    return st


# ---------------------------------------------------------------------------
# the operators

def _run_own(st):
    import packed_xor_popcount_amd as bnn
    case = st["case"]
    op = case["op"]
    if op == "ln_fwd":
        y, mean, rstd = bnn.layernorm_fwd(st["x"], st["gamma"], st["beta"], 1e-5, stats=case["stats"])
        return [y, mean, rstd] if case["stats"] else [y]
    if op == "ln_bwd":
        return list(bnn.layernorm_bwd(st["dy"], st["x"], st["mean"], st["rstd"], st["gamma"]))
    if op == "quant":
        q, s = bnn.quant_f8(st["x"], transpose=case["transpose"])
        return [q.view(torch.float8_e4m3fn), s]
    if op == "f8":
        return [bnn.gemm_f8(st["xq"], st["xs"], st["wq"], st["ws"], case["k"], dtype=DTYPES[case["out"]])]
    return [bnn.gemm_signw_grouped(st["x"], st["wp"], st["offsets"], case["k"], alpha=st["alpha"], rows=st["rows"],
                                   row_scale=st["row_scale"], dtype=DTYPES[case["out"]])]


def _dequantised(q, s, k):
    rows, nb = q.shape[0], q.shape[1] // BLOCK
    v = q.view(torch.float8_e4m3fn).float().reshape(rows, nb, BLOCK)
    return torch.ldexp(v, s[:, :nb].to(torch.int32).unsqueeze(2) - 127).reshape(rows, nb * BLOCK)[:, :k]


def _signs(wp, k):
    """+-1 of packed rows: bit 1 is -1."""
    byte = wp.view(torch.uint8)
    bit = (byte.unsqueeze(-1) >> torch.arange(8, device=DEV, dtype=torch.uint8)) & 1
    return (1.0 - 2.0 * bit.reshape(*byte.shape[:-1], -1)[..., :k].float())


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "ln_fwd":
        x = st["x"].float()
        mean = x.mean(dim=1)
        d = x - mean[:, None]
        rstd = torch.rsqrt(d.square().mean(dim=1) + 1e-5)
        y = (d * rstd[:, None] * st["gamma"] + st["beta"]).to(st["x"].dtype)
        return [y, mean, rstd] if case["stats"] else [y]
    if op == "ln_bwd":
        x, dy = st["x"].float(), st["dy"].float()
        xh = (x - st["mean"][:, None]) * st["rstd"][:, None]
        gr = dy * st["gamma"]
        dx = (gr - gr.mean(dim=1, keepdim=True) - xh * (gr * xh).mean(dim=1, keepdim=True)) * st["rstd"][:, None]
        return [dx.to(st["x"].dtype), (dy * xh).sum(dim=0), dy.sum(dim=0)]
    if op == "quant":
        x = st["x"].float()
        q, s = _quantised(x.t().contiguous() if case["transpose"] else x)
        return [q.view(torch.float8_e4m3fn), s]
    if op == "f8":
        x = _dequantised(st["xq"], st["xs"], case["k"])
        w = _dequantised(st["wq"], st["ws"], case["k"])
        return [torch.matmul(x, w.t()).to(DTYPES[case["out"]])]
    # experts that have rows, each padded to the longest one's number of rows
    counts = torch.tensor(st["counts"])
    active = torch.nonzero(counts).flatten()
    place = torch.full((len(counts),), 0, dtype=torch.int64)
    place[active] = torch.arange(len(active))
    active, place = active.to(DEV), place.to(DEV)
    begin = st["offsets"][:-1].long()
    total = st["expert"].numel()
    at = begin[active][:, None] + torch.arange(int(counts.max()), device=DEV)
    at = at.clamp(max=total - 1)  # rows past an expert's end are computed and not used
    src = st["rows"].long()[at] if st["rows"] is not None else at
    y = torch.bmm(st["x"].float()[src], _signs(st["wp"][active], case["k"]).transpose(1, 2))
    y = y * st["alpha"][active][:, None, :]
    y = y[place[st["expert"]], torch.arange(total, device=DEV) - begin[st["expert"]]]
    if st["row_scale"] is not None:
        y = y * st["row_scale"][:, None]
    return [y.to(DTYPES[case["out"]])]


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        e, size = (2 if case["dtype"] == "bf16" else 4), case["rows"] * case["n"]
        if op == "ln_fwd":
            return {"bytes": 2 * size * e + 8 * case["n"] + (8 * case["rows"] if case["stats"] else 0),
                    "flops": 7 * size}
        return {"bytes": 3 * size * e + 8 * case["rows"] + 12 * case["n"], "flops": 13 * size}
    if op == "quant":
        e, size = (2 if case["dtype"] == "bf16" else 4), case["rows"] * case["k"]
        return {"bytes": size * e + size + size // BLOCK, "flops": 2 * size}
    o = 2 if case["out"] == "bf16" else 4
    n, k = case["n"], case["k"]
    if op == "f8":
        m = case["m"]
        return {"bytes": (m + n) * k + (m + n) * k // BLOCK + m * n * o, "flops": 2 * m * n * k}
    rows = case["tokens"] * case["topk"]
    active = min(case["experts"], rows)
    xrows = case["tokens"] if case["gather"] else rows
    return {"bytes": xrows * k * 2 + active * n * (8 * -(-k // 64) + 4) + rows * n * o, "flops": 2 * rows * n * k}


# ---------------------------------------------------------------------------
# 64 bits, from the definitions

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "ln_fwd":
        x = st["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1.0 / torch.sqrt(var + 1e-5)
        y = torch.addcmul(st["beta"].double(), (x - mean.unsqueeze(1)) * rstd.unsqueeze(1), st["gamma"].double())
        return [y, mean, rstd] if case["stats"] else [y]
    if op == "ln_bwd":
        # the gradient for the given statistics, summed as products
        x, dy = st["x"].double(), st["dy"].double()
        mean, rstd, gamma = st["mean"].double(), st["rstd"].double(), st["gamma"].double()
        n = x.shape[1]
        xh = torch.mul(x - mean.unsqueeze(1), rstd.unsqueeze(1))
        s1 = torch.mv(dy, gamma) / n
        s2 = torch.mv(dy * xh, gamma) / n
        dx = rstd.unsqueeze(1) * (dy * gamma - s1.unsqueeze(1) - xh * s2.unsqueeze(1))
        one = torch.ones(x.shape[0], dtype=torch.float64, device=DEV)
        return [dx, torch.mv((dy * xh).t(), one), torch.mv(dy.t(), one)]
    if op == "quant":
        # values on the e4m3 grid under each block's scale: 3 bits after the
        # leading one, exponents down to -6
        v = st["x"].double()
        v = v.t() if case["transpose"] else v
        rows, k = v.shape
        nb = (k + BLOCK - 1) // BLOCK
        full = torch.zeros(rows, nb * BLOCK, dtype=torch.float64, device=DEV)
        full[:, :k] = v
        full = full.view(rows, nb, BLOCK)
        top = full.abs().amax(dim=2, keepdim=True)
        e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.full_like(top, 448.0)) / 448.0)).clamp(min=-127)
        u = full / torch.exp2(e)
        step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)
        return [(torch.round(u / step) * step).reshape(rows, nb * BLOCK), None]
    if op == "f8":
        # one block of K at a time, scaled after its sum
        nb = st["xq"].shape[1] // BLOCK
        x8, w8 = st["xq"].view(torch.float8_e4m3fn), st["wq"].view(torch.float8_e4m3fn)
        y = torch.zeros(case["m"], case["n"], dtype=torch.float64, device=DEV)
        for b in range(nb):
            part = x8[:, b * BLOCK:(b + 1) * BLOCK].double() @ w8[:, b * BLOCK:(b + 1) * BLOCK].double().t()
            y += part * torch.exp2(st["xs"][:, b].double() - 127)[:, None] * torch.exp2(st["ws"][:, b].double() - 127)
        return [y]
    n, k = case["n"], case["k"]
    total = case["tokens"] * case["topk"]
    y = torch.zeros(total, n, dtype=torch.float64, device=DEV)
    off = st["offsets"].tolist()
    where = torch.arange(k, device=DEV)
    for e in range(case["experts"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        idx = st["rows"][lo:hi].long() if st["rows"] is not None else slice(lo, hi)
        word = st["wp"][e][:, where // 64]
        sign = 1 - 2 * ((word >> (where % 64)) & 1)
        y[lo:hi] = (st["x"][idx].double() @ sign.double().t()) * st["alpha"][e].double()
    if st["row_scale"] is not None:
        y *= st["row_scale"].double()[:, None]
    return [y]
