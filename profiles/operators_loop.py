"""Kernel times of the operators around the binarised layers.

    rocprofv3 --kernel-trace --stats -d OUT -o p -f csv -- python3 profiles/operators_loop.py run OUT/calls.json
    python3 profiles/operators_loop.py table OUT/p_kernel_trace.csv OUT/calls.json

``run`` makes 24 calls of each size with three sets of inputs in turn and notes
how many kernels a call launches; ``table`` prints the median, tenth and
ninetieth percentile of each kernel's time from the trace, in the calls' order.
"""
import csv
import json
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

CALLS = 24


def run(path):
    import torch

    import packed_xor_popcount_amd as bnn
    from perf import operators as ops

    ops.own = True
    notes = []

    def calls(label, states, call, kernels=1):
        torch.cuda.synchronize()
        for i in range(CALLS):
            call(states[i % len(states)])
        torch.cuda.synchronize()
        notes.append([label, kernels, CALLS])
        print(label, flush=True)

    def case(label, c, call=ops.run, kernels=1):
        calls(label, [ops.prepare(c, seed) for seed in range(3)], call, kernels)

    def fast(st):
        return bnn.gemm_f8(st["xq"], st["xs"], st["wq"], st["ws"], st["case"]["k"], dtype=torch.bfloat16, fast=True)

    for c in ops.listed():
        case(c["name"], c, kernels=2 if c["op"] == "ln_bwd" else 1)
        if c["name"] == "f8_large":
            case("f8_large, fast", c, fast)
            case("f8_large, fp32", dict(c, out="fp32"))
    for op, rows, n, dtype, kernels in (("ln_fwd", 1, 4096, "bf16", 1), ("ln_fwd", 16384, 4096, "fp32", 1),
                                        ("ln_fwd", 2048, 20000, "bf16", 1), ("ln_bwd", 1, 4096, "bf16", 1),
                                        ("ln_bwd", 256, 4096, "bf16", 1), ("ln_bwd", 1024, 16384, "bf16", 1),
                                        ("ln_bwd", 1024, 4096, "bf16", 2), ("ln_bwd", 2048, 20000, "bf16", 2)):
        case(f"{op} {rows} x {n} {dtype}",
             {"op": op, "rows": rows, "n": n, "dtype": dtype, "pad": 0, "stats": True}, kernels=kernels)
    for dtype, rows in (("bf16", 4096), ("fp32", 11008)):
        for t in (False, True):
            case(f"quant {rows} x 4096 {dtype} {'transposed' if t else 'rows'}",
                 {"op": "quant", "rows": rows, "k": 4096, "dtype": dtype, "pad": 0, "transpose": t})
    for m in (16, 32, 33, 128, 256, 2048):
        c = {"op": "f8", "m": m, "n": 4096, "k": 4096, "out": "bf16"}
        case(f"f8 {m} x 4096 x 4096", c)
        if m > 32:
            case(f"f8 {m} x 4096 x 4096, fast", c, fast)

    def grouped(label, counts, N, K):
        g = torch.Generator(device="cuda")
        g.manual_seed(1)
        E, R = len(counts), sum(counts)
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[1:] = torch.cumsum(torch.tensor(counts, device="cuda"), 0)
        states = []
        for _ in range(3):
            bits = torch.randint(0, 256, (E, N, -(-K // 64) * 8), generator=g, device="cuda", dtype=torch.uint8)
            states.append((torch.randn(R, K, generator=g, device="cuda").to(torch.bfloat16), bits.view(torch.int64),
                           torch.rand(E, N, generator=g, device="cuda")))
        for name, algo in (("few-row", bnn.ALGO_GEMV), ("tiles", bnn.ALGO_MFMA)):
            calls(f"grouped {label}, {N} x {K}, {name}", states,
                  lambda st: bnn.gemm_signw_grouped(st[0], st[1], off, K, alpha=st[2], dtype=torch.bfloat16, algo=algo))

    def even(r, e):
        return [r // e + (i < r % e) for i in range(e)]

    grouped("256 rows on 64", even(256, 64), 1024, 4096)
    grouped("602 rows on 10", even(602, 10), 700, 1000)
    grouped("2000 rows on 128", even(2000, 128), 1024, 512)
    grouped("4000 rows on 32", even(4000, 32), 2048, 2048)
    grouped("2000 rows on 8", even(2000, 8), 1001, 1001)
    grouped("16384 rows on 1", [16384], 4096, 4096)
    grouped("640 rows on 64 (577 on one)", [577] + [1] * 63, 1024, 4096)
    grouped("1280 rows on 128 (1153 on one)", [1153] + [1] * 127, 4096, 4096)
    with open(path, "w") as f:
        json.dump(notes, f)


def table(trace, notes):
    with open(trace) as f:
        rows = [r for r in csv.DictReader(f) if "bnn" in r["Kernel_Name"]]
    rows.sort(key=lambda r: int(r["Start_Timestamp"]))
    with open(notes) as f:
        notes = json.load(f)
    assert len(rows) == sum(k * n for _, k, n in notes), "the trace and the notes do not fit"
    print("| call | kernel | median us | 10 % .. 90 % | VGPRs | LDS bytes | threads |")
    print("|---|---|---|---|---|---|---|")
    at = 0
    for label, kernels, n in notes:
        for j in range(kernels):
            part = rows[at + j:at + kernels * n:kernels]
            us = sorted((int(r["End_Timestamp"]) - int(r["Start_Timestamp"])) / 1e3 for r in part)
            name = part[0]["Kernel_Name"]
            name = next(k for k in ("ln_fwd_long", "ln_bwd_long", "ln_bwd_finish", "ln_fwd", "ln_bwd", "quant_rows",
                                    "quant_cols", "gemm_f8_rows", "gemm_f8", "signw_grouped_rows", "signw_grouped")
                        if k + "_kernel" in name)
            print(f"| {label if j == 0 else ''} | `{name}_kernel` | {us[n // 2]:.2f} | {us[n // 10]:.2f} .. "
                  f"{us[-1 - n // 10]:.2f} | {part[0]['VGPR_Count']} | {part[0]['LDS_Block_Size']} | "
                  f"{part[0]['Grid_Size_X']} |")
        at += kernels * n


if __name__ == "__main__":
    {"run": run, "table": table}[sys.argv[1]](*sys.argv[2:])
