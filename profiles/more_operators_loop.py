"""Kernel times of the router, the sum of the experts' outputs and the low-rank
adapters.

    rocprofv3 --kernel-trace --stats -d OUT -o p -f csv -- python3 profiles/more_operators_loop.py run OUT/calls.json
    python3 profiles/more_operators_loop.py table OUT/p_kernel_trace.csv OUT/calls.json

``run`` makes 24 calls of each case of perf/more_operators.py (and of some more
sizes) with three sets of inputs in turn, one packing kernel between the cases;
``table`` prints the median, tenth and ninetieth percentile of each kernel's time
from the trace, in the calls' order.
"""
import csv
import json
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

CALLS = 24
KERNELS = tuple(k + "_kernel" for k in (
    "route_one", "route_choose", "route_place", "route_bwd", "group_count", "combine_fwd", "combine_bwd",
    "adapter_small", "adapter_shrink", "adapter_expand", "adapter_both", "adapter_outer",
    "adapter_join", "adapter_tiles"))


def run(path, only=""):
    import torch

    import packed_xor_popcount_amd as bnn
    from perf import more_operators as ops

    labels = []
    mark = torch.zeros(1, 64, device="cuda")

    def case(label, c):
        if only and not any(o in label for o in only.split(",")):
            return
        states = [ops.prepare(c, seed) for seed in range(3)]
        torch.cuda.synchronize()
        bnn.pack_signs(mark)
        for i in range(CALLS):
            ops.run(states[i % 3])
        torch.cuda.synchronize()
        labels.append(label)
        print(label, flush=True)

    ops.own = True
    for c in ops.listed():
        case(c["name"], c)
    more = {"op": "adapter_fwd", "rows": 1, "k": 4096, "n": 4096, "rank": 16, "adapters": 4, "runs": 1, "out": "fp32",
            "pad": 0}
    case("adapter_fwd one row 4096 x 4096 rank 16", more)
    case("adapter_fwd 256 rows 4096 x 4096 rank 16, 16 adapters mixed", dict(more, rows=256, adapters=16))
    case("adapter_fwd 1024 rows 4096 x 4096 rank 16, 4 adapters", dict(more, rows=1024, runs=100, out="bf16"))
    case("adapter_fwd 2048 rows 4096 x 4096 rank 64, 8 adapters", dict(more, rows=2048, adapters=8, rank=64, runs=200))
    case("adapter_fwd 4096 rows 4096 x 4096 rank 16, 16 adapters mixed", dict(more, rows=4096, adapters=16))
    more = {"op": "adapter_bwd", "rows": 1024, "k": 4096, "n": 4096, "rank": 16, "adapters": 4, "runs": 100, "out": "bf16",
            "pad": 0, "kept": "bf16"}
    case("adapter_bwd 1024 rows 4096 x 4096 rank 16", more)
    case("adapter_bwd 4096 rows 4096 x 4096 rank 64", dict(more, rows=4096, rank=64))
    case("adapter_bwd 2048 rows 4096 x 4096 rank 128", dict(more, rows=2048, rank=128))
    route = dict(ops.listed()[1])
    case("combine_fwd 4096 x 4096, 8, fp32", dict(ops.listed()[5], tokens=4096, k=8, dtype="fp32"))
    case("combine_bwd 2000 x 4096, 4, bf16", dict(ops.listed()[7], tokens=2000, dtype="bf16"))
    case("route_fwd 1024 x 64, 8", dict(route, tokens=1024, experts=64))
    case("route_fwd 8192 x 256, 8 bf16", dict(route, tokens=8192, experts=256, dtype="bf16"))
    with open(path, "w") as f:
        json.dump(labels, f)


def table(trace, notes):
    with open(trace) as f:
        rows = list(csv.DictReader(f))
    rows.sort(key=lambda r: int(r["Start_Timestamp"]))
    with open(notes) as f:
        labels = json.load(f)
    at, cases = -1, [[] for _ in labels]
    for r in rows:
        if "bnn" not in r["Kernel_Name"]:
            continue
        if "pack_kernel" in r["Kernel_Name"]:
            at += 1
        else:
            cases[at].append(r)
    print("| call | kernel | median us | 10 % .. 90 % | threads |")
    print("|---|---|---|---|---|")
    for label, part in zip(labels, cases):
        n = len(part) // CALLS
        assert n * CALLS == len(part), "the trace and the notes do not fit"
        for j in range(n):
            mine = part[j::n]
            us = sorted((int(r["End_Timestamp"]) - int(r["Start_Timestamp"])) / 1e3 for r in mine)
            name = next(k for k in KERNELS if k in mine[0]["Kernel_Name"])
            grid = " x ".join(mine[0]["Grid_Size_" + d] for d in "XYZ")
            print(f"| {label if j == 0 else ''} | `{name}` | {us[CALLS // 2]:.2f} | {us[CALLS // 10]:.2f} .. "
                  f"{us[-1 - CALLS // 10]:.2f} | {grid} |")


if __name__ == "__main__":
    {"run": run, "table": table}[sys.argv[1]](*sys.argv[2:])
