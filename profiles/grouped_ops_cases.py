"""Runs the listed cases of perf/more_operators.py and some more and prints the time of a call.

    python3 profiles/grouped_ops_cases.py [--plain] [--rounds 100] [--only NAME,NAME]

Per case three states of inputs and weights are run in turn with the queue kept full (a call shorter than its own launch
from Python, about 6 us, shows that).  Under rocprofv3 --kernel-trace the same loop gives the kernels' times.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import perf.more_operators as ops  # noqa: E402


def gemm(name, T, H, I, E, k, side="forward"):
    return {"name": name, "op": "gemm", "T": T, "H": H, "I": I, "E": E, "k": k, "leg": "gate_up", "side": side,
            "f32": False, "skew": 0.0, "mask": 0.0}


def mx(name, T, H, I, E, k):
    return {"name": name, "op": "mx", "T": T, "H": H, "I": I, "E": E, "k": k, "leg": "gate_up", "skew": 0.0, "mask": 0.0}


# middling rows an expert: 128 x 128 tiles; MXFP4's 32 x 32
MORE = [gemm("gemm 64", 64, 4096, 14336, 8, 2), gemm("gemm 256", 256, 4096, 14336, 8, 2),
        gemm("gemm rows' gradient 256", 256, 7168, 2048, 32, 8, "gradient"), mx("mx 512", 512, 2880, 2880, 128, 4)]


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--plain", action="store_true", help="the plain forms in place of the framework's kernels")
    ap.add_argument("--rounds", type=int, default=100)
    ap.add_argument("--only", default="")
    args = ap.parse_args()
    ops.own = not args.plain
    only = args.only.split(",") if args.only else None
    for case in ops.listed() + ([] if args.plain else MORE):
        if only and case["name"] not in only:
            continue
        states = [ops.prepare(case, seed) for seed in range(3)]
        for _ in range(1 if args.plain else 10):
            for s in states:
                ops.run(s)
        torch.cuda.synchronize()
        marks = [torch.cuda.Event(enable_timing=True) for _ in range(args.rounds + 1)]
        marks[0].record()
        for m in marks[1:]:
            for s in states:
                ops.run(s)
            m.record()
        torch.cuda.synchronize()
        us = sorted(a.elapsed_time(b) * 1000 / len(states) for a, b in zip(marks, marks[1:]))
        print(f"{case['name']}: median {us[len(us) // 2]:.2f} us, min {us[0]:.2f}, max {us[-1]:.2f}", flush=True)
        del states
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main()
