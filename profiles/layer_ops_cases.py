"""Runs the listed cases of perf/operators.py and some more and prints the time of a call.

    python3 profiles/layer_ops_cases.py [--plain | --forward] [--rounds 100] [--only NAME,NAME]

Per case three states of inputs and weights are run in turn, so that a case of more than 85 MB does not find its data
in the 256 MB memory-side cache and a smaller one does.  A call's time is the median over rounds of the time between
events around the three runs, divided by three, with the queue kept full: of a call shorter than its own launch from
Python (about 6 us) it is that.  Under rocprofv3 --kernel-trace the same loop gives the kernels' times (the trace is
ordered by start; each case first runs 10 rounds untimed).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import perf.operators as ops  # noqa: E402


def layer(name, T, H, I, E, k, fmt):
    return {"name": name, "op": "layer", "T": T, "H": H, "I": I, "E": E, "k": k, "fmt": fmt, "route": "precomputed",
            "mask": 0.0, "add": False}


# NVFP4 x NVFP4; an eighth of a layer's columns; more tokens than one unit of work takes (16) on most experts
MORE = [layer("layer nvfp4 x nvfp4 1", 1, 7168, 2048, 32, 8, "nvfp4"),
        layer("layer nvfp4 x nvfp4 3", 3, 7168, 2048, 32, 8, "nvfp4"),
        layer("layer nvfp4 x nvfp4 32", 32, 7168, 2048, 32, 8, "nvfp4"),
        layer("layer fp8 1, I 256", 1, 7168, 256, 32, 8, "fp8_block128"),
        layer("layer fp8 32, k 16 of 32", 32, 7168, 2048, 32, 16, "fp8_block128"),
        layer("layer bf16 32, k 2 of 8", 32, 4096, 14336, 8, 2, "bf16"),
        layer("layer bf16 32, k 4 of 8", 32, 4096, 14336, 8, 4, "bf16"),
        layer("layer bf16 32, k 8 of 8", 32, 4096, 14336, 8, 8, "bf16")]


class NvNorm:
    """The norm's NVFP4 output (no case of perf/operators.py)."""

    def __init__(self, T, H, seed):
        from mixture_experts_ffn_topk_amd import MoEFFN
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *n: torch.randn(n, generator=g, device="cuda").bfloat16()  # noqa: E731
        new = lambda n, t: torch.empty((T, n), dtype=t, device="cuda")  # noqa: E731
        self.moe = MoEFFN(H, 128, 8, 2, T, fmt="nvfp4")
        self.args = (T, rand(T, H), rand(T, H), rand(H), 1e-6)
        self.out = {"residual_out": new(H, torch.bfloat16), "x_norm": new(H, torch.bfloat16),
                    "x_q": new(H // 2, torch.uint8), "x_sf": new(H // 16, torch.uint8)}

    def run(self):
        self.moe.add_rmsnorm(*self.args, x_global_scale=0.01, **self.out)


def forward(s, ws):
    """The same layer by moe_forward_ex."""
    c = s["case"]
    s["moe"].forward(c["T"], s["x"], s["x_sf"], s["topk_idx"], s["topk_weights"],
                     s["logits"] if c["route"] == "from_logits" else None, s["weights"], s["out"], ws,
                     shared=s["shared"], residual=s["residual"])


def measure(name, calls, rounds, warm):
    for c in warm * calls:
        c()
    torch.cuda.synchronize()
    marks = [torch.cuda.Event(enable_timing=True) for _ in range(rounds + 1)]
    marks[0].record()
    for m in marks[1:]:
        for c in calls:
            c()
        m.record()
    torch.cuda.synchronize()
    us = sorted(a.elapsed_time(b) * 1000 / len(calls) for a, b in zip(marks, marks[1:]))
    print(f"{name}: median {us[len(us) // 2]:.2f} us, min {us[0]:.2f}, max {us[-1]:.2f}", flush=True)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--plain", action="store_true", help="the plain forms in place of the framework's kernels")
    ap.add_argument("--forward", action="store_true", help="the layers by moe_forward_ex in place of moe_forward_few")
    ap.add_argument("--rounds", type=int, default=100)
    ap.add_argument("--only", default="")
    args = ap.parse_args()
    ops.own = not args.plain
    only = args.only.split(",") if args.only else None
    warm = 1 if args.plain else 10
    for case in ops.listed() + ([] if args.plain else MORE):
        if (only and case["name"] not in only) or (args.forward and case["op"] != "layer"):
            continue
        states = [ops.prepare(case, seed) for seed in range(3)]
        if args.forward:
            calls = [lambda s=s, ws=s["moe"].alloc_workspace(case["T"]): forward(s, ws) for s in states]
        else:
            calls = [lambda s=s: ops.run(s) for s in states]
        measure(case["name"], calls, args.rounds, warm)
        del states, calls
        torch.cuda.empty_cache()
    if not args.plain and not args.forward:
        for T in (1, 8192):
            if not only or f"norm nvfp4 {T}" in only:
                measure(f"norm nvfp4 {T}", [NvNorm(T, 7168, seed).run for seed in range(3)], args.rounds, warm)


if __name__ == "__main__":
    main()
