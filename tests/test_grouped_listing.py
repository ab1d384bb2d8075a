"""The loads into LDS that grouped.hip writes in assembly: five states have to pass between a vector instruction that writes
a scalar register of their resource (a restored spill too) and the load, and the compiler, which does not see the load,
counts none.  Read from the assembly that hipcc writes for the source."""
import os
import re
import subprocess

import pytest

from mixture_experts_ffn_topk_amd import build

STATES = 5


def scalars(text):
    out = set()
    for a, b, one in re.findall(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b", text):
        out |= {int(one)} if one else set(range(int(a), int(b) + 1))
    return out


def parse(body):
    """(instructions, label -> index of what follows it, label -> indices of the branches to it)"""
    ins, labels, jumps = [], {}, {}
    for line in body.split("\n"):
        t = line.split(";")[0].strip()
        if m := re.match(r"(\.LBB\w+):", t):
            labels[m.group(1)] = len(ins)
        elif t and t[0] not in "._":
            if m := re.match(r"s_c?branch\w* (\.LBB\w+)", t):
                jumps.setdefault(m.group(1), []).append(len(ins))
            ins.append(t)
    return ins, labels, jumps


def written_before(ins, at_label, jumps, i, regs, states):
    """Vector instructions that write one of regs less than `states` states ahead of instruction i, on any path."""
    found = []
    for label in at_label.get(i, []):
        for j in jumps.get(label, []):
            found += step(ins, at_label, jumps, j, regs, states)
    if i > 0 and not ins[i - 1].startswith(("s_branch", "s_endpgm")):
        found += step(ins, at_label, jumps, i - 1, regs, states)
    return found


def step(ins, at_label, jumps, i, regs, states):
    op, _, rest = ins[i].partition(" ")
    if op.startswith("v_") and scalars(rest.split(",")[0]) & regs:
        return [ins[i]]
    states -= int(rest) + 1 if op == "s_nop" else 1
    return written_before(ins, at_label, jumps, i, regs, states) if states > 0 else []


def hazards(text):
    loads, found = 0, []
    for f in re.finditer(r"\n(_ZN3moe\w*):(.*?)\.Lfunc_end", text, re.S):
        ins, labels, jumps = parse(f.group(2))
        at_label = {}
        for name, i in labels.items():
            at_label.setdefault(i, []).append(name)
        for i, t in enumerate(ins):
            if t.startswith("buffer_load") and t.endswith(" lds"):
                loads += 1
                regs = scalars(re.search(r"s\[\d+:\d+\]", t).group(0))
                found += [(f.group(1), t, w) for w in written_before(ins, at_label, jumps, i, regs, STATES)]
    return loads, found


def test_the_check_finds_a_hazard():
    text = """
_ZN3moe1fE:
    v_readlane_b32 s9, v1, 0
    s_cbranch_scc1 .LBB0_2
    s_nop 4
.LBB0_2:
    s_mov_b32 m0, s3
    s_nop 0
    buffer_load_dwordx4 v1, s[8:11], 0 offen lds
    v_readfirstlane_b32 s8, v2
    s_nop 4
    buffer_load_dwordx4 v1, s[8:11], 0 offen lds
.Lfunc_end0:
"""
    loads, found = hazards(text)
    assert loads == 2 and [w for _, _, w in found] == ["v_readlane_b32 s9, v1, 0"]


def test_no_load_reads_a_resource_too_early(tmp_path):
    if not os.path.exists(build.hipcc()):
        pytest.skip("hipcc is not here")
    out = tmp_path / "grouped.s"
    subprocess.run([build.hipcc(), *build.common_flags(), "-x", "hip", "--cuda-device-only", "-S",
                    os.path.join(build.CSRC, "grouped.hip"), "-o", str(out)], check=True, capture_output=True)
    loads, found = hazards(out.read_text())
    assert loads > 100  # (no other instruction is taken for one)
    assert not found, found[:4]
