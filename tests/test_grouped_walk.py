"""The walk over the tiles of the products by expert (csrc/tile_walk.h, compiled for the host): every tile of a plan once,
and no tile outside of its expert's where the plan's starts change between the two times that a workgroup reads them (a
caller's mistake, which must not lead out of a buffer)."""
import shutil
import subprocess

import pytest

from mixture_experts_ffn_topk_amd import build

PROGRAM = r"""
#include <cstdio>
#include <random>
#include <vector>
#include "tile_walk.h"

int main() {
  std::mt19937 r(1);
  long outside = 0, twice = 0, tiles = 0, refused = 0;
  for (int turn = 0; turn < 3000; ++turn) {
    const int E = 1 + r() % 12, p_tiles = 1 + r() % 20, most_q = turn % 2 ? 8 : 1 + r() % 8;
    std::vector<int> before(E), now(E);  // q-tiles of the experts at the first and at the second reading
    for (int& n : before) n = r() % 3 ? r() % 20 : 0;
    for (int e = 0; e < E; ++e) now[e] = turn < 1000 || r() % 2 ? before[e] : r() % 20;
    std::vector<std::vector<int>> seen(E);
    for (int e = 0; e < E; ++e) seen[e].assign(now[e] * p_tiles, 0);
    int upto = 0;
    for (int e = 0, at = 0; e < E; ++e) {
      upto += before[e] * p_tiles;
      for (; at < upto; ++at) {
        const moe::TileIn t = moe::tile_in(at - (upto - now[e] * p_tiles), now[e], p_tiles, most_q);
        ++tiles;
        if (!t.ok) { ++refused; continue; }
        if (t.q < 0 || t.q >= now[e] || t.p < 0 || t.p >= p_tiles) { ++outside; continue; }
        twice += seen[e][t.q * p_tiles + t.p]++;
      }
    }
    if (turn < 1000 && refused) return 2;
    if (turn < 1000)
      for (auto& s : seen) for (int n : s) if (n != 1) return 3;
  }
  std::printf("%ld %ld %ld %d\n", outside, twice, tiles, refused > 0);
}
"""


def test_every_tile_once_and_none_outside(tmp_path):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(PROGRAM)
    # (a division by zero ends the program)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.returncode
    outside, twice, tiles, refused = map(int, run.stdout.split())
    assert outside == 0 and twice == 0 and tiles > 100000 and refused
