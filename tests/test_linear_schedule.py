"""The schedule of the product's form for many tiles, walked on the CPU from its own source
(csrc/kda_linear_tiles.h, compiled by the host's compiler): each part of the output
belongs to one warp once, and each residual that a warp waits for was asked for."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_attention_recurrent_kda_gb300", "csrc")

# argv: rows outer pairs, any number of times.  A line for each: parts that were waited for
# without having been asked for, asked for and not waited for, or twice in a buffer; elements
# that were worked on; parts that were done twice; tiles that the warps did not pass.
PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include <set>
#include "kda_linear_tiles.h"
using namespace kda::linear;

int main(int argc, char **argv) {
  for (int i = 1; i + 2 < argc; i += 3) {
    const int rows = atoi(argv[i]), outer = atoi(argv[i + 1]), most = atoi(argv[i + 2]);
    long long bad = 0, twice = 0, elements = 0, passed = 0;
    const int tiles = Chunks{rows, outer, 0, 1, 0, 0}.tiles_m() * Chunks{rows, outer, 0, 1, 0, 0}.tiles_n();
    const int pairs = tiles < most ? tiles : most;
    std::set<long long> seen;
    for (int pair = 0; pair < pairs; ++pair)
      for (int warp = 0; warp < 32; ++warp) {     // 2 CTAs x 4 x 4
        const Chunks c = {rows, outer, pair, pairs, warp / 16 * 128 + warp / 4 % 4 * kChunkRows,
                          warp % 4 * kChunkCols};
        bool held = false;                        // the buffer: a residual
        Tile of = {-1, -1};
        int count = 0;
        walk_chunks(
            c,
            [&](const Tile &at) {
              bad += held;
              held = true;
              of = at;
            },
            [&](int q, const Tile &at, bool there) {
              bad += q != count++ || there != (at.row < rows && at.col < outer);
              if (!there) return true;
              bad += !held || of.row != at.row || of.col != at.col;
              held = false;
              twice += !seen.insert(static_cast<long long>(at.row) << 32 | at.col).second;
              const int high = rows - at.row < kChunkRows ? rows - at.row : kChunkRows;
              const int wide = outer - at.col < kChunkCols ? outer - at.col : kChunkCols;
              elements += static_cast<long long>(high) * wide;
              return true;
            });
        bad += held;
        passed += count;
      }
    printf("%lld %lld %lld %lld\n", bad, elements - static_cast<long long>(rows) * outer, twice,
           32ll * tiles - passed);
  }
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    at = tmp_path_factory.mktemp("schedule")
    (at / "walk.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(at / "walk.cpp"), "-o",
                    str(at / "walk")], check=True)

    def run(cases):
        out = subprocess.run([str(at / "walk"), *(str(v) for case in cases for v in case)], check=True,
                             capture_output=True, text=True).stdout
        return [tuple(int(v) for v in line.split()) for line in out.splitlines()]
    return run


pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")


@pytest.mark.parametrize("rows,outer", [
    (2000, 4096), (1500, 4096), (2000, 7168), (4000, 4096), (600, 20480), (10000, 7168), (5000, 5000),
    (4160, 7200), (4163, 7203), (16384, 2880), (16384, 2881), (1500, 4100), (9159, 7168), (1024, 4096),
    (65, 40000), (40000, 8), (257, 257), (256, 256), (1, 1), (255, 65), (2049, 2047)])
def test_each_residual_that_is_waited_for_was_asked_for(walk, rows, outer):
    cases = [(rows, outer, pairs) for pairs in (1, 2, 3, 7, *range(60, 77))]
    for case, got in zip(cases, walk(cases), strict=True):
        assert got == (0, 0, 0, 0), case
