"""The cutting of rows into units, parts and groups of steps (row_split.h), on the
CPU: the code that the kernels compile, walked over widths, alignments, numbers of
blocks and ranks."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "linear_layers_b200", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "row_split.h"
using namespace tpl;
constexpr int kWide = %(threads)d * %(units)d, kMost = %(groups)d;

template <int kN>
long walk(int64_t lo, int64_t hi) {
  long bad = 0;
  for (int64_t v = lo; v <= hi; ++v)
    for (int slices = 1; slices <= 8; slices *= 2) {
      const int room_steps = steps_of(Part(static_cast<int>(v / kN), 0, slices).last, kWide);
      const int log = group_log_of(room_steps, kMost);
      const int room = (groups_of(room_steps, log) + 3) / 4 * 4;
      if (room > kMost) ++bad;
      for (int64_t f0 = 0; f0 < kN; ++f0) {
        const RowSplit<kN> row(f0, v);
        if (row.head + row.units * kN + row.tail != v || row.tail >= kN || row.tail < 0 ||
            (row.units && (f0 + row.head) %% kN))
          ++bad;
        int at = 0;
        for (int rank = 0; rank < slices; ++rank) {
          const Part p(row.units, rank, slices);
          if (p.first != at || p.last < p.first) ++bad;
          at = p.last;
          const int steps = steps_of(p.last - p.first, kWide), groups = groups_of(steps, log);
          if (groups > room || (groups << log) < steps) {
            if (bad++ == 0)
              std::printf("v %%lld, %%d per unit, start %%lld, block %%d of %%d: %%d groups, room %%d\n",
                          static_cast<long long>(v), kN, static_cast<long long>(f0), rank, slices,
                          groups, room);
          }
        }
        if (at != row.units) ++bad;
      }
    }
  return bad;
}

int main() {
  long bad = walk<4>(1, 2500) + walk<8>(1, 2500);
  // around the widths of 32·2^k steps of a block, where the groups double
  for (int k = 0; k <= 7; ++k)
    for (int64_t slices = 1; slices <= 8; slices *= 2) {
      const int64_t f = slices * (32LL << k) * kWide * 4, b = 2 * f;
      if (f < (1 << 30) - 200) bad += walk<4>(f - 20, f + 120);
      if (b < (1 << 30) - 200) bad += walk<8>(b - 20, b + 120);
    }
  bad += walk<4>((1 << 30) - 20, 1 << 30) + walk<8>((1 << 30) - 20, 1 << 30);
  std::printf("bad %%ld\n", bad);
  return bad != 0;
}
"""


def test_no_block_has_more_groups_than_its_launch_makes_room_for(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    text = open(os.path.join(CSRC, "logprobs.cu")).read()
    value = lambda name: int(re.search(rf"constexpr int {name} = (\d+);", text).group(1))  # noqa: E731
    src = tmp_path / "walk.cpp"
    src.write_text(PROGRAM % {"threads": value("kThreads"), "units": value("kUnits"),
                              "groups": value("kGroups")})
    exe = tmp_path / "walk"
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
