"""The ranges that bound the copies of the 8-bit floating-point tiles, compiled for the host: every lane of every
copy under the hardware's check, offset >= range - scalar offset in 32 bits."""

import os
import subprocess

from conftest import ROOT

CSRC = os.path.join(ROOT, "moe_expert_grouped_group_amd", "csrc")

# The weights of the last expert: a column tile's 256 rows in two runs of 16 for each 32 rows, 8 waves, two copies
# of 8 rows by 128 bytes a run; the last stage's chunks past K are marked as out of range.
PROGRAM = r"""
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include "fp8_tile_ranges.h"

int main() {
  const uint32_t out = 0xFFFFFF00u;
  long bad = 0, seen = 0, empty = 0;
  auto check = [&](int64_t N, int64_t K, int64_t n0) {
    const int64_t left = N - n0;
    for (int64_t st = 0; st * 128 < K; ++st)
      for (int half = 0; half < 2; ++half) {
        const uint32_t range = (uint32_t)mx::rows_range(left - 16 * half, K, K);
        const uint32_t soff = mx::row_offset(range, (uint32_t)(st * 128));
        empty += range == 0;
        bool wrong = soff > range || (range != 0 && soff != st * 128);
        for (int wave = 0; wave < 8; ++wave)
          for (int j = 0; j < 2; ++j)
            for (int lane = 0; lane < 64; ++lane) {
              const uint32_t row = 32 * wave + 8 * j + lane / 8, chunk = ((lane & 7) ^ ((4 * (j & 1) + (lane >> 4)) & 7)) * 16;
              const bool past = st * 128 + chunk >= K;
              const uint32_t offset = (row * (uint32_t)K + chunk) | (past ? out : 0u);
              const bool read = offset < range - soff;
              const bool there = (int64_t)row + 16 * half < left && !past;
              wrong |= read != there;
              ++seen;
            }
        if (wrong && bad++ < 8) std::printf("N %ld K %ld n0 %ld stage %ld half %d\n", (long)N, (long)K, (long)n0, (long)st, half);
      }
  };
  for (int64_t K : {16, 112, 128, 144, 192, 240, 256, 272, 400, 1024, 4112})
    for (int64_t N = 8; N <= 1040; N += 8)
      for (int64_t n0 = 0; n0 < N; n0 += 256) check(N, K, n0);
  std::printf("%ld seen, %ld empty, %ld bad\n", seen, empty, bad);
  return bad != 0;
}
"""


def test_lanes_of_the_weights_copies(tmp_path):
    """A lane reads where it has a row and a chunk, and nowhere else; tiles of 8 and 16 columns among them."""
    source, program = tmp_path / "ranges.cpp", tmp_path / "ranges"
    source.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", CSRC, str(source), "-o", str(program)], check=True)
    done = subprocess.run([str(program)], stdout=subprocess.PIPE, text=True, timeout=600)
    assert done.returncode == 0, done.stdout
    assert int(done.stdout.split()[2]) > 100, done.stdout
