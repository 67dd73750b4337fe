"""The quotient that decides the codes of 8-bit floating point next to a border, compiled for the host."""

import os
import subprocess

from conftest import ROOT

CSRC = os.path.join(ROOT, "moe_expert_grouped_group_amd", "csrc")

# Nearest e4m3 value (as its place among the finite ones) of the fp32 quotient, and of x / scale from the borders
# themselves: a border has 5 bits and a scale 24, so their product is exact in float64 and no division decides.
PROGRAM = r"""
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>
#include "fp8_quotient.h"

static std::vector<double> codes;

static int nearest(double size, double unit) {   // size / unit, ties to even
  int lo = 0, hi = (int)codes.size() - 1;         // codes[lo] unit <= size, as far as there are codes
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (codes[mid] * unit <= size) lo = mid; else hi = mid;
  }
  const double middle = (codes[lo] + codes[hi]) / 2 * unit;
  return size > middle || (size == middle && lo % 2 == 1) ? hi : lo;
}

int main() {
  for (int m = 0; m < 8; ++m) codes.push_back(m / 512.0);
  for (int e = 1; e < 16; ++e)
    for (int m = 0; m < 8 && !(e == 15 && m == 7); ++m) codes.push_back(std::ldexp(8 + m, e - 10));
  std::mt19937 random(1);
  std::vector<float> scales;
  // (2^-149 / 448 upwards: the smallest scale of a bf16 block is its smallest number over 448)
  for (int e = -141; e <= 119; ++e) {
    scales.push_back((float)std::ldexp(1.0, e));
    for (int i = 0; i < 2; ++i) scales.push_back((float)std::ldexp(1.0 + random() / 4294967296.0, e));
  }
  long bad = 0, seen = 0, tiny = 0;
  for (float scale : scales)
    for (uint32_t b = 0; b < 0x7F80; ++b)
      for (int sign = 0; sign < 2; ++sign) {
        const uint32_t bits = (b | (uint32_t)sign << 15) << 16;
        float x;
        std::memcpy(&x, &bits, 4);
        if (std::fabs(x) > 448.0 * (double)scale * (1 + 0x1p-20)) continue;   // no value of such a block
        const float v = mx::exact_quotient(x, scale);
        ++seen;
        tiny += std::fabs((double)x) < 0x1p-150 * (double)scale;
        const bool right = v == v && std::signbit(v) == std::signbit(x) &&
                           nearest(std::fabs((double)v), 1.0) == nearest(std::fabs((double)x), (double)scale);
        if (!right && bad++ < 8) std::printf("x %a scale %a: %a\n", x, scale, v);
      }
  std::printf("%ld seen, %ld tiny, %ld bad\n", seen, tiny, bad);
  return bad != 0;
}
"""


def test_every_value_under_scales_of_every_size(tmp_path):
    """Every finite bf16 value with every size of scale that a block holding it can have, quotients below the
    smallest number among them: the fp32 quotient rounds to the code of the exact one, with the value's sign."""
    source, program = tmp_path / "quotient.cpp", tmp_path / "quotient"
    source.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-ffp-contract=off", "-I", CSRC, str(source), "-o", str(program)],
                   check=True)
    done = subprocess.run([str(program)], stdout=subprocess.PIPE, text=True, timeout=600)
    assert done.returncode == 0, done.stdout
    assert int(done.stdout.split()[0]) > 10_000_000 and int(done.stdout.split()[2]) > 100_000, done.stdout
