"""sin and cos of the rotary kernels, compiled for the host from their own
source and compared with 64 bits: both ends of each quadrant, where the
integer angle no longer fits an fp32 value, and values in between."""
import subprocess

import pytest

from exact_io_aware_20_gb300 import build

PROGRAM = r"""
#include <cmath>
#include <cstdio>
#include "rope.cuh"
int main() {
  double ends[2] = {0, 0}, inside[2] = {0, 0};
  auto at = [](unsigned long long phase, double* worst) {
    float c, s;
    fa::turn_cos_sin(phase, c, s);
    const double turns = static_cast<double>(static_cast<long long>(phase)) * 0x1p-64;
    const double a = turns * 6.283185307179586476925;
    worst[0] = std::fmax(worst[0], std::fabs(c - std::cos(a)));
    worst[1] = std::fmax(worst[1], std::fabs(s - std::sin(a)));
  };
  for (unsigned long long q = 0; q < 4; ++q)
    for (long long n = 0; n < 4096; ++n) {
      const unsigned long long up = ((1ull << 31) - 1 - n) << 30, down = 0ull - (((1ull << 31) - n) << 30);
      for (unsigned long long low : {0ull, 1ull << 29, (1ull << 30) - 1}) {
        at((q << 62) + up + low, ends);
        at((q << 62) + down + low, ends);
        at((q << 62) + (static_cast<unsigned long long>(n) << 30) + low, ends);
      }
    }
  unsigned long long x = 88172645463325252ull;
  for (int i = 0; i < 4000000; ++i) {
    x ^= x << 13, x ^= x >> 7, x ^= x << 17;
    at(x, inside);
  }
  std::printf("%.4g %.4g %.4g %.4g\n", ends[0], ends[1], inside[0], inside[1]);
}
"""


def test_cos_and_sin_over_the_turn(tmp_path):
    try:
        nvcc = build.nvcc_path()
    except RuntimeError:
        pytest.skip("no nvcc")
    src, exe = tmp_path / "angles.cu", tmp_path / "angles"
    src.write_text(PROGRAM)
    subprocess.run([nvcc] + build.common_flags() + ["-o", str(exe), str(src)], check=True)
    worst = [float(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    # the bound that rope.cuh states
    assert len(worst) == 4 and max(worst) < 7.4e-8, worst
