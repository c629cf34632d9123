"""Which windows fa_cache_keep takes up, compiled for the host from the kernel's
own source: every token whose page it looks up lies in the row of the block
table, whatever the lengths and counts are."""
import subprocess

import pytest

from exact_io_aware_20_gb300 import build

PROGRAM = r"""
#include <climits>
#include <cstdio>
#include "cache_keep.cuh"
int main() {
  long long taken = 0, wrong = 0;
  auto at = [&](long long len, long long n, long long kept, long long N, long long K, long long capacity) {
    const fa::KeepWindow w = fa::keep_window((int)len, (int)n, (int)kept, (int)N, (int)K, capacity);
    // the definition: kept numbers that rise from 0 on and stay below n
    const bool good = 0 <= n && n <= N && n <= len && len <= capacity && 0 <= kept && kept <= K && kept <= n;
    taken += w.valid;
    wrong += w.valid != good;
    if (!w.valid) return;
    // tokens base .. end - 1 are looked up, and none behind the sequence
    wrong += w.base != len - n || w.end != len - n + kept || w.base < 0 || w.end > len || w.end > capacity;
  };
  for (int capacity : {16, 32, 48})
    for (int N : {1, 2, 5, 16, 40})
      for (int K = 1; K <= N; K += 1 + K / 3)
        for (int len = -2; len <= capacity + 2; ++len)
          for (int n = -2; n <= N + 2; ++n)
            for (int kept = -2; kept <= K + 2; ++kept) at(len, n, kept, N, K, capacity);
  // the largest table that is taken, and numbers at the ends of int
  const long long ends[] = {INT_MIN, -1, 0, 1, 7, INT_MAX - 65537ll, INT_MAX - 65536ll, INT_MAX - 65535ll, INT_MAX};
  for (long long len : ends)
    for (long long n : ends)
      for (long long kept : ends)
        for (long long N : {7ll, INT_MAX - 65536ll, (long long)INT_MAX})
          for (long long K : {1ll, 7ll, N}) at(len, n, kept, N, K, INT_MAX - 65536ll);
  std::printf("%lld %lld\n", taken, wrong);
}
"""


def test_windows_stay_in_the_table(tmp_path):
    try:
        nvcc = build.nvcc_path()
    except RuntimeError:
        pytest.skip("no nvcc")
    src, exe = tmp_path / "window.cu", tmp_path / "window"
    src.write_text(PROGRAM)
    subprocess.run([nvcc] + build.common_flags() + ["-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    taken, wrong = map(int, out)
    assert taken > 1000 and wrong == 0
