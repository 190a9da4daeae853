"""The parts of a split contraction (csrc/split_rows.h) on the host: they are the slot's rows, each once and
in order, in whole slices; and at the last row that 31 bits may hold no sum passes them (the program is
built to end at the first signed overflow). Built with the host C++ compiler, so no GPU is involved.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "moe_expert_dispatch_amd", "csrc", "split_rows.h")

DRIVER = r"""
#define __host__
#define __device__
#define __forceinline__ inline
#include <cstdio>
#include <initializer_list>
#include "split_rows.h"
int main() {
  long bad = 0, cases = 0;
  const int most = 2147483647 - 1024;  // rows are fewer than 2^31 - 1024
  auto check = [&](int lo, int hi) {
    for (int slice : {32, 64, 128})
      for (int splits = 1; splits <= 16; ++splits) {
        int at = lo;
        for (int split = 0; split < splits; ++split) {
          int row0 = -1, rows = -1;
          moe::split_rows(lo, hi, slice, splits, split, &row0, &rows);
          bad += row0 != at || rows < 0 || rows > hi - row0;
          bad += row0 + rows < hi && rows % slice != 0;
          at = row0 + rows;
        }
        bad += at != hi;
        ++cases;
      }
  };
  for (int n = 0; n <= 2100; n += n < 300 ? 1 : 37)
    for (int lo : {0, 1, 1000, most - 2100}) check(lo, lo + n);
  for (int n : {0, 1, 31, 127, 128, 129, 1919, 1920, 1921, 1 << 20, 1 << 30, most}) check(most - n, most);
  std::printf("%ld %ld\n", cases, bad);
  return bad != 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host C++ compiler")
def test_parts_are_the_rows_in_order_without_overflow(tmp_path):
    src, exe = tmp_path / "split_rows_check.cpp", tmp_path / "split_rows_check"
    src.write_text(DRIVER)
    subprocess.run(["g++", "-O1", "-std=c++17", "-ftrapv", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out
    cases, bad = map(int, out.stdout.split())
    assert cases > 10000 and bad == 0
