"""Launch grids (csrc/grid.h) on the host: for any number of blocks every
dimension holds fewer than 2^32 threads, all blocks are there, and few are
idle. Built with the host C++ compiler, so no GPU is involved.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "moe_expert_dispatch_amd", "csrc", "grid.h")

DRIVER = r"""
#include <cstdio>
#include <initializer_list>
#include "grid.h"
int main() {
  long bad = 0, cases = 0;
  for (int threads : {64, 128, 256, 320, 512, 1024})
    for (int unit : {1, 8})
      for (int bits = 0; bits < 37; ++bits)
        for (int64_t d : {-9, -8, -1, 0, 1, 3, 8, 1000}) {
          int64_t n = (INT64_C(1) << bits) + d;
          if (n < 1 || n > (INT64_C(1) << 36)) continue;
          const moe::Grid g = moe::fold_grid(n, threads, unit);
          const int64_t all = (int64_t)g.x * g.y;
          bad += (uint64_t)g.x * threads >= (UINT64_C(1) << 32);
          bad += g.y < 1 || g.y > 65535;
          bad += all < n || all - n >= (g.y > 1 ? (int64_t)g.y * unit : 1);
          bad += g.y > 1 && g.x % unit != 0;
          ++cases;
        }
  std::printf("%ld %ld\n", cases, bad);
  return bad != 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host C++ compiler")
def test_every_block_is_there_and_no_line_too_long(tmp_path):
    src, exe = tmp_path / "grid_check.cpp", tmp_path / "grid_check"
    src.write_text(DRIVER)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    cases, bad = map(int, out.stdout.split())
    assert cases > 2000 and bad == 0 and out.returncode == 0
