"""Tokens to a launch (csrc/moeq_grid.h) keep every grid below 2^32 threads, whatever tile the
launch takes, on the CPU: the sizes that reach the limit do not fit a GPU's memory."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_quantized_moe_dequant_amd", "csrc")

PROGRAM = r'''
#include <cstdio>
#include <initializer_list>
#include "moeq_grid.h"
int main() {
  const int tiles[][3] = {{32, 64, 128}, {64, 64, 256}, {128, 64, 512}, {256, 128, 512}, {256, 256, 512}, {128, 128, 512}};
  for (int rows : {1, 31, 33, 4096, 1 << 18, (1 << 18) + 1, 5000003, (1 << 23) - 1, 1 << 23}) {
    const long t = moeq::int8_tokens(rows);
    if (t < 64 || t > 1 << 16) return 1;
    for (auto& m : tiles) {
      const long blocks = ((long)rows + m[0] - 1) / m[0] * ((t + m[1] - 1) / m[1]);
      if (blocks > moeq::GRID_MAX_BLOCKS || blocks * m[2] >= 1l << 32) return 2;
    }
  }
  if (moeq::int8_tokens(8192) != 1 << 16) return 3;
  const long tiles_router = 1024 / 64 * (moeq::ROUTER_TOKENS / 64), groups = moeq::ROUTER_TOKENS / 4;
  if ((tiles_router + 256) * 256 >= 1l << 32 || groups * 256 >= 1l << 32 || tiles_router < 256) return 4;
  std::puts("ok");
}
'''


def test_no_grid_passes_its_limit(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    (tmp_path / "grid.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, str(tmp_path / "grid.cpp"), "-o", str(tmp_path / "grid")], check=True)
    r = subprocess.run([str(tmp_path / "grid")], capture_output=True, text=True)
    assert (r.returncode, r.stdout) == (0, "ok\n")
