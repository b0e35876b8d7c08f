"""Packing and dequantising an INT4 tensor keeps every launch below 2^32 threads (csrc/moeq_grid.h), on the
CPU: the sizes that pass it in one launch, 2^35 weights, hardly fit a GPU's memory."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_moe_dequant_amd", "csrc")

PROGRAM = r'''
#include <cstdio>
#include "moeq_grid.h"
#include "moeq_int4.h"
int main() {
  if (moeq::INT4_BLOCKS * 256 >= 1l << 32 || moeq::INT4_BLOCKS < 1) return 1;
  // what one launch would take for the largest tensor
  const size_t tiles = moeq::int4_tiles(moeq::INT4_MAX_ROWS, moeq::INT4_MAX_COLS);
  if (tiles / 4 * 256 < 1ul << 32) return 2;
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
