"""Build libmoeq.so (gfx950) in-tree with hipcc.

Usage: python -m bit_quantized_moe_dequant_amd.build [--jobs N]

Each .hip source is compiled to an object in parallel, then linked into
bit_quantized_moe_dequant_amd/libmoeq.so. Packed fp32 instructions are disabled
for device code (they are generated only by the compiler, never written by hand).
"""
from __future__ import annotations

import argparse
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmoeq.so")

SOURCES = ["moeq_api.hip", "moeq_gemv.hip", "moeq_aux.hip", "moeq_prefill.hip", "moeq_linear.hip", "moeq_grouped.hip", "moeq_gu_mx4.hip", "moeq_linear_mx8.hip", "moeq_batched.hip", "moeq_convert.hip", "moeq_down_q2k.hip", "moeq_int8.hip", "moeq_router.hip", "moeq_moe.hip", "moeq_int4.hip", "moeq_int4_tiled.hip", "synth.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-function",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE, "-I", CSRC,
]

# Sums that the vector unit reads after every few matrix instructions: kept in vector registers
# (in accumulation registers each would be moved first, 64 of 400 operations of a step). A
# compiler that does not know such a switch builds the file without it: the same results, slower.
EXTRA = {"moeq_int4_tiled.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]}


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    def run(extra):
        cmd = [HIPCC, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        return subprocess.run(cmd, capture_output=True, text=True)

    extra = EXTRA.get(src, [])
    r = run(extra)
    if r.returncode != 0 and extra and "Unknown command line argument" in r.stderr:
        print(f"{src}: built without {' '.join(extra)}, which this compiler does not know", file=sys.stderr)
        r = run([])
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def build(jobs: int | None = None, verbose: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = [s for s in SOURCES if os.path.exists(os.path.join(CSRC, s))]
    jobs = jobs or min(len(srcs), os.cpu_count() or 4, 8)
    with ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--jobs", type=int, default=None)
    a = ap.parse_args()
    try:
        build(a.jobs)
    except RuntimeError as e:
        print(e, file=sys.stderr)
        sys.exit(1)
