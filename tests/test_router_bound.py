"""The error bound of the router's fp32 logits (csrc/moeq_router_bound.h) against sums in the
orders and roundings that the matrix instruction is allowed, on the CPU: the rows of a few
large and many small products that come nearest to it."""
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_quantized_moe_dequant_amd", "csrc")


@pytest.fixture(scope="module")
def constants(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("bound")
    src = d / "unit.cpp"
    src.write_text('#include <cstdio>\n#include "moeq_router_bound.h"\nint main() { std::printf("%.17g %d %d", '
                   'moeq::router_unit(), moeq::RM_FLUSH * moeq::RM_STEP, moeq::RM_K); }\n')
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, str(src), "-o", str(d / "unit")], check=True)
    unit, window, k = subprocess.run([str(d / "unit")], check=True, capture_output=True, text=True).stdout.split()
    return float(unit), int(window), int(k)


def truncated(v):
    """To 24 bits, towards zero."""
    m, e = np.frexp(np.float64(v))
    return np.ldexp(np.trunc(np.ldexp(m, 24)), e - 24)


def rounded(v):
    return np.float64(np.float32(v))


def one_after_another(p, k, to):
    acc = np.float64(0)
    for v in p:
        acc = to(acc + v)
    return acc


def accumulator_last(p, k, to):
    acc = np.float64(0)
    for i in range(0, len(p), k):
        s = np.float64(0)
        for v in p[i:i + k]:
            s = to(s + v)
        acc = to(acc + s)
    return acc


def aligned(p, k, to):
    """All addends of an instruction cut at the last bit of the largest."""
    acc = np.float64(0)
    for i in range(0, len(p), k):
        all_ = np.append(p[i:i + k], acc)
        bit = np.ldexp(1.0, int(np.frexp(np.abs(all_).max())[1]) - 24)
        cut = np.trunc if to is truncated else np.rint
        acc = to(np.sum(cut(all_ / bit) * bit))
    return acc


@pytest.mark.parametrize("order", [one_after_another, accumulator_last, aligned])
@pytest.mark.parametrize("to", [rounded, truncated])
def test_no_allowed_sum_passes_the_bound(constants, order, to):
    unit, window, k = constants
    worst = 0.0
    rng = np.random.default_rng(3)
    rows = [np.concatenate([[1.0], np.full(window - 1, p)]) for p in
            (2.0 ** -24 * (1 + 2.0 ** -10), 2.0 ** -23 * (1 - 2.0 ** -10), 2.0 ** -24, 3 * 2.0 ** -24, 2.0 ** -12)]
    rows += [np.concatenate([[1.0], -np.full(window - 1, 2.0 ** -25 * 1.01)]), rng.standard_normal(window)]
    for p in rows:
        size = np.abs(p).sum()  # |W| |x| of x_i = |p_i|^1/2, W_i = +-x_i
        worst = max(worst, abs(order(p, k, to) - p.sum()) / size)
    assert worst <= unit
    if order is one_after_another:  # these rows come near it: half of it rounded, all but a tenth truncated
        assert worst > (0.45 if to is rounded else 0.9) * unit


def test_the_bound_is_not_loose(constants):
    """A larger bound costs exact logits: an instruction's addends at 2^-23 each, and no more than 1 % above."""
    unit, window, k = constants
    n = window // k * (k + 1)
    assert n * 2.0 ** -23 < unit < 1.01 * n * 2.0 ** -23
