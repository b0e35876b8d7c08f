"""Refusals of the INT8 entry points, on the CPU: every bad argument is answered by its
status before anything is launched."""
import ctypes
import os

import pytest
import torch

import bit_quantized_moe_dequant_amd as mq

pytestmark = pytest.mark.skipif(not os.path.exists(mq.library_path()), reason="libmoeq.so not built")

P = ctypes.c_void_p


def fake(fmt=9, rows=256, cols=512, n=1, data=0x10000, scales=0x20000, stride=1 << 20):
    return mq.MoeqWeight(fmt, rows, cols, n, data, stride, scales, stride, 0, 0)


def linear(w, expert=0, xq=0x100000, xs=0x200000, T=4, bias=0, out=0, y=0x300000):
    return mq._lib().moeq_linear_int8(ctypes.byref(w), expert, P(xq), P(xs), T, P(bias), out, P(y), None)


def dynamic(w, expert=0, x=0x100000, T=40, out=0, y=0x300000, ws=0x400000, n=None):
    n = mq._lib().moeq_linear_int8_workspace_bytes(max(T, 0), 512) if n is None else n
    return mq._lib().moeq_linear_int8_dynamic(ctypes.byref(w), expert, P(x), T, None, out, P(y), P(ws), n, None)


def test_sizes():
    assert mq.plane_bytes(9, 7, 48, 0) == 7 * 48 and mq.plane_bytes(9, 7, 48, 1) == 28
    assert mq.plane_bytes(9, 7, 40, 0) == 0 and mq.packed_bytes(9, 4096, 4096) == 4096 * 4096 + 4 * 4096
    lib = mq._lib()
    assert lib.moeq_linear_int8_workspace_bytes(40, 512) >= 40 * 516
    assert lib.moeq_linear_int8_workspace_bytes(1, 512) > 0
    assert lib.moeq_linear_int8_workspace_bytes(4, 40) == 0 == lib.moeq_linear_int8_workspace_bytes(-1, 64)


def test_linear_refusals():
    assert linear(fake(fmt=6, cols=512)) == -2
    assert linear(fake(cols=40)) == -4
    assert linear(fake(cols=65552)) == -4
    assert linear(fake(rows=0)) == -4
    assert linear(fake(rows=(1 << 23) + 1, cols=16)) == -4
    assert linear(fake(data=0x10008)) == -3
    assert linear(fake(scales=0x20002)) == -3
    assert linear(fake(n=2, stride=100)) == -1
    assert linear(fake(n=2, stride=256 * 512 + 4)) == -3
    assert linear(fake(), expert=1) == -1 and linear(fake(), expert=-1) == -1
    assert linear(fake(), T=-1) == -1
    assert linear(fake(), xq=0) == -1 and linear(fake(), xs=0) == -1 and linear(fake(), y=0) == -1
    assert linear(fake(), xq=0x100008) == -3 and linear(fake(), xs=0x200002) == -3
    assert linear(fake(), bias=0x500002) == -3 and linear(fake(), y=0x300002) == -3
    assert linear(fake(), y=0x300001, out=1) == -3
    assert linear(fake(), out=2) == -1
    assert linear(fake(), T=0) == 0


def test_dynamic_refusals():
    assert dynamic(fake(), ws=0) == -5
    assert dynamic(fake(), n=100) == -5
    assert dynamic(fake(), ws=0x400010) == -3
    assert dynamic(fake(), x=0x100008) == -3 and dynamic(fake(), x=0) == -1
    assert dynamic(fake(fmt=1)) == -2
    assert dynamic(fake(), T=0) == 0


def test_quantize_refusals():
    lib, p = mq._lib(), P(0x100000)
    for fn in (lib.moeq_quantize_int8, lib.moeq_quantize_int8_f32):
        assert fn(p, 4, 40, p, p, None) == -4
        assert fn(p, 4, 0, p, p, None) == -4
        assert fn(p, 4, 65552, p, p, None) == -4
        assert fn(P(0x100008), 4, 64, p, p, None) == -3
        assert fn(p, 4, 64, P(0x100004), p, None) == -3
        assert fn(p, 4, 64, p, P(0x100002), None) == -3
        assert fn(p, -1, 64, p, p, None) == -1
        assert fn(None, 4, 64, p, p, None) == -1
        assert fn(p, 0, 64, p, p, None) == 0


def test_other_entry_points_refuse_the_format():
    lib = mq._lib()
    w = fake()
    assert lib.moeq_linear(ctypes.byref(w), 0, P(0x100000), 1, P(0x300000), None) == -2
    mx = lambda r, c: mq.MoeqWeight(1, r, c, 8, 0x10000, 1 << 20, 0x20000, 1 << 20, 0, 0)
    L = mq.MoeqLayer(1024, 512, 8, 2, mx(512, 1024), mx(512, 1024), mx(1024, 512))
    L.down = mq.MoeqWeight(9, 1024, 512, 8, 0x10000, 1 << 20, 0x20000, 1 << 20, 0, 0)
    assert lib.moeq_workspace_bytes(ctypes.byref(L), 1) == 0


def test_copies_of_a_weight_have_descriptors_of_their_own():
    import copy
    import pickle
    w = mq.Weight(9, 64, 32, 1, torch.zeros(64 * 32, dtype=torch.uint8), torch.zeros(256, dtype=torch.uint8))
    w._ref()
    for c in (copy.copy(w), copy.deepcopy(w), pickle.loads(pickle.dumps(w))):
        c._ref()
        assert c._struct is not w._struct and c._struct.data == c.data.data_ptr()
    assert copy.deepcopy(w).data.data_ptr() != w.data.data_ptr()


def test_binding_refusals():
    w = mq.Weight(9, 64, 32, 1, torch.zeros(64 * 32, dtype=torch.uint8), torch.zeros(256, dtype=torch.uint8))
    x = torch.zeros((3, 32), dtype=torch.bfloat16)
    xq, xs = torch.zeros((3, 32), dtype=torch.int8), torch.zeros(3)
    for bad in (lambda: mq.quantize_int8(x.half()), lambda: mq.quantize_int8(x[0]), lambda: mq.quantize_int8(x[:, ::2]),
                lambda: mq.quantize_int8(x, q=torch.zeros((3, 32), dtype=torch.uint8)),
                lambda: mq.linear_int8(w, xq[:, :16], xs), lambda: mq.linear_int8(w, xq, xs[:2]),
                lambda: mq.linear_int8(w, xq, xs, bias=torch.zeros(63)),
                lambda: mq.linear_int8(w, xq, xs, y=torch.zeros((3, 64), dtype=torch.float16)),
                lambda: mq.linear_int8(w, xq, xs, y=torch.zeros((3, 64)), out_dtype=torch.bfloat16),
                lambda: mq.linear_int8_dynamic(w, xq)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ValueError, match="GPU"):  # well-formed, but not on a GPU
        mq.linear_int8(w, xq, xs, y=torch.zeros((3, 64)))


def test_the_binding_knows_which_calls_store_no_codes():
    """linear_int8_dynamic makes no workspace where the library needs none (an empty one of 256
    bytes), and one wherever it does."""
    lib = mq._lib()
    for cols in (16, 64, 4080, 4096, 4112, 8192, 8208, 16384, 16400, 32768, 32784, 65536):
        for T in range(1, 20):
            stored = T > 16 or cols << (T - 1).bit_length() > 65536  # as in linear_int8_dynamic
            assert (lib.moeq_linear_int8_workspace_bytes(T, cols) > 256) == stored, (T, cols)
            got = dynamic(fake(cols=cols), T=T, ws=0, n=0) if stored else None
            assert got in (None, -5)
