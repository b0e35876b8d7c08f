"""Refusals of the INT4 entry points and of the router's groups, on the CPU; sizes of the planes."""
import ctypes
import os

import pytest
import torch

import bit_quantized_moe_dequant_amd as mq
from tests.int4_ref import FMTS, group_of

pytestmark = pytest.mark.skipif(not os.path.exists(mq.library_path()), reason="libmoeq.so not built")

P = ctypes.c_void_p
A = ctypes.addressof


def fake(fmt=12, rows=256, cols=512, n=1, data=0x10000, scales=0x20000, stride=1 << 20, sstride=1 << 16, scale2=0x30000):
    return mq.MoeqWeight(fmt, rows, cols, n, data, stride, scales, sstride, scale2, 0)


def linear(w, expert=0, x=0x100000, T=3, bias=0, out=0, y=0x200000, ws=0x400000, n=1 << 24):
    return mq._lib().moeq_linear_int4(ctypes.byref(w), expert, P(x), T, P(bias), out, P(y), P(ws), n, None)


def pack(fmt=12, codes=0x100000, scales=0x200000, st=0, zeros=0, rows=32, cols=256, n=1, data=0x300000, out=0x400000, s2=0x500000):
    return mq._lib().moeq_pack_int4(fmt, P(codes), P(scales), st, P(zeros), rows, cols, n, P(data), P(out), P(s2), None)


@pytest.mark.parametrize("fmt", FMTS)
def test_plane_sizes(fmt):
    G = group_of(fmt)
    for rows, cols in [(16, 128), (4096, 4096), (17, 128), (1, G), (33, 3 * G), (5003, 4224)]:
        tiles = -(-rows // 16) * -(-cols // 128)
        assert mq.plane_bytes(fmt, rows, cols, 0) == tiles * 1024
        side = tiles * 16 * (128 // G)
        assert mq.plane_bytes(fmt, rows, cols, 1) == side * (3 if fmt >= mq.FMT_INT4Z_G32 else 2)
        assert mq.packed_bytes(fmt, rows, cols) == mq.plane_bytes(fmt, rows, cols, 0) + mq.plane_bytes(fmt, rows, cols, 1) + 4
    assert mq.plane_bytes(fmt, 16, G + 16, 0) == 0 and mq.plane_bytes(fmt, 0, 128, 0) == 0 and mq.plane_bytes(fmt, 16, 128, 2) == 0
    assert mq.plane_bytes(fmt, (1 << 23) + 1, 128, 0) == 0 and mq.plane_bytes(fmt, 16, (1 << 20) + 128, 0) == 0
    assert mq.plane_bytes(16, 16, 128, 0) == 0


def test_pack_refusals():
    assert pack(fmt=9) == -2 and pack(fmt=16) == -2
    assert pack(codes=0) == -1 and pack(scales=0) == -1 and pack(data=0) == -1 and pack(out=0) == -1 and pack(s2=0) == -1
    assert pack(n=-1) == -1 and pack(st=2) == -1 and pack(zeros=0x600000) == -1 and pack(fmt=15) == -1
    assert pack(cols=192) == -4 and pack(rows=0) == -4
    assert pack(data=0x300008) == -3 and pack(out=0x400008) == -3 and pack(s2=0x500002) == -3 and pack(scales=0x200001) == -3
    assert pack(n=0) == 0


def test_linear_refusals():
    assert linear(fake(T := 12), T=0) == 0
    assert linear(fake(fmt=9)) == -2 and linear(fake(fmt=16)) == -2 and linear(fake(fmt=1)) == -2
    assert linear(fake(), expert=1) == -1 and linear(fake(), expert=-1) == -1 and linear(fake(), T=-1) == -1
    assert linear(fake(), x=0) == -1 and linear(fake(), y=0) == -1 and linear(fake(), out=2) == -1
    assert linear(fake(scale2=0)) == -1 and linear(fake(data=0)) == -1 and linear(fake(scales=0)) == -1
    assert linear(fake(n=0)) == -1 and linear(fake(n=2, stride=1024)) == -1 and linear(fake(n=2, sstride=16)) == -1
    assert linear(fake(cols=448)) == -4 and linear(fake(rows=0)) == -4
    assert linear(fake(data=0x10008)) == -3 and linear(fake(scales=0x20008)) == -3 and linear(fake(n=2, sstride=(1 << 16) + 8)) == -3
    assert linear(fake(), x=0x100008) == -3 and linear(fake(), y=0x200002) == -3 and linear(fake(), bias=0x300002) == -3
    assert linear(fake(), T=17, ws=0) == -5 and linear(fake(), T=17, n=100) == -5 and linear(fake(), T=17, ws=0x400010) == -3
    lib = mq._lib()
    assert lib.moeq_linear_int4_workspace_bytes(16, 512) == 256
    assert lib.moeq_linear_int4_workspace_bytes(17, 4128) >= 17 * 4224 * 2
    assert lib.moeq_linear_int4_workspace_bytes(-1, 512) == 0 and lib.moeq_linear_int4_workspace_bytes(3, 100) == 0
    # the other linears and prefill stages do not take the format
    w = fake()
    assert lib.moeq_linear(ctypes.byref(w), 0, P(0x100000), 3, P(0x200000), None) == -2
    assert lib.moeq_linear_int8(ctypes.byref(w), 0, P(0x100000), P(0x100000), 3, None, 0, P(0x200000), None) == -2


def layer(fg=12, fd=11, H=1024, I=512, E=8, K=2):
    w = lambda f, r, c: fake(f, r, c, E, stride=1 << 20, sstride=1 << 18)
    return mq.MoeqLayer(H, I, E, K, w(fg, I, H), w(fg, I, H), w(fd, H, I))


def test_layers():
    lib = mq._lib()
    size = lambda L, T=1: lib.moeq_workspace_bytes(ctypes.byref(L), T)
    assert 0 < size(layer()) < size(layer(), 64)
    assert size(layer(fd=1)) > 0 and size(layer(fg=1)) > 0  # beside another format
    bad = layer()
    bad.up.fmt = 11  # gate and up agree
    assert size(bad) == 0
    bad = layer()
    bad.down.scale2 = 0
    assert size(bad) == 0
    assert size(layer(I=448)) > 0 and size(layer(fd=12, I=448)) == 0  # whole groups
    L, n = layer(), 1 << 28
    xs = (P(0x200000), P(0x300000), P(0x400000))
    assert lib.moeq_prefill_down(ctypes.byref(L), xs[0], xs[0], xs[1], xs[2], 3, P(0x500000), P(0x600000), n, None) == -2


def router(E=16, K=2):
    return mq.MoeqRouter(1024, E, K, 0, 1, 1.0, 0x100000, 0)


def topk(R, G, T=3):
    g = None if G is None else A(G)
    return mq._lib().moeq_router_topk_groups(ctypes.byref(R), g, P(0x200000), T, P(0x300000), P(0x400000), P(0x500000), 1 << 20, None)


def test_group_refusals():
    G = mq.MoeqRouterGroups
    assert topk(router(), G(4, 2, 0), T=0) == 0 and topk(router(), None, T=0) == 0
    for bad, code in ((G(0, 0, 0), -1), (G(4, 0, 0), -1), (G(4, 5, 0), -1), (G(4, 2, 2), -1), (G(4, 2, -1), -1),
                      (G(3, 2, 0), -4), (G(5, 2, 1), -4)):
        assert topk(router(), bad) == code
    assert topk(router(K=5), G(8, 2, 0)) == -1  # five experts out of two groups of two
    assert topk(router(E=130), G(65, 3, 0)) == -4
    mx = lambda r, c: mq.MoeqWeight(1, r, c, 16, 0x10000, 1 << 20, 0x20000, 1 << 20, 0, 0)
    L, R, g = mq.MoeqLayer(1024, 512, 16, 2, mx(512, 1024), mx(512, 1024), mx(1024, 512)), router(), G(3, 2, 0)
    call = lambda at, T: mq._lib().moeq_moe_forward_groups(A(L), A(R), at, None, P(0x200000), T, P(0x300000), None, None, P(0x500000),
                                                           1 << 30, None)
    assert call(A(g), 3) == -4 and call(None, 0) == 0


def test_binding_refusals():
    w = torch.zeros((16, 64), dtype=torch.bfloat16)
    for kw in (dict(n_groups=3), dict(n_groups=0), dict(n_groups=4, top_groups=0), dict(n_groups=4, top_groups=5),
               dict(n_groups=4, top_groups=1, group_score="mean"), dict(n_groups=8, top_groups=1)):
        with pytest.raises(ValueError):
            mq.Router(w, 3, **kw)
    codes, scales = torch.zeros((2, 20, 128), dtype=torch.uint8), torch.ones((2, 20, 4), dtype=torch.bfloat16)
    for bad in (lambda: mq.pack_int4(codes.int(), scales), lambda: mq.pack_int4(codes, scales.float()),
                lambda: mq.pack_int4(codes, scales[:, :, :3]), lambda: mq.pack_int4(codes, scales[0]),
                lambda: mq.pack_int4(codes, scales[:, :10]), lambda: mq.pack_int4(codes[:, :, ::2], scales),
                lambda: mq.pack_int4(codes, scales, torch.zeros((2, 20, 4))), lambda: mq.pack_int4(None, scales),
                lambda: mq.pack_int4(codes, scales, w=mq.Weight.empty(mq.FMT_INT4_G64, 20, 512, 2, "cpu"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ValueError, match="GPU"):
        mq.pack_int4(codes, scales, w=mq.Weight.empty(mq.FMT_INT4_G64, 20, 256, 2, "cpu"))
    wt = mq.Weight.empty(mq.FMT_INT4_G64, 20, 256, 1, "cpu")
    x = torch.zeros((3, 256), dtype=torch.bfloat16)
    for bad in (lambda: mq.linear_int4(wt, x[:, :128]), lambda: mq.linear_int4(wt, x.float()),
                lambda: mq.linear_int4(wt, x, bias=torch.zeros(19)), lambda: mq.linear_int4(wt, x, y=torch.zeros((2, 20))),
                lambda: mq.linear_int4(wt, x, out_dtype=torch.float16)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ValueError, match="GPU"):
        mq.linear_int4(wt, x)
