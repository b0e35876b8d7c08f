"""A workspace for more tokens serves fewer: its size never falls as the tokens grow. On the CPU."""
import ctypes
import os

import pytest

import bit_quantized_moe_dequant_amd as mq

pytestmark = pytest.mark.skipif(not os.path.exists(mq.library_path()), reason="libmoeq.so not built")


def weight(fmt, rows, cols, n):
    return mq.MoeqWeight(fmt, rows, cols, n, 0x10000, 1 << 40, 0x20000, 1 << 40, 0x30000, 0x40000)


SHAPES = [(768, 2048, 256, 6), (512, 2048, 64, 4), (2048, 768, 256, 8), (4096, 2048, 256, 6), (4096, 2048, 256, 8), (1024, 512, 16, 2),
          (256, 256, 8, 1), (7168, 2048, 256, 8), (512, 5888, 9, 3)]
PAIRS = [("int4_g128", "int4_g128"), ("int4z_g32", "int4_g64"), ("int4_g64", "mxfp4"), ("mxfp4", "int4_g128"), ("mxfp4", "mxfp4"),
         ("iq2_xxs", "q2_k"), ("nvfp4", "q2_k"), ("q2_k", "int4z_g64")]


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("shape", SHAPES)
def test_size_never_falls(shape, pair):
    H, I, E, K = shape
    fg, fd = (mq.FMT_BY_NAME[f] for f in pair)
    L = mq.MoeqLayer(H, I, E, K, weight(fg, I, H, E), weight(fg, I, H, E), weight(fd, H, I, E))
    R = mq.MoeqRouter(H, E, K, 1, 1, 1.0, 0x100000, 0)
    lib = mq._lib()
    sh = mq.MoeqShared(256, weight(9, 256, H, 1), weight(9, 256, H, 1), weight(9, H, 256, 1))
    last = (0, 0, 0)
    for T in list(range(1, 400)) + [512, 1000, 1024, 2048, 5000]:
        now = (lib.moeq_workspace_bytes(ctypes.byref(L), T), lib.moeq_moe_workspace_bytes(ctypes.addressof(L), ctypes.addressof(R), None, T),
               lib.moeq_moe_workspace_bytes(ctypes.addressof(L), ctypes.addressof(R), ctypes.addressof(sh), T))
        assert all(n > 0 for n in now), T
        assert all(a <= b for a, b in zip(last, now)), (T, last, now)
        last = now


@pytest.mark.parametrize("cols", [32, 4096, 4128])
def test_linear_int4_size_never_falls(cols):
    last = 0
    for T in range(0, 300):
        n = mq._lib().moeq_linear_int4_workspace_bytes(T, cols)
        assert n >= last
        last = n


@pytest.mark.gpu
def test_one_workspace_for_all_smaller_batches():
    """The workspace of 70 tokens, for fewer on either side of the change from pairs one by one to tiles."""
    import torch

    from tests.int4_ref import Parts
    H, I, E, K = 512, 2048, 64, 4
    layer = mq.Layer(H, I, E, K, *[Parts(12, E, *s, 3).pack() for s in ((I, H), (I, H), (H, I))])
    ws = layer.workspace(70)
    for T in (70, 22, 60, 1, 23, 49, 2):
        print("[case] workspace", T, flush=True)
        g = torch.Generator(device="cuda").manual_seed(T)
        x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
        ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:K] for _ in range(T)]).to(torch.int32)
        rw = torch.rand((T, K), generator=g, device="cuda")
        y = mq.expert_forward(layer, x, ids, rw, ws=ws)
        assert torch.equal(y, mq.expert_forward(layer, x, ids, rw, ws=mq.Layer(H, I, E, K, layer.gate, layer.up, layer.down).workspace(T)))
    assert mq.check_device_error(ws) == 0
