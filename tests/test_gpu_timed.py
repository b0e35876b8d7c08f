"""gate_up_timed records its events at every size, whichever kernel runs."""
import sys

import pytest
import torch

import bit_quantized_moe_dequant_amd as mq
from tests.int4_ref import Parts

pytestmark = pytest.mark.gpu


def random_weight(fmt, rows, cols, E, g):
    if fmt >= mq.FMT_INT4_G32:
        return Parts(fmt, E, rows, cols, rows).pack()
    w = mq.Weight.empty(fmt, rows, cols, E)
    w.data.copy_(torch.randint(0, 256, w.data.shape, generator=g, device="cuda", dtype=torch.uint8))
    w.scales.copy_(torch.randint(110, 118, w.scales.shape, generator=g, device="cuda", dtype=torch.uint8))
    if fmt == mq.FMT_IQ2_XXS:
        w.grid = torch.randint(1, 40, (2048,), generator=g, device="cuda", dtype=torch.uint8)
    return w


@pytest.mark.parametrize("fmt", ["int4_g128", "int4z_g32", "iq2_xxs", "mxfp4", "nvfp4", "q2_k"])
@pytest.mark.parametrize("T", [1, 3, 40, 130])
def test_events_are_recorded_by_the_call(fmt, T):
    print("[case] timed", fmt, T, file=sys.stderr, flush=True)
    H, I, E, K = 1024, 512, 12, 4
    g = torch.Generator(device="cuda").manual_seed(T)
    f = mq.FMT_BY_NAME[fmt]
    layer = mq.Layer(H, I, E, K, *[random_weight(f, *s, E, g) for s in ((I, H), (I, H), (H, I))])
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:K] for _ in range(T)]).to(torch.int32)
    ws = layer.workspace(T)
    if T > 1:
        mq.route(layer, ids, ws=ws)
    want = mq.gate_up(layer, x, ids, ws=ws)
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(40):  # milliseconds between the events, until the call records them again
        big = torch.ones((4096, 4096), device="cuda") @ torch.ones((4096, 4096), device="cuda")
    stop.record()
    torch.cuda.synchronize()
    before = start.elapsed_time(stop)
    assert before > 10
    h = mq.gate_up_timed(layer, x, ids, start, stop, ws=ws)
    torch.cuda.synchronize()
    ms = start.elapsed_time(stop)
    assert 0 < ms < 1.0, (before, ms)
    assert torch.equal(h.view(torch.int32), want.view(torch.int32))
