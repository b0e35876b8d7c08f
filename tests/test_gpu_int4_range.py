"""INT4 products at the ends of the value range."""
import numpy as np
import pytest
import torch

import bit_quantized_moe_dequant_amd as mq
from tests.int4_ref import Parts, bf16
from tests.test_gpu_int4 import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [mq.FMT_INT4_G128, mq.FMT_INT4_G32, mq.FMT_INT4Z_G64])
@pytest.mark.parametrize("T", [1, 4, 6, 16, 17, 150])
def test_tokens_near_the_largest_numbers(fmt, T):
    """All signs equal, |x| just below 2^112: a group's sum (16 + q) x stays inside fp32's range, and so do
    the outputs, whose scales are small. The sum of stored scales (64 to 128) times the groups does not."""
    say("large tokens", fmt, T)
    p = Parts(fmt, 1, 40, 4096, seed=3)
    p.q[:] = 0
    if p.z is not None:
        p.z[:] = 15
    p.st = torch.full_like(p.st, 0.01)
    w = p.pack()
    xt, xd = bf16(np.full((T, 4096), 255 * 2.0 ** 104))
    ref = xd @ p.values().T
    assert 1e35 < np.abs(ref).min() and np.abs(ref).max() < 1e37
    y = mq.linear_int4(w, xt, out_dtype=torch.float32).double().cpu().numpy()
    # equal signs: 4096 roundings of the sums with 16 + q and 16 + z, 47 / 15 of the result at most each
    assert np.all(np.abs(y - ref) <= 4096 * 2.0 ** -24 * 2 * 5 * np.abs(ref))


@pytest.mark.parametrize("T", [1, 5])
def test_gate_up_near_the_largest_numbers(T):
    """The same inside the routed experts, pair by pair: gate values of 4 from tiny scales, up near 1e36."""
    say("large gate_up", T)
    H, I, E, K = 4096, 64, 4, 2
    gate, up, down = (Parts(mq.FMT_INT4_G64, E, *s, 5 + i) for i, s in enumerate([(I, H), (I, H), (H, I)]))
    gate.q[:], up.q[:] = 9, 0
    gate.st, up.st = torch.full_like(gate.st, 2.0 ** -121), torch.full_like(up.st, 0.01)
    layer = mq.Layer(H, I, E, K, gate.pack(), up.pack(), down.pack())
    x, xd = bf16(np.full((T, H), 2.0 ** 111))
    ids = torch.tensor([[1, 3]] * T, dtype=torch.int32, device="cuda")
    ws = layer.workspace(T)
    if T > 1:
        mq.route(layer, ids, ws=ws)
    h = mq.gate_up(layer, x, ids, ws=ws).double().cpu().numpy()
    a, b = xd @ gate.values(1).T, xd @ up.values(1).T
    ref = (a / (1 + np.exp(-a)) * b)[:, None, :]
    assert np.isfinite(ref).all() and np.all(np.abs(h - ref) <= 1e-3 * np.abs(ref))
