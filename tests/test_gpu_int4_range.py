"""INT4 products at the ends of the value range.

Between rows of bf16 and fp16 (beyond 16 tokens): a row is multiplied by a power of two that brings its
largest value into [2^14, 2^15), where fp16's smallest step is 2^-24. A bf16 value of eight bits keeps
them all down to 2^-31 of that power of two (2^-31 is 2^-17 there, whose eighth bit is 2^-24); below, it
is rounded to half a step, 2^-25 there, 2^-39 of the power of two.

An intermediate value of fp32 (the tiled down) is two such numbers: 22 bits, 2^-23 of it, while the second
is normal, and 2^-39 of the power of two at most where it is not."""
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


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("low", [30, 36, 44])
@pytest.mark.parametrize("T", [3, 16, 17, 70])
def test_small_values_beside_a_large_one(low, out, T):
    """One value of 1 to a token, where the weights are 0, and the others 2^-low of it: up to 16 tokens
    and down to 2^-31 nothing is lost, below that half a step, 2^-39 for each value."""
    say("small beside large", low, out, T)
    p = Parts(mq.FMT_INT4_G64, 1, 50, 640, seed=low)
    p.q[:, :, 77] = 8
    w = p.pack()
    g = np.random.default_rng(T)
    x = (1 + g.random((T, 640))) * np.where(g.random((T, 640)) < 0.5, -1, 1) * 2.0 ** -low
    x[:, 77] = 1.0
    xt, xd = bf16(x)
    ref = xd @ p.values().T
    small = xd.copy()
    small[:, 77] = 0
    tol = p.tol(small, 0) + 2.0 ** -23 * np.abs(ref)
    if T <= mq.INT4_FEW_T:  # there the group that holds the 1 has it in its sum as 24 x 1 before it is taken off
        one = np.zeros_like(xd)
        one[:, 77] = 1
        tol = tol + p.tol(one, 0)
    elif low > 30:  # 2^-25 of the scaled value: 2^-39 of 1, for each of the row's values
        tol = tol + 2.0 ** -39 * np.abs(p.values()).sum(axis=1)
    if out == torch.bfloat16:
        tol = tol + 1.01 * 2.0 ** -8 * np.abs(ref)
    y = mq.linear_int4(w, xt, out_dtype=out).double().cpu().numpy()
    assert np.all(np.abs(y - ref) <= tol), float((np.abs(y - ref) / tol).max())


@pytest.mark.parametrize("low", [8, 18, 30, 45])
def test_small_intermediate_values_beside_a_large_one(low):
    """The down stage of 40 tokens by expert, every h with one value of 1 where the weights are 0."""
    say("small h beside large", low)
    T, H, I, E, K = 40, 1024, 768, 6, 3
    gate, up, down = (Parts(mq.FMT_INT4_G64, E, *s, 5 + i) for i, s in enumerate([(I, H), (I, H), (H, I)]))
    down.q[:, :, 77] = 8
    layer = mq.Layer(H, I, E, K, gate.pack(), up.pack(), down.pack())
    g = np.random.default_rng(low)
    h = (1 + g.random((T, K, I))) * np.where(g.random((T, K, I)) < 0.5, -1, 1) * 2.0 ** -low
    h[:, :, 77] = 1.0
    h = h.astype(np.float32)
    ids = np.stack([g.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    rw = (0.2 + g.random((T, K))).astype(np.float32)
    ti, tr = torch.from_numpy(ids).cuda(), torch.from_numpy(rw).cuda()
    ws = layer.workspace(T)
    mq.route(layer, ti, ws=ws)
    y = mq.down(layer, torch.from_numpy(h).cuda(), ti, tr, ws=ws).double().cpu().numpy()
    hd = h.astype(np.float64)
    hd[:, :, 77] = 0
    ref, tol = np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        t, k = np.nonzero(ids == e)
        r, v, w = rw[t, k].astype(np.float64)[:, None], hd[t, k], down.values(e)
        o, off = v @ w.T, np.maximum(2.0 ** -23 * np.abs(v), 2.0 ** -39) @ np.abs(w).T
        np.add.at(ref, t, r * o)
        np.add.at(tol, t, r * (off + down.tol(v, e) + 2.0 ** -22 * np.abs(o)))
    assert np.all(np.abs(y - ref) <= tol), float((np.abs(y - ref) / tol).max())

@pytest.mark.parametrize("scale,x", [(2.0 ** 110, 2.0 ** -120), (2.0 ** -121, 2.0 ** 111), (2.0 ** 120, 2.0 ** -125)])
@pytest.mark.parametrize("T", [1, 5, 16, 17, 33, 200])
def test_scales_and_tokens_at_opposite_ends(scale, x, T):
    """Outputs near 1 from factors whose partial products leave fp32's range, at every number of tokens."""
    say("opposite ends", scale, x, T)
    g = np.random.default_rng(T)
    p = Parts(mq.FMT_INT4Z_G64, 1, 40, 1024, seed=3)
    p.st = (torch.from_numpy(1 + g.random(p.st.shape)) * scale).to(torch.bfloat16)
    w = p.pack()
    xt, xd = bf16(g.standard_normal((T, 1024)) * x)
    ref = xd @ p.values().T
    assert np.abs(ref).max() < 1e5
    y = mq.linear_int4(w, xt, out_dtype=torch.float32).double().cpu().numpy()
    # x of subnormal size has its last bits at 2^-133 (bf16) already; sums as in tests/int4_ref.py
    assert np.all(np.abs(y - ref) <= p.tol(xd) + 2.0 ** -23 * np.abs(ref)), float((np.abs(y - ref) / (p.tol(xd) + 1e-30)).max())
