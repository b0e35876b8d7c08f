"""Routed INT4 experts tiled over each expert's tokens, every instance of the kernels: groups and zero
points, gate/up in tiles of 32 and of 64 pairs, down of 16 and of 32, chunks that end inside a tile,
and the special cases of the routing there. References and tolerances: tests/test_gpu_int4_moe.py.

A call is tiled where the pairs that share an expert with another, times 1.6 H I bytes, are 67.5 MB
or more; tiled() says so from the sizes, and every test asserts it."""
import numpy as np
import pytest
import torch

import bit_quantized_moe_dequant_amd as mq
from tests.int4_ref import FMTS, Parts, group_of
from tests.test_gpu_int4 import say
from tests.test_gpu_int4_moe import G32, G64, G128, Z32, Z64, Z128, Experts, check

pytestmark = pytest.mark.gpu


def tiled(ex, T):
    touched = ex.E * (1 - (1 - ex.K / ex.E) ** T)
    return T > 1 and (T * ex.K - touched) * 1.6 * ex.H * ex.I >= 15 * 4.5e6


@pytest.mark.parametrize("fmt", FMTS)
def test_every_format(fmt):
    """11 experts, 4 to a token. 29 tokens: 10.5 pairs to an expert (gate/up 32, down 32); 24: 8.7 (down 16);
    90 and 200: 33 and 73 (gate/up 64, chunks of 64 and what is left)."""
    odd = group_of(fmt)
    ex = Experts(1024 + odd, 768 + odd, 11, 4, fmt, fmt, seed=fmt, scale="fp16" if fmt % 2 else "bf16")
    for T in (24, 29, 90, 200):
        say("tiled", fmt, T)
        assert tiled(ex, T)
        check(ex, T, seed=T)


@pytest.mark.parametrize("fg,fd", [(G128, Z32), (Z64, G32), (G32, Z128)])
def test_other_formats_for_down(fg, fd):
    ex = Experts(1152, 896, 9, 3, fg, fd, seed=2)
    for T in (29, 40, 130):
        say("tiled mixed", fg, fd, T)
        assert tiled(ex, T)
        check(ex, T, seed=T)


@pytest.mark.parametrize("T", [40, 150])
def test_every_number_of_pairs_to_an_expert(T):
    """Expert 0 with n pairs, n around the ends of a token tile and of a chunk; one with none; ids out of range."""
    ex = Experts(1024, 640, 10, 4, G128, Z128, seed=T)
    assert tiled(ex, T)
    for n in (0, 1, 15, 16, 17, 31, 32, 33, 40) + (() if T == 40 else (47, 48, 49, 63, 64, 65, 80, 97, 113, 128, 129, 150)):
        say("tiled pairs", T, n)
        ids = 2 + np.stack([np.random.default_rng(100 * n + t).permutation(8)[:4] for t in range(T)]).astype(np.int32)
        ids[:n, 1] = 0
        ids[T - 1, 3], ids[0, 2] = 10, -3
        check(ex, T, seed=n, ids=ids)


@pytest.mark.parametrize("T", [40, 130])
def test_the_same_expert_for_all_and_twice(T):
    ex = Experts(1024, 768, 6, 3, G64, Z64, seed=9)
    assert tiled(ex, T)
    say("tiled uneven", T)
    check(ex, T, seed=1, ids=np.tile(np.array([[4, 0, 5]], np.int32), (T, 1)))
    ids = ex.routing(T, 8)[0]
    ids[:, 2] = ids[:, 0]
    check(ex, T, seed=2, ids=ids)
    check(ex, T, seed=3, ids=np.full((T, 3), 5, np.int32))
    x, r = torch.randn((T, ex.H), device="cuda").to(torch.bfloat16), torch.rand((T, 3), device="cuda")
    y = mq.expert_forward(ex.layer, x, torch.full((T, 3), 6, dtype=torch.int32, device="cuda"), r)  # nobody is routed
    assert bool((y == 0).all())


@pytest.mark.parametrize("T", [40, 140])
def test_experts_and_tokens_that_are_not_finite(T):
    """An expert of NaN that nobody chose leaves no trace, a token with an infinity is NaN alone."""
    ex = Experts(1024, 768, 8, 3, G128, G64, seed=4)
    assert tiled(ex, T)
    say("tiled not finite", T)
    for w in (ex.layer.gate, ex.layer.up, ex.layer.down):
        for e in (0, 7):  # the first, which an id out of range might be taken for, and the last
            w.expert_planes(e)[1][:] = 0xFF
    ids = 1 + np.stack([np.random.default_rng(t).permutation(6)[:3] for t in range(T)]).astype(np.int32)
    ids[0, 0], ids[3, 2] = 8, -1
    xt, ti, tr, y, _, _ = check(ex, T, seed=T, ids=ids)
    bad = xt.clone()
    bad[1, 9], bad[T - 1, 1000] = float("inf"), float("nan")
    got = mq.expert_forward(ex.layer, bad, ti, tr)
    rest = [t for t in range(T) if t not in (1, T - 1)]
    assert torch.equal(got[rest], y[rest]) and bool(got[1].isnan().all()) and bool(got[T - 1].isnan().all())
    assert bool(y.isfinite().all())


@pytest.mark.parametrize("T", [40, 130])
def test_stages_strides_and_noalloc(T):
    """gate_up and down by themselves, experts further apart than their bytes, the forward without a workspace."""
    ex = Experts(1024, 768, 7, 3, G64, Z128, seed=11)
    assert tiled(ex, T)
    say("tiled stages", T)
    xt, ti, tr, y, ref, tol = check(ex, T, seed=T)
    ws = ex.layer.workspace(T)
    mq.route(ex.layer, ti, ws=ws)
    h = mq.gate_up(ex.layer, xt, ti, ws=ws)
    assert torch.equal(mq.down(ex.layer, h, ti, tr, ws=ws), y)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert torch.equal(mq.expert_forward_noalloc(ex.layer, xt, ti, tr, dev_err=err), y) and int(err) == 0
    far = []
    for w in (ex.layer.gate, ex.layer.up, ex.layer.down):
        ds, ss = w.expert_stride + 48, w.scale_expert_stride + 32
        d, s = (torch.full((7 * n,), 0xAB, dtype=torch.uint8, device="cuda") for n in (ds, ss))
        for e in range(7):
            a, b = w.expert_planes(e)
            d[e * ds:e * ds + a.numel()] = a
            s[e * ss:e * ss + b.numel()] = b
        far.append(mq.Weight(w.fmt, w.rows, w.cols, 7, d, s, w.scale2, None, ds, ss))
    assert torch.equal(mq.expert_forward(mq.Layer(1024, 768, 7, 3, *far), xt, ti, tr), y)


@pytest.mark.parametrize("T", [40, 130])
def test_graph_replayed_with_other_inputs(T):
    ex = Experts(1024, 768, 8, 3, G128, G128, seed=41)
    assert tiled(ex, T)
    say("tiled graph", T)
    xt, ti, tr, y, _, _ = check(ex, T, seed=50)
    out, ws = torch.empty_like(y), ex.layer.workspace(T)
    mq.expert_forward(ex.layer, xt, ti, tr, y=out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mq.expert_forward(ex.layer, xt, ti, tr, y=out, ws=ws)
    for r in range(3):
        xt.copy_(torch.randn(xt.shape, device="cuda"))
        ti.copy_(torch.from_numpy(ex.routing(T, r)[0]))
        want = mq.expert_forward(ex.layer, xt, ti, tr).clone()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
