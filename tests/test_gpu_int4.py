"""INT4 weights with group scales on the GPU: the packed layout, dequantisation (bit for bit),
the linear over types, groups, lengths, odd sizes and values that are not finite, against fp64.
Tolerances: tests/int4_ref.py; bf16 outputs add half a step, 2^-8 |y|."""
import sys

import numpy as np
import pytest
import torch

import bit_quantized_moe_dequant_amd as mq
from tests.int4_ref import FMTS, Parts, bf16, packed_reference

pytestmark = pytest.mark.gpu


def say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,rows,cols", [(1, 16, 128), (2, 21, 384), (3, 5, 640)])
def test_packing_and_dequant(fmt, n, rows, cols):
    say("pack", fmt, n, rows, cols)
    p = Parts(fmt, n, rows, cols, seed=rows + fmt, scale="fp16" if fmt % 2 else "bf16", spread=2.0, zmax=255)
    w = p.pack()
    assert (w.fmt, w.rows, w.cols, w.n_experts) == (fmt, rows, cols, n)
    s2 = w.scale2.cpu().numpy()
    for e in range(n):
        big = np.abs(p.s[e]).max()
        assert 64 <= big / s2[e] < 128 and np.log2(s2[e]) == np.round(np.log2(s2[e]))
        data, side = packed_reference(p, e, int(np.log2(s2[e])))
        got = w.expert_planes(e)
        assert np.array_equal(got[0].cpu().numpy(), data)
        assert np.array_equal(got[1].cpu().numpy(), side)
        d = mq.dequant(w, e).cpu().numpy()
        assert np.array_equal(d, p.values(e).astype(np.float32)) and np.array_equal(d.astype(np.float64), p.values(e))


def test_packing_of_extreme_scales():
    """Zeros, infinities, NaN and subnormals among the scales; a tensor of zeros."""
    say("pack extremes")
    p = Parts(mq.FMT_INT4_G64, 3, 20, 256, seed=3, scale="fp16")
    st = p.st.clone()
    st[0] = 0
    st[1, 3, 1], st[1, 4, 2], st[1, 5, 0] = float("inf"), float("nan"), 2.0 ** -24
    st[2] = torch.randint(1, 900, st[2].shape).to(torch.int16).view(torch.float16)  # subnormal
    p.st = st
    w = p.pack()
    assert w.scale2[0].item() == 1.0
    assert bool((mq.dequant(w, 0) == 0).all())
    with np.errstate(invalid="ignore"):
        ref = p.values(1)
    got = mq.dequant(w, 1).cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    fine = np.isfinite(ref)
    # 2^-24 is below 2^-20 of the largest scale's range: rounded to 2^-31 of the largest, times |q - 8|
    step = 2.0 ** -31 * np.abs(p.s[1][np.isfinite(p.s[1])]).max() * 8
    assert np.all(np.abs(got - ref)[fine] <= step)
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)])
    assert np.array_equal(mq.dequant(w, 2).cpu().numpy().astype(np.float64), p.values(2))


def check(p, w, T, seed, out, bias, e=0, scale=1.0):
    g = np.random.default_rng(seed)
    x = g.standard_normal((T, p.cols)) * np.exp(0.5 * g.standard_normal((T, 1))) * scale
    x[:, g.integers(0, p.cols, 2)] *= 8
    xt, xd = bf16(x)
    b = torch.from_numpy(g.standard_normal(p.rows).astype(np.float32)).cuda() if bias else None
    pad = torch.full((T + 2, p.rows), 7.0, dtype=out, device="cuda")
    y = mq.linear_int4(w, xt, expert=e, bias=b, y=pad[1:T + 1])
    ref = xd @ p.values(e).T + (0 if b is None else b.double().cpu().numpy())
    half = 0 if T <= mq.INT4_FEW_T or out == torch.float32 else 1
    tol = p.tol(xd, e, half) + 2.0 ** -23 * np.abs(ref) + (2.0 ** -8 * np.abs(ref) * 1.01 if out == torch.bfloat16 else 0)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.all(err <= tol), float((err / tol).max())
    assert bool((pad[0] == 7).all()) and bool((pad[-1] == 7).all())
    assert torch.equal(mq.linear_int4(w, xt, expert=e, bias=b, out_dtype=out), y)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,cols", [(64, 256), (33, 384), (1, 128), (250, 1152)])
def test_linear(fmt, rows, cols):
    p = Parts(fmt, 2, rows, cols, seed=fmt * 7 + rows, scale="bf16" if rows % 2 else "fp16", spread=1.0)
    w = p.pack()
    for i, T in enumerate((1, 2, 4, 5, 8, 9, 16, 17, 31, 64, 100, 129)):
        say("linear", fmt, rows, cols, T)
        check(p, w, T, seed=i, out=torch.float32 if i % 2 else torch.bfloat16, bias=i % 3 == 0, e=i % 2)


@pytest.mark.parametrize("fmt", [mq.FMT_INT4_G32, mq.FMT_INT4Z_G32, mq.FMT_INT4_G64])
@pytest.mark.parametrize("cols", [32, 64, 96, 160, 4128, 8224])
def test_linear_columns_that_end_inside_a_tile(fmt, cols):
    if cols % (32 << (fmt == mq.FMT_INT4_G64)):
        pytest.skip("not a whole number of groups")
    p = Parts(fmt, 1, 50, cols, seed=cols)
    w = p.pack()
    for T in (1, 7, 16, 40, 200):
        say("linear", fmt, cols, T)
        check(p, w, T, seed=T, out=torch.float32, bias=False)


@pytest.mark.parametrize("cols", list(range(128, 1300, 128)))
def test_linear_steps_that_several_waves_share(cols):
    p = Parts(mq.FMT_INT4Z_G32 if cols % 256 else mq.FMT_INT4_G128, 1, 70, cols, seed=cols)
    w = p.pack()
    for T in (20, 32, 33, 70):
        say("linear shared", cols, T)
        check(p, w, T, seed=T, out=torch.float32, bias=T == 33)


@pytest.mark.parametrize("fmt", FMTS)
def test_linear_of_large_tiles(fmt):
    """Enough rows and tokens for the largest tiles, fp32 and bf16, odd in each size; all zero points."""
    for rows, cols, T in ((8190, 128, 833), (6001, 544 if (fmt - mq.FMT_INT4_G32) % 3 == 0 else 640, 1100)):
        p = Parts(fmt, 1, rows, cols, seed=rows + fmt, spread=0.5, zmax=255)
        w = p.pack()
        for out in (torch.float32, torch.bfloat16):
            say("linear large", fmt, rows, cols, T, out)
            check(p, w, T, seed=T, out=out, bias=True)


@pytest.mark.parametrize("fmt", FMTS[3:])
def test_linear_with_all_zero_points(fmt):
    p = Parts(fmt, 1, 90, 640, seed=fmt, scale="fp16", zmax=255)
    w = p.pack()
    for T in (1, 3, 6, 12, 30, 90, 300):
        say("linear zero points", fmt, T)
        check(p, w, T, seed=T, out=torch.float32, bias=False)


@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** 80])
def test_linear_of_very_small_and_large_tokens(scale):
    p = Parts(mq.FMT_INT4Z_G64, 1, 48, 512, seed=5)
    w = p.pack()
    for T in (1, 6, 50):
        say("linear scale", scale, T)
        check(p, w, T, seed=T, out=torch.float32, bias=False, scale=scale)


@pytest.mark.parametrize("T", [1, 3, 12, 40, 150])
def test_tokens_that_are_not_finite_and_zeros(T):
    """A token with an infinity or a NaN gives NaN, a token of zeros 0, nobody else's change."""
    say("linear not finite", T)
    p = Parts(mq.FMT_INT4_G128, 1, 70, 640, seed=T)
    w = p.pack()
    x = torch.randn((T + 2, 640), device="cuda").to(torch.bfloat16)
    x[T] = 0
    good = mq.linear_int4(w, x, out_dtype=torch.float32)
    assert bool((good[T] == 0).all())
    bad = x.clone()
    bad[0, 639], bad[T + 1, 3] = float("inf"), float("nan")
    y = mq.linear_int4(w, bad, out_dtype=torch.float32)
    assert bool(y[0].isnan().all()) and bool(y[T + 1].isnan().all())
    assert torch.equal(y[1:T + 1], good[1:T + 1])


def test_linear_no_tokens_and_offsets_into_one_buffer():
    say("linear views")
    p = Parts(mq.FMT_INT4_G64, 1, 40, 256, seed=1)
    w = p.pack()
    x = torch.randn((60, 256), device="cuda").to(torch.bfloat16)
    assert mq.linear_int4(w, x[:0]).shape == (0, 40)
    y = mq.linear_int4(w, x, out_dtype=torch.float32)
    for a, b in ((3, 9), (7, 8), (20, 57)):  # a view of the same buffer
        part = mq.linear_int4(w, x[a:b], out_dtype=torch.float32)
        assert bool(((part - y[a:b]).abs() <= 1e-4 * y.abs().max()).all())


def test_linear_in_graphs_and_streams():
    """Captured once and replayed with new inputs between eager calls; two streams at once."""
    p = Parts(mq.FMT_INT4_G128, 1, 96, 512, seed=2)
    w = p.pack()
    for T in (1, 16, 48, 130):
        say("linear graph", T)
        x = torch.randn((T, 512), device="cuda").to(torch.bfloat16)
        y = torch.empty((T, 96), device="cuda")
        ws = mq.linear_int4_workspace(T, 512)
        mq.linear_int4(w, x, y=y, ws=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mq.linear_int4(w, x, y=y, ws=ws)
        for i in range(4):
            x.copy_(torch.randn((T, 512), device="cuda"))
            want = mq.linear_int4(w, x, out_dtype=torch.float32)
            y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = []
        for i in range(8):
            s = streams[i % 2]
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(mq.linear_int4(w, x, out_dtype=torch.float32))
        torch.cuda.synchronize()
        assert all(torch.equal(g, want) for g in got)
