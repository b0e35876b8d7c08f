"""INT8 linears on the GPU against a plain 64-bit form: token quantisation bit for bit,
the product at one token to several tiles, ragged rows and columns, both output types,
bias, extreme codes, tokens of zeros and tokens that are not finite, strides between
experts, another stream, graph capture.

Tolerances. The int32 sum is exact, so with c = sum * xs * ws in fp32 the error is at
most one rounding of the sum and two of the products, 3 * 2^-24 |c|, and with a bias
2^-24 |c + b| more; bf16 outputs add 2^-8 |y| (half a step of eps 2^-7)."""
import sys

import numpy as np
import pytest
import torch

import bit_quantized_moe_dequant_amd as mq

pytestmark = pytest.mark.gpu


def say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


def quant_ref(x):
    """The fp32 rule with numpy's correctly rounded operations."""
    x = x.astype(np.float32)
    a = np.abs(x).max(axis=1)
    with np.errstate(invalid="ignore", divide="ignore"):
        s = (a / np.float32(127)).astype(np.float32)
        q = np.clip(np.rint((x / s[:, None]).astype(np.float32)), -127, 127)
    bad = ~np.isfinite(x).all(axis=1)
    s = np.where(bad, np.float32(np.nan), s)
    q = np.where((bad | (a == 0))[:, None], 0, q)
    return q.astype(np.int8), s


def tokens(T, K, seed, f32=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((T, K), generator=g, device="cuda") * torch.exp(torch.randn((T, 1), generator=g, device="cuda"))
    return x if f32 else x.to(torch.bfloat16)


def weight(rows, cols, seed, n=1, pad=0):
    """An INT8 weight of n experts (pad: extra bytes between them) and its host planes."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    stride, sstride = (rows * cols + 15) // 16 * 16 + pad, rows * 4 + pad
    data = torch.randint(-128, 128, (n, stride), generator=g, device="cuda", dtype=torch.int8)
    scales = torch.rand((n, sstride // 4), generator=g, device="cuda") + 0.5
    w = mq.Weight(mq.FMT_INT8, rows, cols, n, data.view(torch.uint8).reshape(-1), scales.view(torch.uint8).reshape(-1),
                  expert_stride=stride, scale_expert_stride=sstride)
    q = data.cpu().numpy()[:, :rows * cols].reshape(n, rows, cols).astype(np.float64)
    return w, q, scales.cpu().numpy()[:, :rows].astype(np.float64)


def check(y, q, s, wq, ws, bias, bf16):
    """y against q W^T s w (+ b) in 64 bits (q and W whole numbers: the product is exact)."""
    c = (q.astype(np.float64) @ wq.T) * s.astype(np.float64)[:, None] * ws[None, :]
    ref = c if bias is None else c + bias.astype(np.float64)
    tol = 3 * 2.0 ** -24 * np.abs(c) * 1.001 + 2.0 ** -24 * np.abs(ref) * 1.001
    if bf16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    y = y.double().cpu().numpy()
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(y), nan)
    assert np.all((np.abs(y - ref) <= tol)[~nan]), float(np.nanmax(np.abs(y - ref) - tol))


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,K", [(1, 16), (3, 4096), (7, 8208), (5, 1040), (300, 4112), (2, 65536)])
def test_quantize(T, K, f32):
    say("quantize", T, K, f32)
    x = tokens(T, K, T + K, f32)
    if T > 2:
        x[1] = 0
        x[2, K // 2] = float("inf")
    if T > 4:
        x[3, K - 1] = float("nan")
        x[4] = 0
        x[4, 0] = 1e-40 if f32 else torch.finfo(torch.bfloat16).tiny / 64  # a subnormal maximum
    q, s = mq.quantize_int8(x)
    rq, rs = quant_ref(x.float().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)


def test_quantize_every_scale_and_value():
    """bf16 values of all magnitudes under scales of all exponents: the codes are the fp32 rule's."""
    say("quantize all")
    v = torch.arange(0, 0x7F80, 7, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)  # finite, non-negative
    v = torch.cat([v, -v])[: 9344].reshape(-1)
    n = v.numel() // 16 * 16
    rows = torch.stack([v[:n] * f for f in (1.0, 0.37, 2.0 ** -60, 2.0 ** -120)])
    order = torch.argsort(rows[0].float().abs())
    x = rows[:, order].reshape(4 * (n // 16), 16).contiguous().cuda()  # sixteen neighbours to a row: every scale
    q, s = mq.quantize_int8(x)
    rq, rs = quant_ref(x.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)


def test_quantize_ties_and_borders():
    """Values on and next to half codes: the rule is the fp32 quotient's, rounded to even."""
    say("quantize ties")
    s = np.float32(2.0 ** -3)
    base = (np.arange(-126, 127) + 0.5).astype(np.float32) * s
    rows = [base, np.nextafter(base, np.float32(np.inf)), np.nextafter(base, np.float32(-np.inf))]
    for k in (3, 7, 100):  # scales that are not powers of two
        sc = np.float32(k) * np.float32(0.0123)
        rows.append((np.arange(-126, 127) + 0.5).astype(np.float32) * (sc / np.float32(127)))
    x = np.zeros((len(rows), 272), np.float32)
    for i, r in enumerate(rows):
        x[i, :253] = r
        x[i, 260] = 127 * s if i < 3 else np.float32((3, 7, 100)[i - 3]) * np.float32(0.0123)
    q, sc = mq.quantize_int8(torch.from_numpy(x).cuda())
    rq, rs = quant_ref(x)
    assert np.array_equal(sc.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)


SHAPES = [(1, 16, 16), (1, 4096, 4096), (2, 33, 80), (15, 100, 1040), (16, 2048, 4096), (17, 130, 208), (63, 255, 4112),
          (64, 512, 512), (65, 48, 96), (100, 5003, 4112), (128, 300, 2064), (129, 257, 144), (200, 1000, 4096),
          (257, 513, 1168), (511, 1025, 656), (700, 4096, 1024), (1500, 2300, 528)]


@pytest.mark.parametrize("T,rows,cols", SHAPES)
@pytest.mark.parametrize("bf16", [False, True])
def test_linear(T, rows, cols, bf16):
    say("linear", T, rows, cols, bf16)
    w, wq, ws = weight(rows, cols, rows + cols)
    x = tokens(T, cols, T)
    if T > 3:
        x[1] = 0
        x[3, 5] = float("inf")
    bias = torch.randn(rows, device="cuda") if (T + rows) % 2 else None
    b = None if bias is None else bias.cpu().numpy()
    dt = torch.bfloat16 if bf16 else torch.float32
    xq, xs = mq.quantize_int8(x)
    pad = torch.full((T + 2, rows), 7.0, dtype=dt, device="cuda")
    mq.linear_int8(w, xq, xs, bias=bias, y=pad[1:T + 1])
    q, s = quant_ref(x.float().cpu().numpy())
    check(pad[1:T + 1], q, s, wq[0], ws[0], b, bf16)
    assert bool((pad[0] == 7).all()) and bool((pad[-1] == 7).all())  # the rows around are left alone
    y = mq.linear_int8_dynamic(w, x, bias=bias, out_dtype=dt)
    assert torch.equal(y.nan_to_num(123.0), pad[1:T + 1].nan_to_num(123.0))


def test_extreme_codes_and_long_sums():
    """All codes -128 over 65536 columns: the sum 2^30 is exact in int32."""
    say("extremes")
    rows, K = 40, 65536
    for T in (3, 150):
        wq = torch.full((rows, K), -128, dtype=torch.int8, device="cuda")
        wq[1] = 127
        w = mq.Weight(mq.FMT_INT8, rows, K, 1, wq.view(torch.uint8).reshape(-1), torch.ones(rows, device="cuda").view(torch.uint8))
        xq = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
        y = mq.linear_int8(w, xq, torch.ones(T, device="cuda"), out_dtype=torch.float32)
        assert bool((y[:, 0] == 2.0 ** 30).all()) and bool((y[:, 1] == -128.0 * 127 * K).all())


def test_experts_with_strides():
    say("strides")
    w, wq, ws = weight(50, 272, 5, n=3, pad=48)
    x = tokens(20, 272, 3)
    q, s = quant_ref(x.float().cpu().numpy())
    for e in range(3):
        check(mq.linear_int8_dynamic(w, x, expert=e, out_dtype=torch.float32), q, s, wq[e], ws[e], None, False)
        d = mq.dequant(w, e).cpu().numpy()
        assert np.array_equal(d, (wq[e] * ws[e][:, None]).astype(np.float32))


def test_a_token_does_not_depend_on_its_batch():
    say("batch")
    w, _, _ = weight(700, 1040, 8)
    x = tokens(300, 1040, 9)
    y = mq.linear_int8_dynamic(w, x)
    for t0, t1 in ((0, 1), (5, 21), (30, 90), (100, 220)):
        assert torch.equal(mq.linear_int8_dynamic(w, x[t0:t1].contiguous()), y[t0:t1])


def test_streams_and_graph():
    """Another stream than the default one, and a captured call replayed on new inputs."""
    say("graph")
    w, wq, ws = weight(300, 528, 11)
    for T in (1, 40, 300):
        x = tokens(T, 528, T)
        y = torch.empty((T, 300), dtype=torch.float32, device="cuda")
        work = mq.linear_int8_workspace(T, 528)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            mq.linear_int8_dynamic(w, x, y=y, ws=work)
            with torch.cuda.graph(graph, stream=stream):
                mq.linear_int8_dynamic(w, x, y=y, ws=work)
        torch.cuda.synchronize()
        for rep in range(3):
            x.copy_(tokens(T, 528, 50 + rep))
            y.fill_(float("nan"))
            work.fill_(rep)
            eager = mq.linear_int8_dynamic(w, x, out_dtype=torch.float32)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, eager)
        q, s = quant_ref(x.float().cpu().numpy())
        check(y, q, s, wq[0], ws[0], None, False)
        del graph


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9, 13, 16])
@pytest.mark.parametrize("cols", [16, 48, 528, 1040, 2064, 4096, 7168, 8192, 16384])
def test_few_tokens_from_bf16(T, cols):
    """The one-launch form (T <= 16, and T as a power of two times cols <= 65536) and the two beyond it."""
    say("few", T, cols)
    w, wq, ws = weight(37, cols, cols)
    x = tokens(T, cols, T)
    x[T - 1, cols - 1] = 300.0  # the maximum in the row's last place
    if T > 2:
        x[1] = 0
        x[2, 3] = float("nan")
    q, s = quant_ref(x.float().cpu().numpy())
    y = mq.linear_int8_dynamic(w, x, out_dtype=torch.float32)
    check(y, q, s, wq[0], ws[0], None, False)
    two = mq.linear_int8(w, *mq.quantize_int8(x), out_dtype=torch.float32)
    assert torch.equal(y.nan_to_num(123.0), two.nan_to_num(123.0))


def test_no_tokens():
    w, _, _ = weight(20, 32, 1)
    x = torch.empty((0, 32), dtype=torch.bfloat16, device="cuda")
    assert mq.linear_int8_dynamic(w, x).shape == (0, 20)
    q, s = mq.quantize_int8(x)
    assert mq.linear_int8(w, q, s).shape == (0, 20)


@pytest.mark.parametrize("bf16", [False, True])
def test_more_tokens_than_one_launch(bf16):
    """Two launches of the product, the second a few tokens short of a tile."""
    say("launches", bf16)
    T, K, rows = (1 << 17) + 21, 32, 24
    x = tokens(T, K, 61)
    w, wq, ws = weight(rows, K, 62)
    bias = torch.randn(rows, device="cuda")
    dt = torch.bfloat16 if bf16 else torch.float32
    y = mq.linear_int8_dynamic(w, x, bias=bias, out_dtype=dt)
    q, s = quant_ref(x.float().cpu().numpy())
    check(y, q, s, wq[0], ws[0], bias.cpu().numpy(), bf16)
    y = mq.linear_int8_dynamic(w, x, out_dtype=dt)
    check(y, q, s, wq[0], ws[0], None, bf16)


@pytest.mark.parametrize("T,rows,cols", [(40, 72, 144), (300, 520, 144), (1100, 2056, 272), (2050, 4096, 144), (8187, 8192, 144)])
def test_bias_at_every_tile(T, rows, cols):
    """bf16 outputs with a bias are the fp32 outputs without one, plus it, rounded once more;
    the bits do not depend on the batch."""
    say("bias", T, rows, cols)
    x = tokens(T, cols, 71)
    w, _, _ = weight(rows, cols, 72)
    bias = 40.0 * torch.randn(rows, device="cuda")
    plain = mq.linear_int8_dynamic(w, x, out_dtype=torch.float32)
    with_bias = mq.linear_int8_dynamic(w, x, bias=bias, out_dtype=torch.float32)
    assert torch.equal(with_bias, plain + bias)
    y = mq.linear_int8_dynamic(w, x, bias=bias)
    assert torch.equal(y, (plain + bias).to(torch.bfloat16))
    assert torch.equal(mq.linear_int8_dynamic(w, x, bias=bias[:]), y)
    odd = torch.empty(rows + 1, device="cuda")[1:]  # not 16-byte aligned
    odd.copy_(bias)
    assert torch.equal(mq.linear_int8_dynamic(w, x, bias=odd), y)
    for t, n in ((0, 1), (3, 16), (T - 33, 33)):
        assert torch.equal(mq.linear_int8_dynamic(w, x[t:t + n], bias=bias), y[t:t + n])
