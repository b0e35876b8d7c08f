"""The router against a plain 64-bit form: ids equal, weights to fp32 rounding, for
every scoring rule, with and without bias, at one token to several hundred and odd
expert counts; exact ties, masked experts, NaN and infinities; graph capture.

Tolerances. The logits are fp64 sums of exact products, so ids have to be equal unless
two keys are within 1e-9 of each other (none of the seeded inputs has such a pair, which
is asserted). The weights are fp64 values rounded to fp32: 2^-24 relative, 2^-23 taken."""
import sys

import numpy as np
import pytest
import torch

import bit_quantized_moe_dequant_amd as mq

pytestmark = pytest.mark.gpu
SCORES = ["softmax", "sigmoid", "sqrtsoftplus"]


def say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


def scores_ref(z, kind):
    with np.errstate(all="ignore"):
        if kind == "softmax":
            e = np.exp(z - z.max(axis=1, keepdims=True))
            return e / e.sum(axis=1, keepdims=True)
        if kind == "sigmoid":
            return 1.0 / (1.0 + np.exp(-z))
        return np.sqrt(np.maximum(z, 0) + np.log1p(np.exp(-np.abs(z))))


def route_ref(x, w, K, kind, norm, scale, bias):
    with np.errstate(all="ignore"):
        s = scores_ref(x.astype(np.float64) @ w.astype(np.float64).T, kind)
    key = s if bias is None else s + bias.astype(np.float64)
    key = np.where(np.isnan(key), -np.inf, key)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :K]
    rw = np.take_along_axis(s, ids, 1)
    if norm:
        tot = rw.sum(axis=1, keepdims=True)
        rw = np.where(tot == 0, 0.0, rw / np.where(tot == 0, 1.0, tot))
    return ids, rw * scale, key


def make(T, H, E, seed, bias=True, spread=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    w = (spread * torch.randn((E, H), generator=g, device="cuda") / H ** 0.5).to(torch.bfloat16)
    b = 0.2 * torch.randn(E, generator=g, device="cuda") if bias else None
    return x, w, b


def host(t):
    return None if t is None else t.float().cpu().numpy()


def check(ids, rw, ref):
    rid, rrw, _ = ref
    assert np.array_equal(ids.cpu().numpy(), rid)
    got = rw.cpu().numpy().astype(np.float64)
    fine = np.isfinite(rrw)
    assert np.array_equal(got[~fine], rrw[~fine], equal_nan=True)  # infinities and NaNs as they are
    assert np.all(np.abs(got - rrw)[fine] <= 2.0 ** -23 * np.abs(rrw[fine]) + 1e-45)


CASES = [(1, 4096, 256, 6), (1, 8, 1, 1), (2, 24, 7, 7), (5, 1032, 180, 8), (8, 4096, 256, 6), (9, 512, 65, 3),
         (16, 2048, 1024, 16), (33, 4104, 300, 5), (64, 4096, 256, 6), (130, 768, 257, 4), (700, 1024, 100, 8),
         (2, 65536, 70, 2)]


@pytest.mark.parametrize("T,H,E,K", CASES)
@pytest.mark.parametrize("kind", SCORES)
def test_router(T, H, E, K, kind):
    say("router", T, H, E, K, kind)
    bias, norm = (T + E) % 2 == 0, (T + K) % 2 == 0
    x, w, b = make(T, H, E, T * 7 + E, bias)
    ids, rw = mq.router_topk(mq.Router(w, K, scoring=kind, normalize=norm, scale=2.5, bias=b), x)
    ref = route_ref(host(x), host(w), K, kind, norm, 2.5, host(b))
    top = -np.sort(-ref[2], axis=1)[:, :K + 1]
    assert E == 1 or np.abs(np.diff(top, axis=1)).min() > 1e-9  # no near ties among the inputs
    check(ids, rw, ref)


@pytest.mark.parametrize("kind", SCORES)
@pytest.mark.parametrize("T", [3, 200])
def test_near_ties_are_decided_in_64_bits(T, kind):
    """Experts whose logits differ by a few parts in 1e8: below what an fp32 sum resolves."""
    say("near ties", T, kind)
    x, w, _ = make(T, 2048, 64, 5)
    w[1::2] = w[0::2]
    w[1::2, 100] = (w[0::2, 100].float() + 2.0 ** -20).to(torch.bfloat16)  # most stay equal, some move by one step
    ids, rw = mq.router_topk(mq.Router(w, 8, scoring=kind, normalize=True), x)
    ref = route_ref(host(x), host(w), 8, kind, True, 1.0, None)
    key = -np.sort(-ref[2], axis=1)[:, :9]
    gap = np.abs(np.diff(key, axis=1))
    clear = ((gap == 0) | (gap > 1e-12)).all(axis=1)
    assert clear.any()
    assert np.array_equal(ids.cpu().numpy()[clear], ref[0][clear])


@pytest.mark.parametrize("T,H,E,K", [(65, 8, 5, 2), (100, 16, 3, 3), (66, 1032, 64, 1), (257, 2056, 513, 16), (90, 8200, 33, 6)])
@pytest.mark.parametrize("kind", SCORES)
def test_many_tokens_at_odd_sizes(T, H, E, K, kind):
    """Beyond the one-launch form: rows shorter than a step, parts of the hidden size that
    end inside one, rows longer than a lane's registers hold."""
    say("many", T, H, E, K, kind)
    x, w, b = make(T, H, E, T + H)
    for bias in (b, None):
        ids, rw = mq.router_topk(mq.Router(w, K, scoring=kind, bias=bias), x)
        ref = route_ref(host(x), host(w), K, kind, False, 1.0, host(bias))
        key = -np.sort(-ref[2], axis=1)[:, :K + 1]
        assert np.abs(np.diff(key, axis=1)).min() > 1e-12
        check(ids, rw, ref)


@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** 60, 2.0 ** 100])
@pytest.mark.parametrize("T", [4, 100])
def test_magnitudes_beyond_fp32(T, scale):
    """Logits whose products or sums leave fp32's range on either side: order by the fp64 logit."""
    say("magnitudes", T, scale)
    x, w, _ = make(T, 512, 40, 31)
    x, w = (x.float() * scale).to(torch.bfloat16), (w.float() * scale).to(torch.bfloat16)
    x[1] = 0
    ids, _ = mq.router_topk(mq.Router(w, 5, scoring="softmax"), x)
    z = x.double().cpu().numpy() @ w.double().cpu().numpy().T
    assert np.array_equal(ids.cpu().numpy(), np.argsort(-z, axis=1, kind="stable")[:, :5])


def wide(T, E, seed):
    """Numbers of one magnitude in fp64 from factors at both ends of bf16's range: x near
    2^126, w below 2^-126 (subnormal)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, 256), generator=g).sign() * 2.0 ** torch.randint(120, 127, (T, 256), generator=g)
    w = torch.randint(-127, 128, (E, 256), generator=g).double() * 2.0 ** -133
    return x.to(torch.bfloat16).cuda(), w.float().to(torch.bfloat16).cuda()


@pytest.mark.parametrize("T", [4, 100])
def test_weights_below_the_normal_range(T):
    say("subnormal", T)
    x, w = wide(T, 40, 12)
    assert bool((w != 0).any(dim=1).all()) and float(w.float().abs().max()) < 2.0 ** -126
    for kind in SCORES:
        ids, rw = mq.router_topk(mq.Router(w, 5, scoring=kind, normalize=True), x)
        ref = route_ref(host(x), host(w), 5, kind, True, 1.0, None)
        key = -np.sort(-ref[2], axis=1)[:, :6]
        clear = (np.abs(np.diff(key, axis=1)) > 1e-12 * np.abs(key[:, :1])).all(axis=1)
        assert clear.mean() > 0.5
        assert np.array_equal(ids.cpu().numpy()[clear], ref[0][clear])


@pytest.mark.parametrize("T", [4, 100])
def test_softmax_over_logits_whose_sums_overflow_on_the_way(T):
    """Exact logits of 0 and small numbers, of which some pass 2^128 in their partial sums:
    the experts that are not chosen must not spoil the denominator."""
    say("overflow on the way", T)
    g = torch.Generator().manual_seed(5)
    x = torch.zeros((T, 512))
    x[:, :256] = 2.0 ** 70
    x[:, 256:] = torch.randn((T, 256), generator=g) / 16
    w = torch.randn((40, 512), generator=g)
    w[:, :256] = 0
    for e in (3, 17, 31):             # + and - 2^140, in halves and in turn
        w[e] = 0
        w[e, :128], w[e, 128:256] = 2.0 ** 70, -2.0 ** 70
    w[22] = 0
    w[22, 0:256:2], w[22, 1:256:2] = 2.0 ** 70, -2.0 ** 70
    x, w = x.to(torch.bfloat16).cuda(), w.to(torch.bfloat16).cuda()
    for K in (1, 5):
        ids, rw = mq.router_topk(mq.Router(w, K, scoring="softmax"), x)
        ref = route_ref(host(x), host(w), K, "softmax", False, 1.0, None)
        assert np.isfinite(ref[1]).all() and np.array_equal(ids.cpu().numpy(), ref[0])
        # the other denominators' terms: fp32 sums of at most 40 numbers below 4
        assert np.all(np.abs(rw.cpu().numpy() - ref[1]) <= 2.0 ** -18 * ref[1])


@pytest.mark.parametrize("T", [64, 100])
def test_softmax_weights_beside_a_large_common_part(T):
    """An activation outlier adds the same large number to every logit. Up to 64 tokens the
    weights are fp64 throughout; beyond, logits that are not chosen enter the denominator
    with the error of fp32 sums, at most 2^-16 |W_e| |x|."""
    say("outlier", T)
    x, w, _ = make(T, 1024, 96, 44)
    x[:, 5], w[:, 5] = 512.0, 1.0
    ids, rw = mq.router_topk(mq.Router(w, 6, scoring="softmax"), x)
    X, W = host(x).astype(np.float64), host(w).astype(np.float64)
    ref = route_ref(host(x), host(w), 6, "softmax", False, 1.0, None)
    assert np.array_equal(ids.cpu().numpy(), ref[0])
    d = 0.0 if T <= 64 else 2.0 ** -16 * np.linalg.norm(X, axis=1)[:, None] * np.linalg.norm(W, axis=1).max()
    assert np.all(np.abs(rw.cpu().numpy() - ref[1]) <= (2.0 ** -23 + np.expm1(d)) * ref[1])
    ids2, rw2 = mq.router_topk(mq.Router(w, 6, scoring="softmax", normalize=True), x)
    check(ids2, rw2, route_ref(host(x), host(w), 6, "softmax", True, 1.0, None))  # no denominator: exact


def test_one_workspace_for_several_sizes():
    """A workspace for the most tokens serves fewer, one call after another."""
    x, w, b = make(300, 256, 60, 8)
    r = mq.Router(w, 4, scoring="sigmoid", bias=b)
    ws = r.workspace(300)
    for T in (300, 1, 64, 65, 9, 300):
        ids, rw = mq.router_topk(r, x[:T], ws=ws)
        check(ids, rw, route_ref(host(x[:T]), host(w), 4, "sigmoid", False, 1.0, host(b)))


def test_exact_ties_take_the_lowest_id():
    say("ties")
    for T in (1, 150):
        x, w, _ = make(T, 64, 128, 3)
        w[:] = w[0:1]
        ids, rw = mq.router_topk(mq.Router(w, 6, scoring="softmax"), x)
        assert bool((ids == torch.arange(6, device="cuda", dtype=torch.int32)).all())
        assert bool(((rw - 1 / 128).abs() < 2.0 ** -24).all())


@pytest.mark.parametrize("kind", SCORES)
def test_masks_and_values_that_are_not_finite(kind):
    say("masks", kind)
    E, K = 70, 6
    for T in (4, 160):
        x, w, b = make(T, 256, E, 9)
        low = torch.finfo(torch.float32).min
        b[:] = float("-inf")
        b[[3, 40, 66]] = 0.0          # three experts left; the rest by id
        b[50] = low                   # finite: before every -inf
        b[7] = float("nan")           # as -inf
        ids, rw = mq.router_topk(mq.Router(w, K, scoring=kind, normalize=True, bias=b), x)
        check(ids, rw, route_ref(host(x), host(w), K, kind, True, 1.0, host(b)))
        x[1] = float("nan")           # one token's logits are all NaN: ids by number, weights NaN
        x[2] = 0
        x[3, 5] = float("inf")        # logits of +-inf
        ids, rw = mq.router_topk(mq.Router(w, K, scoring=kind), x)
        assert ids[1].tolist() == list(range(K)) and bool(rw[1].isnan().all())
        assert ids[2].tolist() == list(range(K))
        i = ids.cpu().numpy()
        assert i.min() >= 0 and i.max() < E and all(len(set(r)) == K for r in i)
        ref = route_ref(host(x), host(w), K, kind, False, 1.0, None)
        if kind != "softmax":         # softmax of an infinite logit is NaN everywhere
            check(ids, rw, ref)


def test_weights_that_underflow():
    """All chosen scores 0 in fp64: weights 0, not NaN."""
    x = torch.full((2, 64), -200.0, device="cuda").to(torch.bfloat16)
    w = torch.ones((16, 64), device="cuda").to(torch.bfloat16)
    ids, rw = mq.router_topk(mq.Router(w, 4, scoring="sigmoid", normalize=True), x)
    assert bool((rw == 0).all()) and ids[0].tolist() == [0, 1, 2, 3]


def test_large_values_do_not_overflow():
    """Products beyond fp32's range stay finite in fp64."""
    x = torch.zeros((1, 64), device="cuda").to(torch.bfloat16)
    w = torch.zeros((8, 64), device="cuda").to(torch.bfloat16)
    x[0, 0], x[0, 1] = 1e30, 1.0
    w[:, 0] = 1e30
    w[5, 1] = 1.0
    w[2, 0], w[2, 1] = 2e30, 0.0
    ids, rw = mq.router_topk(mq.Router(w, 2, scoring="softmax"), x)
    assert ids[0].tolist()[0] == 2 and bool((rw[0] == torch.tensor([1.0, 0.0], device="cuda")).all())


def test_graph_and_streams():
    say("graph")
    for T in (1, 20, 300):
        x, w, b = make(T, 1024, 128, T)
        r = mq.Router(w, 6, scoring="sigmoid", normalize=True, bias=b)
        ids = torch.empty((T, 6), dtype=torch.int32, device="cuda")
        rw = torch.empty((T, 6), device="cuda")
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            mq.router_topk(r, x, ids=ids, rw=rw)
            with torch.cuda.graph(graph, stream=stream):
                mq.router_topk(r, x, ids=ids, rw=rw)
        torch.cuda.synchronize()
        for rep in range(4):
            x.copy_(make(T, 1024, 128, 90 + rep)[0])
            ids.fill_(-1)
            eager = mq.router_topk(r, x)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(ids, eager[0]) and torch.equal(rw, eager[1])
        check(ids, rw, route_ref(host(x), host(w), 6, "sigmoid", True, 1.0, host(b)))
        del graph


def test_no_tokens():
    _, w, _ = make(1, 64, 8, 1)
    ids, rw = mq.router_topk(mq.Router(w, 2), torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    assert ids.shape == (0, 2) == rw.shape
