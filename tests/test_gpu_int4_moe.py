"""Routed experts with INT4 weights, alone and beside other formats, and the whole layer with the
router's groups, INT4 experts and the INT8 shared expert, against fp64.

Tolerance of the experts: h is off by the gate's and up's (tests/int4_ref.py), at most
1.1 |u| dg + |g| du + 2^-20 |h| (silu's slope is below 1.1; its fast exponential), which the down
matrix carries on (2-norms: the errors' signs are independent), with h's own rounding to 16 bits
(2^-16) and the down product's error; 2^-22 of the parts for the route weights and the sum."""
import sys

import numpy as np
import pytest
import torch

import bit_quantized_moe_dequant_amd as mq
from tests.int4_ref import Parts, bf16
from tests.test_gpu_int4 import say

pytestmark = pytest.mark.gpu
G32, G64, G128, Z32, Z64, Z128 = range(mq.FMT_INT4_G32, mq.FMT_INT4Z_G128 + 1)


class Experts:
    def __init__(self, H, I, E, K, fg, fd, seed=1, scale="bf16"):
        self.H, self.I, self.E, self.K = H, I, E, K
        self.p = [Parts(fg, E, I, H, seed, scale), Parts(fg, E, I, H, seed + 1, scale), Parts(fd, E, H, I, seed + 2, scale)]
        self.layer = mq.Layer(H, I, E, K, *[p.pack() for p in self.p])
        self.w = {}

    def mat(self, i, e):
        if (i, e) not in self.w:
            self.w[i, e] = self.p[i].values(e)
        return self.w[i, e]

    def routing(self, T, seed):
        g = np.random.default_rng(seed)
        ids = np.stack([g.permutation(self.E)[:self.K] for _ in range(T)]).astype(np.int32)
        rw = (0.2 + g.random((T, self.K))).astype(np.float32)
        return ids, rw

    def reference(self, xd, ids, rw):
        """(y, its bound) over the valid ids."""
        T = xd.shape[0]
        y, tol = np.zeros((T, self.H)), np.zeros((T, self.H))
        for e in range(self.E):
            t, k = np.nonzero(ids == e)
            if t.size == 0:
                continue
            x = xd[t]
            g, u, r = x @ self.mat(0, e).T, x @ self.mat(1, e).T, rw[t, k].astype(np.float64)[:, None]
            h = g / (1 + np.exp(-g)) * u
            dh = 1.1 * np.abs(u) * self.p[0].tol(x, e) + np.abs(g) * self.p[1].tol(x, e) + 2.0 ** -16 * np.abs(h) * 1.1
            D = self.mat(2, e)
            o = h @ D.T
            np.add.at(y, t, r * o)
            np.add.at(tol, t, np.abs(r) * (4 * np.sqrt(dh ** 2 @ (D ** 2).T) + self.p[2].tol(h, e) + 2.0 ** -22 * np.abs(o)))
        return y, tol


def check(ex, T, seed, ids=None):
    g = np.random.default_rng(seed)
    xt, xd = bf16(g.standard_normal((T, ex.H)))
    i0, rw = ex.routing(T, seed)
    ids = i0 if ids is None else ids
    ti, tr = torch.from_numpy(ids).cuda(), torch.from_numpy(rw).cuda()
    y = mq.expert_forward(ex.layer, xt, ti, tr)
    ref, tol = ex.reference(xd, ids, rw)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.all(err <= tol + 1e-30), float((err / (tol + 1e-30)).max())
    assert torch.equal(mq.expert_forward(ex.layer, xt, ti, tr), y)
    return xt, ti, tr, y, ref, tol


SHAPES = [
    # H, I, E, K, gate/up, down, scales
    (256, 128, 8, 2, G128, G128, "bf16"),
    (512, 320, 12, 4, G64, G64, "fp16"),
    (288, 96, 5, 3, G32, G32, "bf16"),
    (384, 160, 9, 6, Z128, Z32, "fp16"),
    (128, 64, 3, 1, Z32, Z64, "bf16"),
    (1024, 512, 16, 8, G32, G128, "bf16"),
]


@pytest.mark.parametrize("shape", SHAPES)
def test_experts(shape):
    H, I, E, K, fg, fd, scale = shape
    ex = Experts(H, I, E, K, fg, fd, seed=H + I, scale=scale)
    for T in (1, 2, 4, 5, 9, 17, 40, 130, 300):
        say("experts", shape, T)
        check(ex, T, seed=T)


def test_uneven_routing_and_ids_out_of_range():
    """All tokens to the same experts, one expert without a token, ids outside the range."""
    ex = Experts(256, 192, 7, 3, G64, Z64, seed=9)
    for T in (1, 3, 6, 33, 200):
        say("experts uneven", T)
        ids = np.tile(np.array([[4, 0, 6]], np.int32), (T, 1))
        check(ex, T, seed=T, ids=ids)
        ids = ex.routing(T, 5)[0]
        ids[0, 1], ids[T - 1, 0] = 7, -1
        ws = ex.layer.workspace(T)
        xt, ti, tr, y, ref, tol = check(ex, T, seed=T + 1, ids=ids)
        assert mq.check_device_error(ws) & mq.DEVERR_EXPERT_ID
        ti[0, 1], ti[T - 1, 0] = 0, 0
        mq.expert_forward(ex.layer, xt, ti, tr)
        assert mq.check_device_error(ws) == 0
        ids[:] = 7  # nobody is routed
        z = mq.expert_forward(ex.layer, xt, torch.from_numpy(ids).cuda(), tr)
        assert bool((z == 0).all())
        mq.check_device_error(ws)


def test_an_expert_that_nobody_chose_may_hold_nan():
    ex = Experts(256, 128, 6, 2, G128, G128, seed=4)
    for w in (ex.layer.gate, ex.layer.up, ex.layer.down):
        for e in (0, 5):  # the first: what an id out of range is clamped to
            w.expert_planes(e)[1][:] = 0xFF
    for T in (1, 4, 20, 140):
        say("experts nan", T)
        ids = 1 + np.stack([np.random.default_rng(t).permutation(4)[:2] for t in range(T)]).astype(np.int32)
        ids[0, 0] = 9
        check(ex, T, seed=T, ids=ids)


def test_tokens_that_are_not_finite_stay_alone():
    ex = Experts(256, 128, 6, 2, G128, G64, seed=6)
    for T in (2, 8, 50, 150):
        say("experts not finite", T)
        xt, ti, tr, y, _, _ = check(ex, T, seed=T)
        bad = xt.clone()
        bad[1, 9] = float("inf")
        got = mq.expert_forward(ex.layer, bad, ti, tr)
        rest = [t for t in range(T) if t != 1]
        assert torch.equal(got[rest], y[rest]) and bool(got[1].isnan().all())


@pytest.mark.parametrize("T", [1, 3, 12, 140])
def test_stages_and_noalloc(T):
    """gate_up and down by themselves, with the fp32 h between them; the forward without a workspace."""
    say("experts stages", T)
    ex = Experts(384, 256, 8, 3, G64, Z128, seed=11)
    xt, ti, tr, y, ref, tol = check(ex, T, seed=T)
    ws = ex.layer.workspace(T)
    if T > 1:
        mq.route(ex.layer, ti, ws=ws)
    h = mq.gate_up(ex.layer, xt, ti, ws=ws)
    xd = xt.double().cpu().numpy()
    for t in (0, T - 1):
        for k in range(3):
            e = int(ti[t, k])
            g, u = xd[t] @ ex.mat(0, e).T, xd[t] @ ex.mat(1, e).T
            hr = g / (1 + np.exp(-g)) * u
            dh = 1.1 * np.abs(u) * ex.p[0].tol(xd[t:t + 1], e)[0] + np.abs(g) * ex.p[1].tol(xd[t:t + 1], e)[0] + 2.0 ** -20 * np.abs(hr)
            assert np.all(np.abs(h[t, k].double().cpu().numpy() - hr) <= dh)
    y2 = mq.down(ex.layer, h, ti, tr, ws=ws)
    assert np.all(np.abs(y2.double().cpu().numpy() - ref) <= tol)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert torch.equal(mq.expert_forward_noalloc(ex.layer, xt, ti, tr, dev_err=err), y) and int(err) == 0


@pytest.mark.parametrize("shape", [(256, 2944, 7, 6), (128, 5888, 4, 3)])
def test_pairs_whose_h_is_too_long_for_one_work_group(shape):
    """A few tokens with gate/up pair by pair and down by expert, the stages of one token without route."""
    H, I, E, K = shape
    ex = Experts(H, I, E, K, Z64, G64, seed=21)
    for T in (1, 2, 5):
        say("experts long", shape, T)
        xt, ti, tr, y, ref, tol = check(ex, T, seed=T)
        if T == 1:
            ws = ex.layer.workspace(1)
            h = mq.gate_up(ex.layer, xt, ti, ws=ws)
            got = mq.down(ex.layer, h, ti, tr, ws=ws)
            assert np.all(np.abs(got.double().cpu().numpy() - ref) <= tol)


@pytest.mark.parametrize("T", [1, 3, 30, 200])
def test_the_same_expert_twice(T):
    say("experts twice", T)
    ex = Experts(256, 192, 6, 3, G128, Z64, seed=31)
    ids = ex.routing(T, 8)[0]
    ids[:, 2] = ids[:, 0]
    check(ex, T, seed=T, ids=ids)
    ids[:] = 5
    check(ex, T, seed=T, ids=ids)


@pytest.mark.parametrize("T", [1, 6, 45, 330])
def test_graphs_and_streams(T):
    """Two captured graphs on workspaces of their own, replayed in turn with other inputs beside eager calls
    on another stream."""
    say("experts graph", T)
    ex = Experts(384, 192, 8, 3, G64, G64, seed=41)
    calls = []
    for i in range(2):
        xt, ti, tr, y, _, _ = check(ex, T, seed=50 + i)
        out, ws = torch.empty_like(y), torch.zeros(mq.workspace_bytes(ex.layer, T) + 256, dtype=torch.uint8, device="cuda")
        ws = ws[-ws.data_ptr() % 256:]
        mq.expert_forward(ex.layer, xt, ti, tr, y=out, ws=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mq.expert_forward(ex.layer, xt, ti, tr, y=out, ws=ws)
        calls.append((graph, xt, ti, tr, out, ws))  # the graph's workspace lives as long as it
    side = torch.cuda.Stream()
    for r in range(3):
        want = []
        for i, (_, xt, ti, tr, out, _) in enumerate(calls):
            g = torch.Generator(device="cuda")
            g.manual_seed(100 * r + i)
            xt.copy_(torch.randn(xt.shape, generator=g, device="cuda"))
            ti.copy_(torch.from_numpy(ex.routing(T, 7 * r + i)[0]))
            out.zero_()
            want.append(mq.expert_forward(ex.layer, xt, ti, tr).clone())
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            other = mq.expert_forward(ex.layer, calls[0][1], calls[0][2], calls[0][3])
        for graph, *_ in calls:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(other, want[0])
        for call, w in zip(calls, want):
            assert torch.equal(call[4], w)


@pytest.mark.parametrize("T", [1, 6, 30, 150])
@pytest.mark.parametrize("int4_down", [True, False])
def test_beside_another_format(T, int4_down):
    """INT4 in one projection and MXFP4 in the other, against the same layer's own values (the MXFP4
    projection's by mq.dequant). MXFP4 takes 8-bit activations from 128 tokens on: 4 % of the RMS."""
    say("experts mixed", T, int4_down)
    H, I, E, K = 512, 512, 6, 2
    g = torch.Generator(device="cuda").manual_seed(T)

    def mx(rows, cols):
        w = mq.Weight.empty(mq.FMT_MXFP4, rows, cols, E)
        w.data.copy_(torch.randint(0, 256, w.data.shape, generator=g, device="cuda", dtype=torch.uint8))
        w.scales.copy_(torch.randint(120, 123, w.scales.shape, generator=g, device="cuda", dtype=torch.uint8))
        return w

    i4 = [Parts(G64, E, *s, 30 + i).pack() for i, s in enumerate([(I, H), (I, H), (H, I)])]
    ws = [mx(I, H), mx(I, H), i4[2]] if int4_down else [i4[0], i4[1], mx(H, I)]
    layer = mq.Layer(H, I, E, K, *ws)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:K] for _ in range(T)]).to(torch.int32)
    rw = torch.rand((T, K), generator=g, device="cuda")
    y = mq.expert_forward(layer, x, ids, rw).double()
    ref = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        G, U, D = (mq.dequant(w, e).double() for w in ws)
        t, k = (ids == e).nonzero(as_tuple=True)
        a, b = x[t].double() @ G.t(), x[t].double() @ U.t()
        ref.index_add_(0, t, rw[t, k].double()[:, None] * ((a * torch.sigmoid(a) * b) @ D.t()))
    rms = ref.pow(2).mean().sqrt()
    err = (y - ref).pow(2).mean().sqrt() / rms
    assert float(err) < (2e-3 if T < 128 else 0.06), float(err)


def test_weights_in_strided_buffers():
    """Experts further apart than their bytes."""
    say("experts strided")
    ex = Experts(256, 128, 5, 2, Z64, G32, seed=21)
    xt, ti, tr, y, _, _ = check(ex, 6, seed=1)
    far = []
    for w in (ex.layer.gate, ex.layer.up, ex.layer.down):
        ds, ss = w.expert_stride + 48, w.scale_expert_stride + 32
        d, s = (torch.full((5 * n,), 0xAB, dtype=torch.uint8, device="cuda") for n in (ds, ss))
        for e in range(5):
            a, b = w.expert_planes(e)
            d[e * ds:e * ds + a.numel()] = a
            s[e * ss:e * ss + b.numel()] = b
        far.append(mq.Weight(w.fmt, w.rows, w.cols, 5, d, s, w.scale2, None, ds, ss))
    layer = mq.Layer(256, 128, 5, 2, *far)
    assert torch.equal(mq.expert_forward(layer, xt, ti, tr), y)


@pytest.mark.parametrize("T,shared", [(1, 256), (1, 0), (4, 64), (7, 256), (20, 128), (140, 256)])
@pytest.mark.parametrize("kind,by", [("sigmoid", "top2"), ("softmax", "max")])
def test_whole_layer_with_groups(T, shared, kind, by):
    """Router with groups, INT4 experts and the INT8 shared expert in one call, against its parts:
    the router's own entry point (exact), the experts' fp64 values, the shared expert by its own
    linears (their sums are exact; h's code may be the neighbour: one code of h for every 1e-3
    of them that may lie next to a half, five times over), one rounding to bf16."""
    from tests.test_gpu_int8 import quant_ref
    from tests.test_gpu_moe import int8_weight
    say("moe int4", T, shared, kind, by)
    H, I, E, K = 512, 256, 24, 4
    ex = Experts(H, I, E, K, G64, Z128, seed=T)
    g = torch.Generator(device="cuda").manual_seed(T)
    w = (torch.randn((E, H), generator=g, device="cuda") / H ** 0.5).to(torch.bfloat16)
    router = mq.Router(w, K, scoring=kind, normalize=True, scale=2.5, n_groups=6, top_groups=2, group_score=by)
    sh = [int8_weight(shared, H, g), int8_weight(shared, H, g), int8_weight(H, shared, g)] if shared else None
    moe = mq.MoeLayer(ex.layer, router, mq.SharedExpert(*[s[0] for s in sh]) if shared else None)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    y, ids, rw = mq.moe_forward(moe, x)
    rid, rrw = mq.router_topk(router, x)
    assert torch.equal(rid, ids) and torch.equal(rrw, rw)
    assert bool(((ids // 4).sort(dim=1)[0].diff(dim=1) != 0).sum(dim=1).max() < 2)  # two groups at most
    xd = x.double().cpu().numpy()
    ref, tol = ex.reference(xd, ids.cpu().numpy(), rw.cpu().numpy())
    if shared:
        (gq, gs), (uq, us), (dq, ds) = [s[1] for s in sh]
        q, s = (a.astype(np.float64) for a in quant_ref(x.float().cpu().numpy()))
        gate, up = (q @ gq.T) * s[:, None] * gs, (q @ uq.T) * s[:, None] * us
        h = (gate / (1 + np.exp(-gate)) * up).astype(np.float32)
        hq, hs = quant_ref(h)
        frac = np.abs(h / hs[:, None] - np.floor(h / hs[:, None]) - 0.5)
        flips = (frac < 1e-3).sum(axis=1)[:, None] * hs[:, None] * 127.0 * ds
        ref = ref + (hq.astype(np.float64) @ dq.T) * hs.astype(np.float64)[:, None] * ds
        tol = tol + flips + 2.0 ** -20 * (np.abs(hq.astype(np.float64)) @ np.abs(dq).T) * hs[:, None] * ds
    tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.all(err <= tol), float((err / tol).max())
    # replayed from a graph, with eager calls of other tokens between
    out, ws = torch.empty_like(y), moe.workspace(T)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mq.moe_forward(moe, x, y=out, ws=ws)
    for i in range(3):
        x.copy_(torch.randn((T, H), generator=g, device="cuda"))
        want = mq.moe_forward(moe, x)[0]
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_a_prompt_through_the_whole_layer_with_groups():
    """1100 tokens x 4096 x 240 experts in 8 groups: the ids are the router's own, the sum the experts' for them."""
    say("moe int4 prompt")
    T, H, I, E, K = 1100, 4096, 64, 240, 3
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def int4(rows, cols):
        codes = torch.randint(0, 256, (E, rows, cols // 2), generator=g, device="cuda", dtype=torch.uint8)
        s = (0.5 + torch.rand((E, rows, cols // 64), generator=g, device="cuda")) / (4 * cols ** 0.5)
        return mq.pack_int4(codes, s.to(torch.bfloat16))

    layer = mq.Layer(H, I, E, K, int4(I, H), int4(I, H), int4(H, I))
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn((E, H), generator=g, device="cuda") / 64).to(torch.bfloat16)
    r = mq.Router(w, K, scoring="sigmoid", normalize=True, n_groups=8, top_groups=3)
    y, ids, rw = mq.moe_forward(mq.MoeLayer(layer, r), x)
    ids2, rw2 = mq.router_topk(r, x)
    assert torch.equal(ids, ids2) and torch.equal(rw, rw2)
    want = mq.expert_forward(layer, x, ids, rw)
    # one rounding of the same sum to bf16, 2^-8, and 2^-20 of the row for sums in another order
    assert bool(((y.float() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * want.abs().amax(dim=1, keepdim=True)).all())
