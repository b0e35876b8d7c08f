"""The whole layer (router, routed experts, INT8 shared expert, bf16 sum) against the
64-bit oracle, over formats, token counts, with and without a shared expert; the routing
it returns against the router's own entry point; graph capture, streams, repeats.

Tolerance of y: half a bf16 step of the result (2^-8 |y|); the routed part within the
library's projection tolerance (2e-3, floored at the RMS); for the shared part, whose
sums are exact, fp32 rounding (2^-20 of its largest term) and one code of h for every
h that lies within 1e-3 of a rounding border (its fp32 value may fall on either side)."""
import sys

import numpy as np
import pytest
import torch

import bit_quantized_moe_dequant_amd as mq
from bit_quantized_moe_dequant_amd import synth, workloads
from oracle import moe
from tests.helpers import TOL, oracle_weight_fn
from tests.test_gpu_int8 import quant_ref
from tests.test_gpu_router import host, route_ref

pytestmark = pytest.mark.gpu
MX, NV, Q2, IQ = mq.FMT_MXFP4, mq.FMT_NVFP4, mq.FMT_Q2_K, mq.FMT_IQ2_XXS


def say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def int8_weight(rows, cols, g):
    q = (torch.randn((rows, cols), generator=g, device="cuda") * 32).round().clamp(-127, 127).to(torch.int8)
    s = (0.5 + torch.rand(rows, generator=g, device="cuda")) / (32 * cols ** 0.5)
    w = mq.Weight(mq.FMT_INT8, rows, cols, 1, q.view(torch.uint8).reshape(-1), s.view(torch.uint8))
    return w, (q.double().cpu().numpy(), s.double().cpu().numpy())


class Case:
    def __init__(self, H, I, E, K, fg, fd, shared, kind="sqrtsoftplus", norm=True, bias=True, seed=1):
        self.spec = workloads.LayerSpec(H, I, E, K, fg, fd, seed=8100 + seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.H, self.K, self.kind, self.norm, self.g = H, K, kind, norm, g
        self.rw = (torch.randn((E, H), generator=g, device="cuda") / H ** 0.5).to(torch.bfloat16)
        self.rb = 0.1 * torch.randn(E, generator=g, device="cuda") if bias else None
        self.router = mq.Router(self.rw, K, scoring=kind, normalize=norm, scale=1.5, bias=self.rb)
        self.sh = None
        if shared:
            ws = [int8_weight(shared, H, g), int8_weight(shared, H, g), int8_weight(H, shared, g)]
            self.sh, shared_mod = [w[1] for w in ws], mq.SharedExpert(*[w[0] for w in ws])
        self.layer = workloads.build_layer(mq, self.spec)
        self.moe = mq.MoeLayer(self.layer, self.router, shared_mod if shared else None)
        self.wfn = oracle_weight_fn(self.spec)

    def x(self, T, seed):
        bits = synth.activations_bf16(seed, T, self.H)
        return bits, cuda(bits.view(np.int16)).view(torch.bfloat16)

    def check(self, bits, xt, y, ids, rw, rows=None):
        ref_ids, ref_rw, _ = route_ref(host(xt), host(self.rw), self.K, self.kind, self.norm, 1.5, host(self.rb))
        assert np.array_equal(ids.cpu().numpy(), ref_ids)
        assert np.allclose(rw.cpu().numpy(), ref_rw, rtol=2.0 ** -23, atol=0)
        rows = list(range(xt.shape[0])) if rows is None else rows
        if xt.shape[0] < 128:
            routed, _ = moe.moe_layer(bits[rows], ref_ids[rows], ref_rw[rows].astype(np.float32), self.wfn)
        else:  # MXFP8 activations from 128 tokens: that path has tests of its own, its value is taken
            routed = mq.expert_forward(self.layer, xt, ids, rw).double().cpu().numpy()[rows]
        rms = np.sqrt(np.mean(routed ** 2))
        tol = TOL * np.maximum(np.abs(routed), rms)
        ref = routed.copy()
        if self.sh:
            (gq, gs), (uq, us), (dq, ds) = self.sh
            q, s = quant_ref(host(xt)[rows])
            q, s = q.astype(np.float64), s.astype(np.float64)
            gate, up = (q @ gq.T) * s[:, None] * gs, (q @ uq.T) * s[:, None] * us
            h = (gate / (1 + np.exp(-gate)) * up).astype(np.float32)
            hq, hs = quant_ref(h)
            sh = (hq.astype(np.float64) @ dq.T) * hs.astype(np.float64)[:, None] * ds
            frac = np.abs(h / hs[:, None] - np.floor(h / hs[:, None]) - 0.5)
            flips = (frac < 1e-3).sum(axis=1)[:, None] * hs[:, None] * 127.0 * ds
            ref = ref + sh
            tol = tol + flips + 2.0 ** -20 * (np.abs(hq.astype(np.float64)) @ np.abs(dq).T) * hs[:, None] * ds
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        got = y.double().cpu().numpy()[rows]
        assert np.isfinite(got).all()
        assert np.all(np.abs(got - ref) <= tol), float((np.abs(got - ref) / tol).max())


SHAPES = [
    # H, I, E, K, gate/up, down, shared, T
    (1024, 512, 16, 6, MX, MX, 512, 1),
    (1024, 512, 16, 6, MX, MX, 0, 1),
    (1024, 512, 16, 6, MX, MX, 528, 2),
    (512, 512, 9, 3, MX, MX, 16, 5),
    (1024, 512, 16, 8, MX, MX, 272, 8),
    (1024, 512, 16, 6, MX, MX, 512, 9),
    (1024, 512, 16, 6, MX, MX, 512, 16),
    (1024, 1024, 20, 1, NV, Q2, 512, 1),
    (1024, 512, 16, 6, NV, Q2, 512, 3),
    (1024, 512, 16, 6, NV, MX, 512, 1),
    (1024, 512, 16, 6, NV, Q2, 80, 17),
    (512, 256, 8, 2, IQ, Q2, 256, 1),
    (512, 256, 8, 2, IQ, Q2, 256, 12),
    (512, 256, 8, 2, IQ, MX, 256, 40),
    (512, 256, 8, 2, MX, MX, 256, 200),
    (288, 96, 5, 2, MX, MX, 48, 1),       # off the matrix-instruction kernels
    (288, 96, 5, 2, MX, MX, 48, 7),
]


@pytest.mark.parametrize("shape", SHAPES)
def test_layer(shape):
    H, I, E, K, fg, fd, shared, T = shape
    say("moe", shape)
    c = Case(H, I, E, K, fg, fd, shared, kind=["softmax", "sigmoid", "sqrtsoftplus"][T % 3], norm=T % 2 == 1,
             bias=(T + H // 32) % 2 == 1, seed=T)
    bits, xt = c.x(T, 70 + T)
    pad = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device="cuda")
    y, ids, rw = mq.moe_forward(c.moe, xt, y=pad[1:T + 1])
    c.check(bits, xt, y, ids, rw, rows=None if T <= 20 else [0, 1, T // 2, T - 1])
    assert bool((pad[0] == 7).all()) and bool((pad[-1] == 7).all())
    again = mq.moe_forward(c.moe, xt)
    rid, rrw = mq.router_topk(c.router, xt)
    assert torch.equal(again[0], y) and torch.equal(rid, ids) and torch.equal(rrw, rw)
    assert mq.check_device_error(c.moe.workspace(T)) == 0


def test_wide_hidden_size():
    """A hidden size whose tokens' codes do not fit the first launch, off the FP4 kernels."""
    say("moe wide")
    for T in (1, 12):
        c = Case(8192, 256, 6, 2, MX, MX, 64, seed=90 + T)
        bits, xt = c.x(T, 91)
        c.check(bits, xt, *mq.moe_forward(c.moe, xt))


def test_a_token_that_is_not_finite_stays_alone():
    say("moe nan")
    c = Case(1024, 512, 16, 6, MX, MX, 512, seed=93)
    for T in (4, 16):
        _, xt = c.x(T, 94)
        good = mq.moe_forward(c.moe, xt)
        bad = xt.clone()
        bad[2, 7] = float("nan")
        y, ids, rw = mq.moe_forward(c.moe, bad)
        rest = [t for t in range(T) if t != 2]
        for a, b in zip((y, ids, rw), good):
            assert torch.equal(a[rest], b[rest])
        assert bool(y[2].isnan().all()) and ids[2].tolist() == list(range(6))


def test_c_entry_without_routing_outputs_and_an_initialised_workspace():
    """ids and rw may be NULL; the workspace only needs moeq_workspace_init."""
    say("moe null outputs")
    c = Case(512, 512, 12, 4, MX, MX, 256, seed=95)
    lib = mq._lib()
    for T in (1, 8, 20):
        _, xt = c.x(T, 96 + T)
        ref = mq.moe_forward(c.moe, xt)[0]
        n = lib.moeq_moe_workspace_bytes(*c.moe._refs, T)
        raw = torch.randint(0, 256, (n + 512,), dtype=torch.uint8, device="cuda")
        off = (-raw.data_ptr()) % 256
        ws = raw[off:off + n]
        tail = raw[off + n:].clone()
        stream = torch.cuda.current_stream().cuda_stream
        assert lib.moeq_workspace_init(ws.data_ptr(), n, stream) == 0
        y = torch.empty_like(ref)
        for _ in range(2):
            assert lib.moeq_moe_forward(*c.moe._refs, xt.data_ptr(), T, y.data_ptr(), None, None, ws.data_ptr(), n, stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(y, ref) and torch.equal(raw[off + n:], tail)


def test_full_size():
    for T in (1, 3):
        say("moe full size", T)
        c = Case(4096, 2048, 256, 6, MX, MX, 2048, seed=40 + T)
        bits, xt = c.x(T, 5)
        c.check(bits, xt, *mq.moe_forward(c.moe, xt))
        del c
        torch.cuda.empty_cache()


def test_tokens_after_another_and_streams():
    """One token after another through one workspace, then two streams side by side."""
    c = Case(1024, 512, 16, 6, MX, MX, 512, seed=3)
    say("moe streams")
    xs = [c.x(T, 200 + i)[1] for i, T in enumerate((1, 1, 4, 1, 16, 2))]
    alone = [mq.moe_forward(c.moe, x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for rep in range(5):
        for i, x in enumerate(xs):
            s = streams[(i + rep) % 2]
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append((i, mq.moe_forward(c.moe, x)))
    torch.cuda.synchronize()
    for i, r in got:
        for a, b in zip(r, alone[i]):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("fg,fd,T", [(MX, MX, 1), (MX, MX, 6), (NV, Q2, 2), (MX, MX, 20), (MX, MX, 160)])
def test_graph(fg, fd, T):
    """Two graphs of the same layer, replayed in turn with eager calls between."""
    say("moe graph", fg, fd, T)
    c = Case(512, 512, 12, 4, fg, fd, 256, seed=T)
    x = [c.x(T, 300)[1], c.x(T, 301)[1]]
    out = [torch.empty((T, 512), dtype=torch.bfloat16, device="cuda") for _ in x]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(stream):
        for i in range(2):
            mq.moe_forward(c.moe, x[i], y=out[i])
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                mq.moe_forward(c.moe, x[i], y=out[i])
            graphs.append(graph)
    torch.cuda.synchronize()
    for rep in range(4):
        for i in range(2):
            x[i].copy_(c.x(T, 310 + 2 * rep + i)[1])
            out[i].fill_(float("nan"))
        eager = [mq.moe_forward(c.moe, v)[0] for v in x]
        torch.cuda.synchronize()
        for i in (0, 1):
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(out[i], eager[i]), (rep, i)
    del graphs


@pytest.mark.parametrize("T,shared", [(24, 272), (40, 272), (300, 2064), (1100, 2064), (2060, 2064)])
def test_shared_expert_of_many_tokens(T, shared):
    """Every tile of the shared expert's products, with channels and tokens past its end; the
    shared part alone is the same for a token on its own."""
    say("moe many", T, shared)
    c = Case(256, 256, 12, 4, MX, MX, shared, seed=90)
    bits, xt = c.x(T, 600)
    y, ids, rw = mq.moe_forward(c.moe, xt)
    c.check(bits, xt, y, ids, rw)
    routed = mq.expert_forward(c.layer, xt, ids, rw)
    assert bool(routed.isfinite().all())
    # the routed experts' scales to 2^-127: nothing beside the shared part, which has the same
    # bits in every form
    c.layer.down.scales.zero_()
    y = mq.moe_forward(c.moe, xt)[0]
    for t in (0, T // 2, T - 1):
        one = mq.moe_forward(c.moe, xt[t:t + 1])[0].float()
        assert bool(((y[t:t + 1].float() - one).abs() <= 1e-30).all())


def test_one_workspace_per_stream():
    """Calls of many sizes keep one workspace to a stream, that of the largest, and give what
    they give with one of their own."""
    c = Case(512, 512, 12, 4, MX, MX, 256, seed=80)
    say("moe workspaces")
    sizes = (1, 7, 200, 20, 2, 65, 130, 1, 200)
    got = []
    for T in sizes:
        x = c.x(T, 500 + T)[1]
        got.append((x, mq.moe_forward(c.moe, x), mq.router_topk(c.moe.router, x)))
    assert len(c.moe._ws.kept) == 1 == len(c.moe.router._ws.kept)
    for x, r, chosen in got:
        fresh = mq.MoeLayer(c.moe.layer, c.moe.router, c.moe.shared)
        for a, b in zip(r, mq.moe_forward(fresh, x)):
            assert torch.equal(a, b)
        assert torch.equal(chosen[0], r[1]) and torch.equal(chosen[1], r[2])


def test_layer_then_linear():
    """As a decoder runs them: the attention output through an INT8 projection, then the layer."""
    c = Case(512, 512, 12, 4, MX, MX, 256, seed=77)
    proj, (pq, ps) = int8_weight(512, 512, c.g)
    for T in (1, 5):
        _, a = c.x(T, 400 + T)
        x = mq.linear_int8_dynamic(proj, a)
        y, ids, rw = mq.moe_forward(c.moe, x)
        q, s = quant_ref(host(a))
        lin = (q.astype(np.float64) @ pq.T) * s.astype(np.float64)[:, None] * ps
        assert np.all(np.abs(x.double().cpu().numpy() - lin) <= 2.0 ** -8 * np.abs(lin) * 1.001 + 1e-30)
        c.check(x.cpu().view(torch.int16).numpy().view(np.uint16), x, y, ids, rw)


def test_no_tokens():
    c = Case(512, 512, 12, 4, MX, MX, 256, seed=78)
    y, ids, rw = mq.moe_forward(c.moe, torch.empty((0, 512), dtype=torch.bfloat16, device="cuda"))
    assert y.shape == (0, 512) and ids.shape == (0, 4)
