"""The whole layer at a prompt against its definition in 64 bits, where the routed experts'
MXFP4 projections take their activations as MXFP8 (from 128 tokens on): nothing of the
library's own goes into the reference.

Tolerance of y. The routed part of the reference quantises x (bit for bit the library's rule)
for an MXFP4 gate/up and its own h for an MXFP4 down. The library's h is within 2e-3 of that h
(floored at the RMS), so its codes may be any between those of the two ends, under the scale
of either end's block maximum: every product with such a code moves by at most the interval.
The projection tolerance of 2e-3, the shared part's and the bf16 rounding come on top, as for
fewer tokens (test_gpu_moe)."""
import numpy as np
import pytest
import torch

import bit_quantized_moe_dequant_amd as mq
from oracle import moe, mxfp8
from oracle.codecs import E4M3, bf16_to_f64, f64_to_e4m3fn_rne
from tests.helpers import TOL
from tests.test_gpu_int8 import quant_ref
from tests.test_gpu_moe import IQ, MX, NV, Q2, Case, host, say
from tests.test_gpu_router import route_ref

pytestmark = pytest.mark.gpu


def code_values(h, E):
    """The numbers that values h stand for under the block exponents E."""
    s = np.ldexp(1.0, E.astype(np.int64) - 127)[..., None]
    v = E4M3[f64_to_e4m3fn_rne(h.reshape(*E.shape, 32) / s)] * s
    return v.reshape(h.shape)


def quantised(h, delta):
    """MXFP8 of h, and how far it may move where h is within delta."""
    mid = mxfp8.dequantize(*mxfp8.quantize(h))
    blocks = lambda a: np.abs(a).reshape(h.shape[0], -1, 32).max(axis=2)
    ends = [mxfp8.block_exponent_code(np.maximum(blocks(h) + d, 0)) for d in
            (-delta.reshape(h.shape[0], -1, 32).max(axis=2), delta.reshape(h.shape[0], -1, 32).max(axis=2))]
    dev = np.zeros_like(h)
    for E in ends:
        for v in (h - delta, h + delta):
            dev = np.maximum(dev, np.abs(code_values(v, E) - mid))
    return mid, dev


def routed_ref(c, X, ids, rw, fg, fd):
    if fg == MX:
        X = mxfp8.dequantize(*mxfp8.quantize(X))
    T, K = ids.shape
    h = np.stack([[moe.swiglu(c.wfn(0, e) @ X[t], c.wfn(1, e) @ X[t]) for e in ids[t]] for t in range(T)])
    hq, dev = h, np.zeros_like(h)
    if fd == MX:
        delta = TOL * np.maximum(np.abs(h), np.sqrt(np.mean(h ** 2)))
        hq, dev = (a.reshape(h.shape) for a in quantised(h.reshape(T * K, -1), delta.reshape(T * K, -1)))
    y, tol = np.zeros((T, c.H)), np.zeros((T, c.H))
    for t in range(T):
        for k in range(K):
            D = c.wfn(2, ids[t, k])
            y[t] += rw[t, k] * (D @ hq[t, k])
            tol[t] += abs(rw[t, k]) * (np.abs(D) @ dev[t, k])
    return y, tol + TOL * np.maximum(np.abs(y), np.sqrt(np.mean(y ** 2)))


def shared_ref(c, X):
    (gq, gs), (uq, us), (dq, ds) = c.sh
    q, s = (a.astype(np.float64) for a in quant_ref(X))
    gate, up = (q @ gq.T) * s[:, None] * gs, (q @ uq.T) * s[:, None] * us
    h = (gate / (1 + np.exp(-gate)) * up).astype(np.float32)
    hq, hs = (a.astype(np.float64) for a in quant_ref(h))
    frac = np.abs(h / hs[:, None] - np.floor(h / hs[:, None]) - 0.5)
    flips = (frac < 1e-3).sum(axis=1)[:, None] * hs[:, None] * 127.0 * ds
    return (hq @ dq.T) * hs[:, None] * ds, flips + 2.0 ** -20 * (np.abs(hq) @ np.abs(dq).T) * hs[:, None] * ds


@pytest.mark.parametrize("fg,fd,T,kind,norm", [(MX, MX, 128, "sqrtsoftplus", True), (MX, MX, 301, "softmax", False),
                                               (MX, IQ, 140, "softmax", True), (IQ, MX, 129, "sigmoid", True),
                                               (NV, MX, 200, "sigmoid", False), (NV, Q2, 256, "softmax", False)])
def test_layer_at_a_prompt(fg, fd, T, kind, norm):
    say("moe prompt", fg, fd, T, kind)
    c = Case(512, 256, 12, 3, fg, fd, 272, kind=kind, norm=norm, bias=kind == "sigmoid", seed=T)
    bits, xt = c.x(T, 40 + T)
    y, ids, rw = mq.moe_forward(c.moe, xt)
    ref_ids, ref_rw, _ = route_ref(host(xt), host(c.rw), c.K, kind, norm, 1.5, host(c.rb))
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    assert np.allclose(rw.cpu().numpy(), ref_rw, rtol=2.0 ** -23, atol=0)
    rows = [0, 1, 5, T // 2, T - 2, T - 1]
    X = bf16_to_f64(bits)[rows]
    routed, tol = routed_ref(c, X, ref_ids[rows], ref_rw[rows], fg, fd)
    shared, more = shared_ref(c, host(xt)[rows])
    ref, tol = routed + shared, tol + more
    tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(y.double().cpu().numpy()[rows] - ref)
    full, _ = moe.moe_layer_f64(X, ref_ids[rows], ref_rw[rows], c.wfn)
    rms = np.sqrt(np.mean(full ** 2))
    say(f"largest error {(err / tol).max():.3f} of the tolerance; tolerance {tol.mean() / rms:.3f} of the routed RMS, "
        f"8-bit activations {np.sqrt(np.mean((routed - full) ** 2)) / rms:.4f}")
    assert np.all(err <= tol)
