"""The router where its fp32 sums, its bounds or its ties are at their worst, against the
64-bit form of test_gpu_router (and with its tolerances)."""
import numpy as np
import pytest
import torch

import bit_quantized_moe_dequant_amd as mq
from tests.test_gpu_router import SCORES, check, host, make, route_ref, say, scores_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("T", [4, 64, 100])
def test_weights_of_chosen_experts_whose_fp32_sums_overflow(T, norm):
    """Exact logits of 0 whose partial sums pass 2^128 and come back (by whole multiples of
    2^127, so that every order of summation gives 0), above logits that are all negative."""
    say("chosen overflow", T, norm)
    g = torch.Generator().manual_seed(15)
    x = torch.zeros((T, 1024))
    x[:, [0, 1, 512, 768]] = 2.0 ** 63
    x[:, 256:272] = torch.rand((T, 16), generator=g) + 0.5
    w = torch.zeros((40, 1024))
    w[:, 256:272] = -(torch.rand((40, 16), generator=g) + 0.5) / 8
    for e, sign in ((7, 1.0), (30, -1.0)):
        w[e] = 0
        w[e, [0, 1]], w[e, [512, 768]] = sign * 2.0 ** 64, -sign * 2.0 ** 64
    x, w = x.to(torch.bfloat16).cuda(), w.to(torch.bfloat16).cuda()
    for K in (1, 2, 5):
        ids, rw = mq.router_topk(mq.Router(w, K, scoring="softmax", normalize=norm), x)
        ref = route_ref(host(x), host(w), K, "softmax", norm, 1.0, None)
        assert np.isfinite(ref[1]).all() and ref[0][0, 0] == 7
        check(ids, rw, ref)


@pytest.mark.parametrize("scale", [2.0 ** 60, 2.0 ** 100])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("T", [4, 100])
def test_weights_at_magnitudes_beyond_fp32(T, norm, scale):
    """Exact logits beyond 2^128: the largest takes the whole weight, the others follow in the
    order of their logits."""
    say("weights beyond fp32", T, norm, scale)
    x, w, _ = make(T, 512, 40, 31)
    x, w = (x.float() * scale).to(torch.bfloat16), (w.float() * scale).to(torch.bfloat16)
    x[1] = 0
    z = x.double().cpu().numpy() @ w.double().cpu().numpy().T
    order = np.argsort(-z, axis=1, kind="stable")
    for K in (1, 5):
        ids, rw = mq.router_topk(mq.Router(w, K, scoring="softmax", normalize=norm), x)
        s = np.take_along_axis(scores_ref(z, "softmax"), order[:, :K], 1)
        check(ids, rw, (order[:, :K], s / s.sum(axis=1, keepdims=True) if norm else s, None))
