"""Pairs whose expert id is out of range: the INT4 gate/up stage writes zeros for them, pair by pair
and tiled alike, and the rest as without them."""
import numpy as np
import pytest
import torch

import bit_quantized_moe_dequant_amd as mq
from tests.int4_ref import Parts, group_of
from tests.test_gpu_int4 import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [mq.FMT_INT4_G128, mq.FMT_INT4Z_G32, mq.FMT_INT4_G64])
@pytest.mark.parametrize("T", [1, 5, 60, 200])
def test_gate_up_writes_zeros_for_pairs_out_of_range(fmt, T):
    """h starts as NaN. 12 experts, 4 to a token: from 60 tokens on the products are tiled, in tiles of
    32 pairs and (200 tokens, more than 64 of them out of range) of 64."""
    say("gate_up skipped", fmt, T)
    H, I, E, K = 1024, 512 + group_of(fmt), 12, 4
    g = np.random.default_rng(T)
    w = [Parts(fmt, E, *s, 60 + i).pack() for i, s in enumerate([(I, H), (I, H), (H, I)])]
    layer = mq.Layer(H, I, E, K, *w)
    x = torch.from_numpy(g.standard_normal((T, H))).to(torch.bfloat16).cuda()
    ids = np.stack([g.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    full = torch.from_numpy(ids.copy()).cuda()
    out = g.random((T, K)) < 0.4
    out[0, 1], out[T - 1, K - 1], out[0, 0] = True, True, False
    ids[out] = np.where(g.random(out.sum()) < 0.5, -1, np.where(g.random(out.sum()) < 0.5, E, 1 << 30))
    part = torch.from_numpy(ids).cuda()

    def stage(i):
        ws = layer.workspace(T)
        if T > 1:
            mq.route(layer, i, ws=ws)
        h = torch.full((T, K, I), float("nan"), device="cuda")
        mq.gate_up(layer, x, i, h=h, ws=ws)
        return h, mq.check_device_error(ws)

    want, err = stage(full)
    assert err == 0 and not bool(want.isnan().any())
    h, err = stage(part)
    skipped = torch.from_numpy(out).cuda()
    assert err & mq.DEVERR_EXPERT_ID
    assert bool((h[skipped] == 0).all())
    assert torch.equal(h[~skipped], want[~skipped])  # a pair's sum does not depend on the others in its tile
    h, _ = stage(torch.full_like(part, E))
    assert bool((h == 0).all())
