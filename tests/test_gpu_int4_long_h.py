"""Few tokens of INT4 experts at the sizes that decide where h goes: parts that fill more than half of a
work-group's LDS, nearly all of it, or more than it has (then the down is tiled, from one token on)."""
import numpy as np
import pytest

import bit_quantized_moe_dequant_amd as mq
from tests.test_gpu_int4 import say
from tests.test_gpu_int4_moe import G32, G64, G128, Z32, Z64, Experts, check

pytestmark = pytest.mark.gpu

SHAPES = [  # H, I, E, K, gate/up, down: KB of h in a work-group
    (256, 1664, 9, 6, Z64, G128),    # 59
    (128, 768, 20, 16, Z64, G64),    # 73
    (256, 2048, 10, 7, G128, Z32),   # 84
    (256, 2048, 16, 8, Z64, G128),   # 96.4
    (128, 16896, 3, 1, Z64, G128),   # 99
    (160, 2944, 9, 8, G32, Z64),     # 138
    (128, 6400, 6, 5, Z64, Z32),     # 188
    (128, 2048, 20, 16, Z64, G128),  # 193
]


@pytest.mark.parametrize("shape", SHAPES)
def test_few_tokens(shape):
    H, I, E, K, fg, fd = shape
    ex = Experts(H, I, E, K, fg, fd, seed=I)
    for T in (1, 2, 5):
        say("long h", shape, T)
        xt, ti, tr, y, ref, tol = check(ex, T, seed=T)
        ws = ex.layer.workspace(T)
        if T > 1:
            mq.route(ex.layer, ti, ws=ws)
        h = mq.gate_up(ex.layer, xt, ti, ws=ws)
        got = mq.down(ex.layer, h, ti, tr, ws=ws).double().cpu().numpy()
        assert np.all(np.abs(got - ref) <= tol)
