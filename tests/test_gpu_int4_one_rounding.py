"""The output type of an INT4 linear decides nothing but the last rounding, at the largest tiles too."""
import pytest
import torch

import bit_quantized_moe_dequant_amd as mq
from tests.int4_ref import FMTS, Parts
from tests.test_gpu_int4 import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,cols,T", [(250, 1152, 9), (250, 1152, 129), (4096, 512, 1600), (6016, 640, 1100)])
def test_bf16_outputs_are_the_rounded_fp32_ones(fmt, rows, cols, T):
    say("one rounding", fmt, rows, cols, T)
    p = Parts(fmt, 1, rows, cols, seed=rows + fmt, scale="fp16", zmax=255)
    w = p.pack()
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, cols), generator=g, device="cuda").to(torch.bfloat16)
    y = mq.linear_int4(w, x, out_dtype=torch.float32)
    assert torch.equal(mq.linear_int4(w, x), y.to(torch.bfloat16))
