"""A mixture of experts of no tokens is refused, forward and in the decode step."""
import pytest
import torch

import fp4_precision_gemms_amd as F
from _util import need_gpu

pytestmark = pytest.mark.gpu


def test_no_tokens():
    need_gpu()
    layer = F.moe.MXFP4MoE(4, 2, 64, 32, device="cuda")
    with torch.no_grad():
        layer.gate_up.zero_()
        layer.down.zero_()
    q1, q2 = F.linear.quantize_experts(layer.gate_up.detach()), F.linear.quantize_experts(layer.down.detach())
    u8 = dict(dtype=torch.uint8, device="cuda")
    for call in (lambda: layer(torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(0, 4, device="cuda")),
                 lambda: F.moe.moe_decode(torch.zeros(0, 64, **u8), torch.zeros(0, 2, **u8), torch.zeros(0, 4, device="cuda"),
                                          2, *q1[2:], *q2[2:])):
        with pytest.raises(F.Fp4Error) as e:
            call()
        assert e.value.status == 2
