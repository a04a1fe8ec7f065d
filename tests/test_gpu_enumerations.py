"""Enumerations beyond 32 bits are refused, not taken by their low bits."""
import pytest
import torch

import fp4_precision_gemms_amd as F
from _util import need_gpu

pytestmark = pytest.mark.gpu

FAR = [2 ** 32, 2 ** 32 + 1, -2 ** 32, 2 ** 40 + 1]


@pytest.mark.parametrize("far", FAR)
def test_refused(far):
    need_gpu()
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    x, w = z(4, 64), z(64)
    logits, ids = z(4, 8, dtype=torch.float32), z(4, 2, dtype=torch.int32)
    q, s = z(4, 64, dtype=torch.uint8), z(4, 2, dtype=torch.uint8)
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    for call in (lambda: F.fp4_hadamard_quantize(z(64, 64), far),
                 lambda: F.fp4_rmsnorm_quantize(x, w, fmt=far),
                 lambda: F.fp4_quantize_grouped(x, off, had=far), lambda: F.fp4_quantize_grouped(x, off, rnd=far),
                 lambda: F.fp4_quantize_grouped(x, off, had=F.HAD_DET, had_n=far + 32),
                 lambda: F.fp4_moe_route(logits, 2, far),
                 lambda: F.fp4_moe_route_backward(z(4, 2, dtype=torch.float32), logits, ids, far),
                 lambda: F.fp4_glu(x, far), lambda: F.fp4_glu_quantize(x, far), lambda: F.fp4_glu_quantize(x, fmt=far),
                 lambda: F.fp4_glu_backward(z(4, 32), q, s, far)):
        with pytest.raises(F.Fp4Error) as e:
            call()
        assert e.value.status == 4
    with pytest.raises(OverflowError):
        F.fp4_moe_route(logits, 2, 2 ** 70)
