"""The layers' gradients have no gradients: a backward pass through them is refused
and not left out without a word."""
import pytest
import torch

import fp4_precision_gemms_amd as F
from _util import need_gpu

pytestmark = pytest.mark.gpu


def layers():
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x = torch.randn(64, 64, **bf)
    off = torch.tensor([0, 40, 64], dtype=torch.int32, device="cuda")
    logits = torch.randn(64, 3, device="cuda")

    def filled(layer):
        with torch.no_grad():
            for p in layer.parameters():
                p.normal_(0, 0.1)
        return layer

    linear, norm = filled(F.linear.MXFP4Linear(64, 96, device="cuda")), filled(F.linear.MXFP4NormLinear(64, 96, device="cuda"))
    grouped, moe = filled(F.linear.MXFP4GroupedLinear(2, 64, 96, device="cuda")), filled(F.moe.MXFP4MoE(3, 2, 64, 32, device="cuda"))
    return {"linear": (lambda t: linear(t), x), "norm": (lambda t: norm(t)[0], x), "grouped": (lambda t: grouped(t, off), x),
            "moe": (lambda t: moe(t, logits), x),
            "route": (lambda t: F.moe.RouteFunction.apply(t, 2, F.SCORE_SOFTMAX, False)[1], logits)}


@pytest.mark.parametrize("name", ["linear", "norm", "grouped", "moe", "route"])
def test_a_second_derivative_is_refused(name):
    need_gpu()
    call, value = layers()[name]
    leaf = value.clone().requires_grad_(True)
    y = call(leaf)
    weight = torch.randn_like(y).requires_grad_(True)
    plain, = torch.autograd.grad((y.float() * weight.float()).sum(), leaf, retain_graph=True)
    first, = torch.autograd.grad((y.float() * weight.float()).sum(), leaf, create_graph=True)
    assert torch.equal(first.detach(), plain)
    # beside a part that has a second derivative
    loss = first.float().square().sum() + leaf.float().square().sum()
    with pytest.raises(RuntimeError, match="once_differentiable"):
        loss.backward()
