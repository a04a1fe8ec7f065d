"""The gated activation where sigma is below 2^-126 and its products are not: the far
gates' outputs and gradients keep their values, not 0."""
import numpy as np
import pytest
import torch

import _mx_ref as R
import fp4_precision_gemms_amd as F
from _moe import E24, act_parts, glu_near
from _util import need_gpu, say

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8       # half a step of bf16


@pytest.mark.parametrize("act", [F.ACT_SILU, F.ACT_GELU])
def test_far_gates(act):
    """sigma to its half step of 2^-149 or its roundings, times the other factors;
    bf16 values to theirs, below 2^-126 to a step of 2^-133."""
    need_gpu()
    say("glu tail", act)
    rng = np.random.default_rng(act)
    rows, cols = 40, 256
    g = rng.uniform(-104, -84, (rows, cols))
    if act == F.ACT_GELU:                                # s = 2 sqrt(2/pi) (g + 0.044715 g^3) in that range
        g = rng.uniform(-11.05, -10.1, (rows, cols))
    u = np.exp2(rng.uniform(0, 60, (rows, cols))) * rng.choice([-1, 1], (rows, cols))
    x = torch.from_numpy(np.concatenate((g, u), 1)).bfloat16()
    y, xq, xs = F.fp4_glu(x.cuda(), act, checkpoint=True)
    v = x.double().numpy()
    g, u = v[:, :cols], v[:, cols:]
    s, _, _ = act_parts(g, act)
    sigma = np.exp(s) / (1 + np.exp(s))
    assert (sigma < 2.0 ** -126).mean() > 0.3 and (np.abs(g * sigma * u) > 2.0 ** -126).mean() > 0.6
    ref = g * sigma * u
    near = glu_near(s) * np.abs(ref) + 2.0 ** -149 * np.abs(g * u)
    assert (np.abs(y.double().cpu().numpy() - ref) <= near + HALF * (np.abs(ref) + near) + 2.0 ** -134).all()

    # at the checkpoint's values: gates are a few steps of E4M3 there
    dy = torch.from_numpy(rng.standard_normal((rows, cols)) * 1e3).bfloat16()
    dx = F.fp4_glu_backward(dy.cuda(), xq, xs, act).double().cpu().numpy()
    v = R.mxfp8_values(xq.cpu().numpy(), xs.cpu().numpy())
    g, u, d = v[:, :cols], v[:, cols:], dy.double().numpy()
    s, _, gds = act_parts(g, act)
    sigma = np.exp(s) / (1 + np.exp(s))
    slope = sigma + gds * sigma / (1 + np.exp(s))
    ref = np.concatenate((d * u * slope, d * g * sigma), 1)
    rel, step = glu_near(s) + 8 * E24, 2.0 ** -149
    near = np.concatenate((np.abs(d * u) * (rel * sigma + step) * (1 + np.abs(gds)), np.abs(d * g) * (rel * sigma + step)), 1)
    assert (np.abs(dx - ref) <= near + HALF * (np.abs(ref) + near) + 2.0 ** -134).all()
    assert (dx[:, cols:][np.abs(ref[:, cols:]) > 2.0 ** -130] != 0).all()
