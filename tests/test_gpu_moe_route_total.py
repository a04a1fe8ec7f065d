"""The softmax over all experts: its total is one for the weights and their
gradient, and a token's alone."""
import pytest
import torch

import fp4_precision_gemms_amd as F
from _util import need_gpu, say

pytestmark = pytest.mark.gpu

# every number of lanes a token and of experts a lane
SIZES = [(7, 2), (30, 3), (60, 6), (100, 8), (200, 8), (256, 12), (40, 20), (128, 20), (250, 17), (500, 9), (1024, 8)]


@pytest.mark.parametrize("E,k", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient_divides_by_the_weights_total(E, k, dtype):
    """With the gradient of one weight j alone the top expert's is -(p_top w_j), p_top
    the top weight: one product in binary32, so the same bits where the two passes
    have the same total."""
    need_gpu()
    say("route total", E, k, dtype)
    torch.manual_seed(E)
    T = 301
    l = (torch.randn(T, E) * 2).to(dtype).cuda()
    l[::3] = (torch.rand(T, E) * 8).to(dtype).cuda()[::3]
    l[1::3] = -5.3125
    l[1::3, E // 2] = 0.0                                # hundreds of equal ones below the top
    l = l.contiguous()
    ids, w = F.fp4_moe_route(l, k, F.SCORE_SOFTMAX, False)
    for j in (1, k - 1):
        g = torch.zeros(T, k, device="cuda")
        g[:, j] = 1.0
        d = F.fp4_moe_route_backward(g, l, ids, F.SCORE_SOFTMAX, False)
        top = d.gather(1, ids[:, :1].long())[:, 0]
        assert torch.equal(top, (-(w[:, 0] * w[:, j])).to(dtype))


@pytest.mark.parametrize("E,k", SIZES)
@pytest.mark.parametrize("score,normalize", [(F.SCORE_SOFTMAX, False), (F.SCORE_SOFTMAX, True), (F.SCORE_SIGMOID, True)])
def test_a_token_beside_one_with_infinite_logits(E, k, score, normalize):
    """The tokens that share a wave do not change each other's bits."""
    need_gpu()
    say("route neighbours", E, k, score, normalize)
    torch.manual_seed(E + 1)
    T = 403
    l = torch.randn(T, E, device="cuda") * 3
    other = l.clone()
    other[::4] = float("inf")
    other[::8, 1:] = 1.0
    kept = torch.ones(T, dtype=torch.bool, device="cuda")
    kept[::4] = False
    g = torch.randn(T, k, device="cuda")
    a, b = (F.fp4_moe_route(t, k, score, normalize) for t in (l, other))
    assert torch.equal(a[0][kept], b[0][kept]) and torch.equal(a[1][kept], b[1][kept])
    da, db = (F.fp4_moe_route_backward(g, t, i[0], score, normalize) for t, i in ((l, a), (other, b)))
    assert torch.equal(da[kept], db[kept])
    if score == F.SCORE_SOFTMAX:
        share = 1.0 / (k if normalize else E)            # all logits infinite: equal parts
        assert ((b[1][4] - share).abs() <= 2.0 ** -22 * share).all()
        assert b[1][0].tolist() == [1.0] + [0.0] * (k - 1)


@pytest.mark.parametrize("E,k", SIZES)
def test_masked_logits_get_zero_from_gradients_that_are_no_numbers(E, k):
    """Zero for every logit that is no choice, as documented, whatever the weights'
    gradient."""
    need_gpu()
    say("route masked", E, k)
    torch.manual_seed(E + 2)
    T, inf = 37, float("inf")
    l = torch.randn(T, E, device="cuda")
    masked = torch.rand(T, E, device="cuda") < 0.4
    l = l.masked_fill(masked, -inf).masked_fill(masked & (torch.rand(T, E, device="cuda") < 0.3), float("nan"))
    for score, normalize in ((F.SCORE_SOFTMAX, False), (F.SCORE_SOFTMAX, True), (F.SCORE_SIGMOID, True), (F.SCORE_SIGMOID, False)):
        ids, w = F.fp4_moe_route(l, k, score, normalize)
        g = torch.randn(T, k, device="cuda")
        g[1::3, 0], g[2::3, 0] = inf, float("nan")
        d = F.fp4_moe_route_backward(g, l, ids, score, normalize)
        assert not d[masked].any()                       # a NaN counts as one here
        live = (ids[:, 0] >= 0)
        live[0::3] = False
        assert not torch.isfinite(d[live].gather(1, ids[live][:, :1].long())).any() or score == F.SCORE_SIGMOID
