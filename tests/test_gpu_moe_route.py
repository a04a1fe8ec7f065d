"""The router against 64 bits: its choice exactly, weights and gradients within
the binary32 roundings of their formulas."""
import numpy as np
import pytest
import torch

import fp4_precision_gemms_amd as F
from _moe import E24, route, route_weights
from _util import need_gpu, say

pytestmark = pytest.mark.gpu

KINDS = [(F.SCORE_SOFTMAX, True), (F.SCORE_SOFTMAX, False), (F.SCORE_SIGMOID, True), (F.SCORE_SIGMOID, False)]
SIZES = [(1, 1, 1), (1, 64, 6), (5, 2, 2), (3, 7, 7), (130, 40, 4), (67, 63, 8), (9, 65, 64), (33, 128, 1),
         (130, 200, 8), (5, 256, 64), (7, 257, 5), (4, 512, 9), (3, 777, 8), (6, 1024, 64)]


def inputs(T, E, dtype, seed, masked):
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((T, E)) * 2
    if masked:
        v[rng.random((T, E)) < 0.3] = -np.inf
        v[rng.random((T, E)) < 0.05] = np.nan
        v[rng.random((T, E)) < 0.2] = 0.0
        v[rng.random((T, E)) < 0.1] = -0.0
        v[::5] = -np.inf
        v[2::7] = -1e4 + np.round(v[2::7] * 4)            # every sigmoid is zero in binary32
        if T > 3:
            v[3, :2] = torch.finfo(dtype).min
    return torch.from_numpy(v).to(dtype)


def bound(logits, E):
    """Relative error of a weight: the largest difference of logits (or of their
    log sigmoids, each a few half steps of itself), exponentials, the sum of up to
    16 values a lane and 6 steps over the lanes, the quotient."""
    d = np.where(np.isfinite(logits), np.abs(logits), 0).max(1, keepdims=True)
    return (6 * d + 64) * E24


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("masked", [False, True])
def test_route_and_its_gradient(T, E, k, dtype, masked):
    need_gpu()
    l = inputs(T, E, dtype, T * 1000 + E, masked)
    exact = l.double().numpy()
    g = np.random.default_rng(E).standard_normal((T, k)).astype(np.float32)
    for score, normalize in KINDS:
        say("route", T, E, k, dtype, masked, score, normalize)
        ids, w = F.fp4_moe_route(l.cuda(), k, score, normalize)
        d = F.fp4_moe_route_backward(torch.from_numpy(g).cuda(), l.cuda(), ids, score, normalize)
        torch.cuda.synchronize()
        assert d.dtype == dtype
        want, ref = route(exact, k, score == F.SCORE_SIGMOID, normalize)
        assert np.array_equal(ids.cpu().numpy(), want)
        near = bound(exact, E)
        assert (np.abs(w.cpu().double().numpy() - ref) <= near * ref + 2.0 ** -126).all()

        # the formula's gradient, by torch's differentiation in 64 bits
        v = torch.from_numpy(np.where(np.isnan(exact), -np.inf, exact)).clamp(min=-1e30).requires_grad_(True)
        live = torch.from_numpy(want >= 0)
        (route_weights(v, torch.from_numpy(want), score == F.SCORE_SIGMOID, normalize)
         * torch.from_numpy(g).double()).sum().backward()
        dref = torch.nan_to_num(v.grad).numpy()
        dref[~np.isfinite(np.where(np.isnan(exact), -np.inf, exact))] = 0
        dref[~live.numpy().any(1)] = 0
        got = d.cpu().double().numpy()
        p = np.zeros((T, E))
        at, j = np.nonzero(want >= 0)
        p[at, want[at, j]] = ref[at, j]
        if not normalize and not score:
            p = torch.softmax(v.detach(), 1).numpy()
        elif not normalize:
            p = 1 / (1 + np.exp(-np.clip(v.detach().numpy(), -700, 700)))
        size = p * (np.abs(g).max(1, keepdims=True) + (np.abs(g) * ref).sum(1, keepdims=True))
        out = 2.0 ** -8 if dtype == torch.bfloat16 else E24
        tol = 2 * near * size + out * np.abs(dref) + 2.0 ** -126
        assert (np.abs(got - dref) <= tol * (1 + out)).all()
        assert not got[~np.isfinite(exact)].any()


@pytest.mark.parametrize("score,normalize", KINDS)
def test_gradient_against_differences(score, normalize):
    """(f(l + h) - f(l - h)) / 2 h with f the sum of g w by the kernel itself: off
    by h^2 / 6 of a third derivative (at most 2 sum |g| here) and by the weights'
    2^-21 over h."""
    need_gpu()
    torch.manual_seed(5)
    E, k, h = 24, 3, 2.0 ** -6
    l = torch.randn(1, E).mul(64).round().div(32)            # exact steps, no ties within h
    l[0] += torch.randperm(E) * 0.25
    g = torch.randn(1, k)
    ids, _ = F.fp4_moe_route(l.cuda(), k, score, normalize)
    d = F.fp4_moe_route_backward(g.cuda(), l.cuda(), ids, score, normalize).cpu()
    step = torch.eye(E) * h
    ends = []
    for s in (step, -step):
        i, w = F.fp4_moe_route((l + s).cuda(), k, score, normalize)
        assert torch.equal(i.cpu(), ids.cpu().expand(E, k))
        ends.append((w.cpu().double() * g.double()).sum(1))
    diff = (ends[0] - ends[1]) / (2 * h)
    near = (h * h / 3 + 2.0 ** -21 / h) * g.abs().sum()
    assert ((d[0].double() - diff).abs() <= near).all()


def test_infinite_logits_share():
    need_gpu()
    inf = float("inf")
    l = torch.tensor([[1.0, inf, -3.0, inf], [inf, 2.0, 3.0, -inf]])
    for score in (F.SCORE_SOFTMAX, F.SCORE_SIGMOID):
        ids, w = F.fp4_moe_route(l.cuda(), 3, score, True)
        assert ids.tolist() == [[1, 3, 0], [0, 2, 1]]
        if score == F.SCORE_SOFTMAX:
            assert w.tolist() == [[0.5, 0.5, 0.0], [1.0, 0.0, 0.0]]
            # of all experts, beside a token of ordinary logits in the same wave
            both = torch.cat((l, torch.tensor([[0.0, 0.0, -inf, float("nan")]])))
            assert F.fp4_moe_route(both.cuda(), 3, score, False)[1].tolist() == w.tolist() + [[0.5, 0.5, 0.0]]
        d = F.fp4_moe_route_backward(torch.ones(2, 3, device="cuda"), l.cuda(), ids, score, True)
        assert torch.isfinite(d).all()


def test_ids_that_are_none_are_not_looked_at():
    need_gpu()
    l = torch.randn(6, 50, device="cuda")
    ids, _ = F.fp4_moe_route(l, 4)
    for bad in (-1, -7, 50, 2 ** 31 - 1, -2 ** 31):
        ids[:, 2] = bad
        g = torch.randn(6, 4, device="cuda")
        g[:, 2] = float("nan")
        for score, normalize in KINDS:
            d = F.fp4_moe_route_backward(g, l, ids, score, normalize)
            assert torch.isfinite(d).all()


def test_preallocated_outputs_and_unaligned_slices():
    """Decode steps over a slice of a batch's logits, odd widths."""
    need_gpu()
    for dtype in (torch.float32, torch.bfloat16):
        l = torch.randn(9, 41, device="cuda").to(dtype)
        want = F.fp4_moe_route(l, 3)
        out = (torch.full((9, 3), 77, dtype=torch.int32, device="cuda"), torch.zeros(9, 3, device="cuda"))
        for t in range(9):
            F.fp4_moe_route(l[t:t + 1], 3, out=(out[0][t:t + 1], out[1][t:t + 1]))
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        g = torch.randn(9, 3, device="cuda")
        whole = F.fp4_moe_route_backward(g, l, want[0])
        part = torch.empty_like(l)
        for t in range(9):
            F.fp4_moe_route_backward(g[t:t + 1], l[t:t + 1], want[0][t:t + 1], out=part[t:t + 1])
        assert torch.equal(whole, part)


def test_rows_off_the_vector_loads_alignment():
    """The same values at an address that whole rows of four cannot be loaded from."""
    need_gpu()
    for dtype in (torch.float32, torch.bfloat16):
        for E, k in ((40, 4), (200, 8), (1024, 20)):
            l = torch.randn(9, E, device="cuda").to(dtype)
            off = torch.empty(9 * E + 1, dtype=dtype, device="cuda")[1:].view(9, E)
            off.copy_(l)
            g = torch.randn(9, k, device="cuda")
            out = torch.empty(9 * E + 1, dtype=dtype, device="cuda")[1:].view(9, E)
            for score, normalize in KINDS:
                a, b = (F.fp4_moe_route(t, k, score, normalize) for t in (l, off))
                assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
                want = F.fp4_moe_route_backward(g, l, a[0], score, normalize)
                assert torch.equal(want, F.fp4_moe_route_backward(g, off, a[0], score, normalize, out=out))
