"""The router in every kernel that its sizes choose, several choices of each: ids
exactly, weights and gradients within the roundings that enter them, counted from
the differences of logits and not from their size."""
import numpy as np
import pytest
import torch

import fp4_precision_gemms_amd as F
from _moe import route
from _util import need_gpu, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24                 # half a step of binary32, relative
TINY = 2.0 ** -125             # exponentials below 2^-126 are 0
# 16 lanes a token with 1, 2, 4, 8, 16 experts each, a wave with 1, 2, 4, 8, 16
SIZES = [(13, 16, 16), (7, 32, 11), (11, 64, 16), (67, 100, 8), (33, 128, 16), (21, 256, 8), (19, 200, 12), (9, 256, 16),
         (5, 40, 20), (3, 64, 64), (6, 128, 64), (6, 256, 40), (5, 512, 33), (9, 300, 5), (4, 1024, 64)]
KINDS = ["any", "ties", "one lane", "few live", "far"]
SCORES = [(F.SCORE_SOFTMAX, True), (F.SCORE_SOFTMAX, False), (F.SCORE_SIGMOID, True), (F.SCORE_SIGMOID, False)]


def logits_of(rng, T, E, k, kind, dtype):
    v = rng.standard_normal((T, E)) * 2
    if kind == "ties":
        v = np.round(v * 2) / 2
    elif kind == "one lane":
        # neighbours four at a time go to one lane, the next four to the next: the
        # largest ones all with lane 3 (of either number of lanes, as far as E reaches)
        lanes = 16 if k <= 16 and E <= 256 else 64
        each = -(-E // lanes)
        run = min(4, 1 << (each - 1).bit_length())
        v[:, (np.arange(E) // run) % lanes == min(3, E - 1)] += 12
    elif kind == "few live":
        live = rng.permuted(np.broadcast_to(np.arange(E), (T, E)), axis=1) < np.arange(T)[:, None] % (k + 1)
        v = np.where(live, v, rng.choice([-np.inf, np.nan], (T, E)))
    elif kind == "far":
        v[::3] = -1e4 + np.round(v[::3] * 16)              # every sigmoid is zero in binary32
        v[1::3, ::2] = torch.finfo(dtype).min
        v[2::3] *= 30
    return torch.from_numpy(v).to(dtype)


def spread(rel, part, live):
    """The relative error of a sum of positive parts with relative errors `rel`."""
    part = np.where(live, part, 0.0)
    with np.errstate(all="ignore"):
        return np.nan_to_num((np.where(live, rel, 0.0) * part).sum(1, keepdims=True) / part.sum(1, keepdims=True))


def over_top(l, top):
    """exp(l - top) and the relative error of the kernel's: the difference rounded
    once (a u in the exponent), the exponential a step (2 u), its argument's roundings
    (3 u)."""
    with np.errstate(all="ignore"):
        a = np.where(l > -np.inf, np.minimum(top - l, 104.0), 104.0)
        return np.where(l > -np.inf, np.exp(-(top - l)), 0.0), (a + 5) * U


def log_sigmoid(l):
    """log sigma(l) and its error: 1 + exp(-|l|) rounded (1 u, and 5 u of the
    exponential), the logarithm to a step and an absolute 2 u, two products, the
    difference; for l < -17 the sum is 1 and the result l itself."""
    with np.errstate(all="ignore"):
        s = np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l)))
        return s, np.where(l < -17, np.exp(np.minimum(l, 0)), (11 + np.abs(s)) * U)


def reference(l, g, k, sigmoid, normalize):
    """(ids, weights, their bound, gradient, its bound) in 64 bits."""
    l = np.where(np.isnan(l), -np.inf, l)
    T, E = l.shape
    ids, w = route(l, k, sigmoid, normalize)
    live = ids >= 0
    at = np.maximum(ids, 0)
    rows = np.arange(T)[:, None]
    c = np.where(live, l[rows, at], -np.inf)
    top = np.where(live[:, :1], c[:, :1], 0.0)
    adds, quotient = 22 * U, 3 * U
    dense = not sigmoid and not normalize
    near_0 = np.exp(-np.clip(np.abs(c), 0, 700))
    sigma, rest = (np.where(v < 0, near_0, 1.0) / (1 + near_0) for v in (c, -c))       # sigma and 1 - sigma
    if dense:
        part, rel = over_top(l, top)
        p = part / np.where(live[:, :1], part.sum(1, keepdims=True), 1.0)
        prel = rel + spread(rel, part, l > -np.inf) + adds + quotient
        wrel = prel[rows, at]
    elif not sigmoid:
        part, rel = over_top(c, top)
        wrel = rel + spread(rel, part, live) + adds + quotient
    elif normalize:
        s, off = log_sigmoid(np.where(live, c, 0.0))
        part, rel = over_top(np.where(live, s, -np.inf), s[:, :1])
        rel = rel + off + off[:, :1]
        wrel = rel + spread(rel, part, live) + adds + quotient
    else:
        wrel = np.full(w.shape, 10 * U)          # exponential 5, sum 1, reciprocal 2, product 1, quotient by 1
    wnear = np.where(live, wrel * w + TINY, 0.0)
    g = np.where(live, g.astype(np.float64), 0.0)
    inner = (g * w).sum(1, keepdims=True)
    inner_near = (np.abs(g) * w * (wrel + 8 * U) + TINY * np.abs(g)).sum(1, keepdims=True)
    if sigmoid and not normalize:
        each, near = g * sigma * rest, 20 * U * np.abs(g * sigma * rest) + TINY * np.abs(g)
    else:
        each = w * (g - inner)
        near = w * (np.abs(g - inner) * (wrel + 3 * U) + inner_near) + TINY * (np.abs(g) + np.abs(inner))
        if sigmoid:
            near = rest * (near + 11 * U * np.abs(each)) + TINY * np.abs(each)
            each = each * rest
    d, dnear = np.zeros((T, E)), np.zeros((T, E))
    if dense:
        full = np.zeros((T, E))
        np.add.at(full, (np.broadcast_to(rows, at.shape), at), g)
        d = p * (full - inner)
        dnear = p * (np.abs(full - inner) * (prel + 3 * U) + inner_near) + TINY * (np.abs(full) + np.abs(inner))
        dnear[l == -np.inf] = 0
    else:
        np.add.at(d, (np.broadcast_to(rows, at.shape), at), np.where(live, each, 0.0))
        np.add.at(dnear, (np.broadcast_to(rows, at.shape), at), np.where(live, near, 0.0))
    return ids, w, wnear, d, dnear


def within(got, ref, near):
    bad = np.argwhere(~(np.abs(got.double().cpu().numpy() - ref) <= near))
    worst = [(tuple(i), got[tuple(i)].item(), ref[tuple(i)], near[tuple(i)]) for i in bad[:4]]
    assert not len(bad), (len(bad), worst)


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", KINDS)
def test_route_and_its_gradient(T, E, k, dtype, kind):
    need_gpu()
    rng = np.random.default_rng(E * 100 + k)
    l = logits_of(rng, T, E, k, kind, dtype)
    g = rng.standard_normal((T, k)).astype(np.float32)
    for score, normalize in SCORES:
        say("route bounds", T, E, k, dtype, kind, score, normalize)
        ids, w = F.fp4_moe_route(l.cuda(), k, score, normalize)
        d = F.fp4_moe_route_backward(torch.from_numpy(g).cuda(), l.cuda(), ids, score, normalize)
        torch.cuda.synchronize()
        want, ref, near, dref, dnear = reference(l.double().numpy(), g, k, score == F.SCORE_SIGMOID, normalize)
        assert np.array_equal(ids.cpu().numpy(), want)
        assert near.max() < 2.0 ** -12                   # no row's bound lets anything pass
        within(w, ref, near)
        out = 2.0 ** -8 if dtype == torch.bfloat16 else U
        within(d, dref, dnear + out * (np.abs(dref) + dnear))
