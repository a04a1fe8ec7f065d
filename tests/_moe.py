"""Plain references, in 64 bits, of the operators around the experts' products:
router, sorted slots, gated activation."""
import numpy as np
import torch

import _mx_ref as R

E24 = 2.0 ** -24       # half a step of binary32, relative


def route(logits, k, sigmoid, normalize):
    """(ids, weights) of logits [T, E] (float64 that hold the logits' own values):
    the first of the largest that are left, k times."""
    left = np.where(np.isnan(logits), -np.inf, logits)
    with np.errstate(all="ignore"):
        top = left.max(1, keepdims=True)
        over = np.where(left == top, 1.0, np.exp(left - top))
        over[left == -np.inf] = 0.0
        log = np.minimum(left, 0) - np.log1p(np.exp(-np.abs(left)))
    ids = np.full((len(left), k), -1)
    a = np.zeros((len(left), k))
    rows = np.arange(len(left))
    work = left.copy()
    for j in range(k):
        at = work.argmax(1)                          # the first one
        live = work[rows, at] > -np.inf
        ids[live, j] = at[live]
        with np.errstate(all="ignore"):
            if not sigmoid:
                v = over[rows, at]
            elif normalize:
                d = log[rows, at] - log[rows, np.maximum(ids[:, 0], 0)]
                v = np.where(log[rows, at] == log[rows, np.maximum(ids[:, 0], 0)], 1.0, np.exp(d))
            else:
                v = np.exp(log[rows, at])
        a[live, j] = v[live]
        work[rows, at] = -np.inf
    total = a.sum(1, keepdims=True) if normalize else (1.0 if sigmoid else over.sum(1, keepdims=True))
    with np.errstate(all="ignore"):
        return ids, np.where(ids >= 0, a / total, 0.0)


def route_weights(logits, ids, sigmoid, normalize):
    """The same weights as a differentiable function of torch float64 logits."""
    live = ids >= 0
    l = logits.gather(1, ids.clamp(min=0)).masked_fill(~live, -float("inf"))
    if not sigmoid:
        return torch.softmax(l, 1).masked_fill(~live, 0) if normalize else \
            (torch.softmax(logits, 1).gather(1, ids.clamp(min=0)).masked_fill(~live, 0))
    if normalize:
        return torch.softmax(torch.nn.functional.logsigmoid(l), 1).masked_fill(~live, 0)
    return torch.sigmoid(l).masked_fill(~live, 0)


def sort(ids, experts):
    flat = np.where((ids >= 0) & (ids < experts), ids, experts).ravel()
    order = np.argsort(flat, kind="stable")
    offsets = np.searchsorted(flat[order], np.arange(experts + 1))
    position = np.empty_like(flat)
    position[order] = np.arange(flat.size)
    return offsets, order, np.where(flat == experts, -1, position).reshape(ids.shape)


def act_parts(g, gelu):
    """(s, sigma, g s'(g)) of float64 gates; act = g sigma, act' = sigma + g s' sigma (1 - sigma)."""
    c = 2 * np.sqrt(2 / np.pi)
    s = c * (g + 0.044715 * g ** 3) if gelu else g
    with np.errstate(all="ignore"):
        return s, 1 / (1 + np.exp(-s)), c * (g + 3 * 0.044715 * g ** 3) if gelu else g


def act_value(g, gelu):
    return g * act_parts(g, gelu)[1]


def glu_near(s):
    """Relative error of act(g) u w in binary32: s off by 4 half steps of its own
    (|s| of them in the exponential), the exponential and the reciprocal by a step
    each, the sum and four products by half a step."""
    return (4 * np.abs(s) + 16) * E24


def e4m3(v):
    return torch.from_numpy(np.clip(v, -448, 448)).to(torch.float32).to(torch.float8_e4m3fn).double().numpy()


def e2m1(v):
    mid = (R.GRID[:-1] + R.GRID[1:]) / 2
    a = np.abs(v)[..., None]
    n = np.where(np.arange(7) % 2 == 1, a >= mid, a > mid).sum(-1)
    return np.copysign(R.GRID[n], v)


def check_quantized(values, scale_bytes, ref, near, top):
    """Values [R, C] that codes stand for and their scale bytes [R, C/32] against
    `ref` known to +-near: the scale between those of the two ends of the block's
    largest magnitude, each value between those of ref's two ends."""
    lo, hi = np.abs(ref) - near, np.abs(ref) + near
    low = R.block_exponents(np.maximum(lo, 0).astype(np.float64), top)
    high = R.block_exponents(hi.astype(np.float64), top)
    assert ((scale_bytes >= low) & (scale_bytes <= high)).all()
    s = np.exp2(np.repeat(scale_bytes.astype(np.float64), 32, 1) - 127)
    to = e4m3 if top == 8 else e2m1
    assert (values >= to((ref - near) / s) * s).all() and (values <= to((ref + near) / s) * s).all()
