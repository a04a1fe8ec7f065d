"""The gated activation against 64 bits: outputs within the roundings of binary32
and of their own type, the checkpoint bit for bit, gradients at the checkpoint's
values by the formula and by differences."""
import numpy as np
import pytest
import torch

import _mx_ref as R
import fp4_precision_gemms_amd as F
from _moe import E24, act_parts, act_value, check_quantized, glu_near
from _util import need_gpu, say, ungroup_scales, untile_codes

pytestmark = pytest.mark.gpu

SHAPES = [(1, 32), (1, 1408), (3, 96), (33, 736), (70, 1024), (5, 1056), (17, 2080), (2, 14336), (1030, 1056)]
ACTS = [F.ACT_SILU, F.ACT_GELU]
HALF = 2.0 ** -8       # half a step of bf16


def gpu(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def inputs(rows, cols, seed=0, wide=True):
    rng = np.random.default_rng(rows * 10000 + cols + seed)
    x = rng.standard_normal((rows, 2 * cols)) * 1.5
    if wide:                                             # far gates, zeros, tiny values
        x[rng.random(x.shape) < 0.05] *= 20
        x[rng.random(x.shape) < 0.02] = 0
        x[rng.random(x.shape) < 0.02] *= 1e-20
    return rng, torch.from_numpy(x).bfloat16()


def reference(x, act, w):
    v = x.double().numpy()
    c = v.shape[1] // 2
    g, u = v[:, :c], v[:, c:]
    s = act_parts(g, act)[0]
    y = act_value(g, act) * u * w[:, None]
    # sigma below 2^-126 is flushed
    return y, glu_near(s) * np.abs(y) + 2.0 ** -125 * np.abs(g * u * w[:, None])


def row_weights(rng, rows, how):
    """(w by row, weights, order) of none, by row, by way of an order."""
    if how == "none":
        return np.ones(rows), None, None
    w = rng.standard_normal(rows).astype(np.float32)
    if how == "rows":
        return w.astype(np.float64), w, None
    order = rng.permutation(rows)
    return w[order].astype(np.float64), w, order


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("how", ["none", "rows", "order"])
def test_forward(rows, cols, act, how):
    need_gpu()
    say("glu", rows, cols, act, how)
    rng, x = inputs(rows, cols)
    w, weights, order = row_weights(rng, rows, how)
    wg, og = None if weights is None else gpu(weights), None if order is None else gpu(order, torch.int32)
    ref, near = reference(x, act, w)
    y, xq, xs = F.fp4_glu(x.cuda(), act, wg, og, checkpoint=True)
    plain = F.fp4_glu(x.cuda(), act, wg, og)
    torch.cuda.synchronize()
    assert torch.equal(y, plain)
    assert (np.abs(y.double().cpu().numpy() - ref) <= near + HALF * (np.abs(ref) + near) + 2.0 ** -134).all()
    wq, ws = R.mxfp8(x.float().numpy())
    assert np.array_equal(xq.cpu().numpy(), wq) and np.array_equal(xs.cpu().numpy(), ws)
    codes, scales = (t.cpu().numpy() for t in F.fp4_glu_quantize(x.cuda(), act, wg, og))
    check_quantized(R.mxfp8_values(codes, scales), scales, ref, near, 8)
    codes, scales = F.fp4_glu_quantize(x.cuda(), act, wg, og, fmt=F.FMT_MXFP4)
    assert codes.shape == F.code_shape(rows, cols) and scales.shape == F.scale_shape(rows, cols)
    c, s = untile_codes(codes.cpu().numpy(), rows), ungroup_scales(scales.cpu().numpy(), cols // 32)
    check_quantized(R.mxfp4_values(c, s), s, ref, near, 2)


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("how", ["none", "rows", "order"])
def test_backward(rows, cols, act, how):
    need_gpu()
    say("glu back", rows, cols, act, how)
    rng, x = inputs(rows, cols, 1)
    w, weights, order = row_weights(rng, rows, how)
    codes, scales = R.mxfp8(x.float().numpy())
    v = R.mxfp8_values(codes, scales)
    dy = torch.from_numpy(rng.standard_normal((rows, cols)) * 1e-2).bfloat16()
    wg, og = None if weights is None else gpu(weights), None if order is None else gpu(order, torch.int32)
    got = F.fp4_glu_backward(dy.cuda(), gpu(codes), gpu(scales), act, wg, og)
    torch.cuda.synchronize()
    dx = (got if how == "none" else got[0]).double().cpu().numpy()
    d, g, u = dy.double().numpy(), v[:, :cols], v[:, cols:]
    s, sigma, gds = act_parts(g, act)
    both = sigma * (1 / (1 + np.exp(np.clip(s, -700, 700))))
    slope = sigma + gds * both
    dw = d * w[:, None]
    ref = np.concatenate((dw * u * slope, dw * g * sigma), 1)
    rel, tiny = glu_near(s) + 8 * E24, 2.0 ** -125
    near = np.concatenate((np.abs(dw * u) * (rel * (sigma + np.abs(gds) * both) + tiny * (1 + np.abs(gds))),
                           np.abs(dw * g) * (rel * sigma + tiny)), 1)
    assert (np.abs(dx - ref) <= near + HALF * (np.abs(ref) + near) + 2.0 ** -134).all()
    if how != "none":
        terms = d * g * sigma * u
        by_row = terms.sum(1)
        n = 8 * -(-cols // 512) + 12                     # a lane's sum, the lanes' and the waves'
        tol = (np.abs(terms) * (rel + n * E24) + tiny * np.abs(d * g * u)).sum(1)
        want, bound = np.empty(rows), np.empty(rows)
        at = np.arange(rows) if order is None else order
        want[at], bound[at] = by_row, tol
        assert (np.abs(got[1].double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    """The kernel's dx and dweights against central differences of the forward
    formula in 64 bits: off by h^2 / 6 of a third derivative (below 4 |u| here),
    rounding and the outputs' own steps."""
    need_gpu()
    rng = np.random.default_rng(3)
    rows, cols, h = 6, 64, 1e-4
    x = torch.from_numpy(rng.standard_normal((rows, 2 * cols)) * 2).bfloat16()
    codes, scales = R.mxfp8(x.float().numpy())
    v = R.mxfp8_values(codes, scales)
    w = rng.standard_normal(rows).astype(np.float32)
    dy = torch.from_numpy(rng.standard_normal((rows, cols))).bfloat16()
    dx, dw = F.fp4_glu_backward(dy.cuda(), gpu(codes), gpu(scales), act, gpu(w))
    torch.cuda.synchronize()
    d = dy.double().numpy()

    def f(g, u, ww):
        return act_value(g, act) * u * ww

    g, u, ww = v[:, :cols], v[:, cols:], w.astype(np.float64)[:, None]
    dg = d * (f(g + h, u, ww) - f(g - h, u, ww)) / (2 * h)
    du = d * (f(g, u + h, ww) - f(g, u - h, ww)) / (2 * h)
    ref = np.concatenate((dg, du), 1)
    size = np.concatenate((np.abs(d * ww * u), np.abs(d * ww * g)), 1)
    near = (1e-7 + 64 * E24) * size + 1e-10
    assert (np.abs(dx.double().cpu().numpy() - ref) <= near + HALF * (np.abs(ref) + near)).all()
    wref = (d * (f(g, u, ww + h) - f(g, u, ww - h)) / (2 * h)).sum(1)
    assert (np.abs(dw.double().cpu().numpy() - wref) <= 1e-5 * np.abs(d * g * u).sum(1)).all()


@pytest.mark.parametrize("offsets", [[0, 3, 3, 9], [2, 2, 7], [4, 4, 4], [0, 40], [-3, 5], [30, 10]])
@pytest.mark.parametrize("cols", [96, 2080])
def test_rows_of_no_expert_are_left_as_they_were(offsets, cols):
    need_gpu()
    rows = 12
    say("glu offsets", offsets, cols)
    rng, x = inputs(rows, cols, 2, wide=False)
    lo, hi = offsets[0], offsets[-1]
    live = np.zeros(rows, bool)
    live[max(lo, 0):max(hi, 0)] = True
    x[~live] = float("nan")
    off = gpu(np.array(offsets), torch.int32)
    order = rng.permutation(rows)
    w, og = gpu(rng.standard_normal(rows).astype(np.float32)), gpu(order, torch.int32)
    whole = F.fp4_glu(x.cuda(), F.ACT_SILU, w, og, checkpoint=True) + F.fp4_glu_quantize(x.cuda(), F.ACT_SILU, w, og)
    fill = [torch.full_like(t, 7) for t in whole]
    F.fp4_glu(x.cuda(), F.ACT_SILU, w, og, off, checkpoint=True, out=fill[:3])
    F.fp4_glu_quantize(x.cuda(), F.ACT_SILU, w, og, off, out=fill[3:])
    torch.cuda.synchronize()
    for a, b in zip(fill, whole):
        assert torch.equal(a[live], b[live]) and (a[~live] == 7).all()
    dy = torch.randn(rows, cols).bfloat16().cuda()
    dx, dw = F.fp4_glu_backward(dy, whole[1], whole[2], F.ACT_SILU, w, og)
    out = (torch.full_like(dx, 7), torch.full_like(dw, 7))
    F.fp4_glu_backward(dy, whole[1], whole[2], F.ACT_SILU, w, og, off, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out[0][live], dx[live]) and (out[0][~live] == 7).all()
    slots = order[live]
    assert torch.equal(out[1][slots], dw[slots]) and not out[1][order[~live]].any()
    c4 = F.fp4_glu_quantize(x.cuda(), F.ACT_SILU, w, og, fmt=F.FMT_MXFP4)
    o4 = [torch.full_like(t, 9) for t in c4]
    F.fp4_glu_quantize(x.cuda(), F.ACT_SILU, w, og, off, F.FMT_MXFP4, out=o4)
    a, b = (untile_codes(t.cpu().numpy(), rows) for t in (o4[0], c4[0]))
    assert np.array_equal(a[live], b[live]) and (a[~live] == 9).all()


def test_extreme_gates():
    """Far gates: the limits, not a NaN; a NaN or an infinity reaches its own
    output (and its checkpoint block's gradients), no other."""
    need_gpu()
    big = 3e38
    cols = 64
    x = torch.ones(4, 2 * cols)
    x[0, :8] = torch.tensor([big, -big, 1e30, -1e30, 1e-30, -1e-30, 100.0, -100.0])
    x[1, 3], x[2, cols + 5], x[3, 40] = float("nan"), float("inf"), float("inf")
    x = x.bfloat16()
    for act in ACTS:
        y, xq, xs = F.fp4_glu(x.cuda(), act, checkpoint=True)
        v = y.float().cpu()
        xb = x.float()
        assert v[0, 0] == xb[0, 0] and v[0, 1] == 0 and v[0, 2] == xb[0, 2] and v[0, 3] == 0
        assert v[0, 6] == 100 and abs(float(v[0, 7])) < 1e-30
        assert torch.isnan(v[1, 3]) and torch.isfinite(v[1, :3]).all() and torch.isfinite(v[1, 4:]).all()
        assert v[2, 5] == float("inf") and v[3, 40] == float("inf")
        assert xs[1].tolist()[0] == 255 and xs[2].tolist()[2] == 255 and xs[3].tolist()[1] == 255
        dx = F.fp4_glu_backward(torch.ones(4, cols, device="cuda").bfloat16(), xq, xs, act).cpu().float()
        assert torch.isfinite(dx[0]).all()
        assert torch.isnan(dx[1, :32]).all() and torch.isfinite(dx[1, 32:cols]).all()
        assert torch.isnan(dx[2, :32]).all() and torch.isnan(dx[3, 32:cols]).all() and torch.isfinite(dx[3, :32]).all()


@pytest.mark.parametrize("fmt", [F.FMT_MXFP8, F.FMT_MXFP4])
def test_every_output_of_one_call(fmt):
    """The C entry point writes whichever outputs it is given."""
    need_gpu()
    rng, x = inputs(37, 1056, 4)
    x = x.cuda()
    y, xq, xs = F.fp4_glu(x, F.ACT_GELU, checkpoint=True)
    codes, scales = F.fp4_glu_quantize(x, F.ACT_GELU, fmt=fmt, out=None)
    out = [torch.zeros_like(t) for t in (y, codes, scales, xq, xs)]
    status = F.lib().fp4_glu(x.data_ptr(), None, None, None, 0, F.ACT_GELU, 37, 1056, out[0].data_ptr(), fmt,
                             *(t.data_ptr() for t in out[1:]), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert status == 0 and torch.equal(out[0], y) and torch.equal(out[3], xq) and torch.equal(out[4], xs)
    values = R.mxfp8_values if fmt == F.FMT_MXFP8 else R.mxfp4_values
    def rows(c, s):
        c, s = c.cpu().numpy(), s.cpu().numpy()
        return (c, s) if fmt == F.FMT_MXFP8 else (untile_codes(c, 37), ungroup_scales(s, 33))
    assert np.array_equal(values(*rows(out[1], out[2])), values(*rows(codes, scales)))
    # the checkpoint alone
    only = [torch.zeros_like(t) for t in (xq, xs)]
    status = F.lib().fp4_glu(x.data_ptr(), None, None, None, 0, F.ACT_GELU, 37, 1056, None, fmt, None, None,
                             only[0].data_ptr(), only[1].data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert status == 0 and torch.equal(only[0], xq) and torch.equal(only[1], xs)


def test_orders_out_of_range():
    """A row whose order names no row has weight 0 and no entry in dweights."""
    need_gpu()
    rng, x = inputs(4, 64, 3, wide=False)
    order = torch.tensor([2, -1, 4, 0], dtype=torch.int32, device="cuda")
    w = torch.tensor([2.0, 3.0, 5.0, 7.0], device="cuda")
    y, xq, xs = F.fp4_glu(x.cuda(), F.ACT_SILU, w, order, checkpoint=True)
    by_row = torch.tensor([5.0, 0.0, 0.0, 2.0], device="cuda")
    assert torch.equal(y, F.fp4_glu(x.cuda(), F.ACT_SILU, by_row))
    dy = torch.randn(4, 64, device="cuda").bfloat16()
    want = F.fp4_glu_backward(dy, xq, xs, F.ACT_SILU, by_row)
    dw = torch.full((4,), 9.0, device="cuda")
    dx, _ = F.fp4_glu_backward(dy, xq, xs, F.ACT_SILU, w, order, out=(torch.empty_like(want[0]), dw))
    assert torch.equal(dx, want[0]) and dw[1] == 9 and dw[3] == 9 and dw[2] == want[1][0] and dw[0] == want[1][3]


def test_beyond_32_bit_offsets():
    """More than 2^32 bytes and 2^31 elements: the last rows as in a small call."""
    need_gpu()
    rows, cols = 70000, 16384
    x = torch.zeros(rows, 2 * cols, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, 2 * cols, device="cuda").bfloat16()
    y, xq, xs = F.fp4_glu(x, checkpoint=True)
    ys, xqs, xss = F.fp4_glu(x[-3:].clone(), checkpoint=True)
    assert torch.equal(y[-3:], ys) and torch.equal(xq[-3:], xqs) and torch.equal(xs[-3:], xss) and not y[:-3].any()
    dx = F.fp4_glu_backward(y, xq, xs)
    assert torch.equal(dx[-3:], F.fp4_glu_backward(ys, xqs, xss)) and not dx[:-3].any()
    codes, scales = F.fp4_glu_quantize(x)
    cs, ss = F.fp4_glu_quantize(x[-3:].clone())
    assert torch.equal(codes[-3:], cs) and torch.equal(scales[-3:], ss)
