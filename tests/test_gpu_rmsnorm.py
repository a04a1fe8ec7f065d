"""fp4_rmsnorm_quantize and fp4_rmsnorm_backward against plain references:
h, rstd, codes and scales bit for bit (the sum of squares is held in 64 bits,
so they do not depend on its order), the gradients within bounds from the
number of roundings, and against differences."""
import numpy as np
import pytest
import torch

import _mx_ref as R
import fp4_precision_gemms_amd as F
from _util import need_gpu, say, sentinel_u8, untile_codes, ungroup_scales

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24      # half a step of binary32
U16 = 2.0 ** -8       # half a step of bf16


def bf(v):
    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(torch.bfloat16).cuda()


def inputs(rows, cols, seed, residual=True):
    rng = np.random.default_rng(seed)
    x = R.to_bf16(rng.standard_normal((rows, cols)) * 1.5)
    r = R.to_bf16(rng.standard_normal((rows, cols))) if residual else None
    w = R.to_bf16(1 + 0.1 * rng.standard_normal(cols))
    return x, r, w


def check_forward(x, r, w, eps, fmt, got, rows, cols):
    codes, scales, h, rstd = got
    href, rref, y = R.rmsnorm(x, r, w, eps)
    assert np.array_equal(h.float().cpu().numpy(), href, equal_nan=True)
    assert np.array_equal(rstd.cpu().numpy().view(np.uint32) & 0x7FFFFFFF,
                          rref.view(np.uint32) & 0x7FFFFFFF) or np.array_equal(rstd.cpu().numpy(), rref, equal_nan=True)
    if fmt == F.FMT_MXFP8:
        c, s = R.mxfp8(y)
        got_c, got_s = codes.cpu().numpy(), scales.cpu().numpy()
    else:
        c, s = R.mxfp4(y)
        got_c = untile_codes(codes.cpu().numpy(), rows)
        got_s = ungroup_scales(scales.cpu().numpy(), cols // 32)
    assert np.array_equal(got_s, s)
    assert np.array_equal(got_c, c)
    return y


# every launch shape: a wave per row (2048 rows and more), a workgroup of 256
# and of 1024 threads per row, at their borders
SHAPES = [(1, 32), (1, 4096), (3, 64), (5, 2048), (2, 2080), (7, 4128), (33, 5152), (4, 8192), (3, 8224),
          (2, 16384), (2, 16416), (1, 32768), (2048, 96), (2047, 96), (2049, 1024), (2050, 1056), (2051, 2048),
          (2048, 2080), (2049, 4096), (2048, 4128)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("fmt", [F.FMT_MXFP8, F.FMT_MXFP4])
@pytest.mark.parametrize("residual", [True, False])
def test_forward_bits(rows, cols, fmt, residual):
    need_gpu()
    say("rmsnorm", rows, cols, fmt, residual)
    x, r, w = inputs(rows, cols, rows * 7 + cols, residual)
    got = F.fp4_rmsnorm_quantize(bf(x), bf(w), None if r is None else bf(r), 1e-5, fmt)
    torch.cuda.synchronize()
    check_forward(x, r, w, 1e-5, fmt, got, rows, cols)


@pytest.mark.parametrize("fmt", [F.FMT_MXFP8, F.FMT_MXFP4])
def test_forward_special_values(fmt):
    """Zero rows, rows with a NaN, an infinity, the largest and the smallest
    values, a residual that cancels x, one row whose square sum passes
    binary32's range; weights of zero and of both signs."""
    need_gpu()
    rows, cols = 9, 256
    x, r, w = inputs(rows, cols, 3)
    x[0], r[0] = 0, 0
    x[1, 40] = np.nan
    x[2, 70] = np.inf
    x[3] = 3.0e38
    r[3] = 0
    x[4], r[4] = 1e-40, 0
    x[5] = R.to_bf16(np.full(cols, 2.0 ** -126))
    r[5] = -x[5]
    x[6], r[6] = 0, 0
    x[6, 3] = -5
    r[7] = -x[7]
    r[7, 33] = 1.0
    w[32:64] = 0
    w[64:96] *= -1
    x, r = R.to_bf16(x), R.to_bf16(r)
    for eps in (0.0, 1e-5):
        say("rmsnorm special", fmt, eps)
        got = F.fp4_rmsnorm_quantize(bf(x), bf(w), bf(r), eps, fmt)
        torch.cuda.synchronize()
        check_forward(x, r, w, eps, fmt, got, rows, cols)


def test_e4m3_rounding_borders():
    """Values at and next to every midpoint of E4M3, and past 448: h r w with
    r made 1 by the row's own norm is not exact, so the row is built from
    equal magnitudes (r is then fl(1 / v)) and the weight carries the value."""
    need_gpu()
    cols = 512
    tab = R.e4m3_table()
    mids = (tab[1:] + tab[:-1]) / 2
    vals = np.concatenate((tab, mids, [464.0, 480.0, 500.0, 511.0]))
    vals = R.to_bf16(np.resize(vals, cols - cols // 32))
    w = np.zeros(cols, np.float32)
    at = np.arange(cols) % 32 != 0
    w[at], w[~at] = vals, R.to_bf16(np.full(cols // 32, 256.0))     # each block's scale is 2^0 or 2^1
    x = np.ones((2, cols), np.float32)
    x[1] = -1
    got = F.fp4_rmsnorm_quantize(bf(x), bf(w), None, 0.0, F.FMT_MXFP8)
    torch.cuda.synchronize()
    y = check_forward(x, None, w, 0.0, F.FMT_MXFP8, got, 2, cols)
    assert np.array_equal(np.abs(y[0]), np.abs(w))


def test_forward_writes_only_its_outputs():
    """MXFP4 padding rows and the tail of the last scale group stay as they
    were; y is the norm rounded to bf16; h in place of x and of the residual."""
    need_gpu()
    rows, cols = 5, 288
    x, r, w = inputs(rows, cols, 11)
    codes = sentinel_u8(F.code_shape(rows, cols))
    scales = sentinel_u8(F.scale_shape(rows, cols))
    for place in ("x", "residual"):
        gx, gr = bf(x), bf(r)
        y = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
        out = (codes, scales, gx if place == "x" else gr, torch.empty(rows, device="cuda"))
        got = F.fp4_rmsnorm_quantize(gx, bf(w), gr, 1e-6, F.FMT_MXFP4, out=out, y=y)
        torch.cuda.synchronize()
        yref = check_forward(x, r, w, 1e-6, F.FMT_MXFP4, got, rows, cols)
        assert np.array_equal(y.float().cpu().numpy(), R.to_bf16(yref))
    assert (codes.view(-1, 32, 16)[:, rows:] == 0xCD).all()
    assert (scales[1, :, 1:] == 0xCD).all()


def back_reference(dy, h, w, r, dh):
    dy, h, w, r = (v.astype(np.float64) for v in (dy, h, w, r[:, None]))
    g = dy * w
    C = h.shape[1]
    c = (g * h).sum(1, keepdims=True)
    dx = r * g - h * r ** 3 * c / C + (0 if dh is None else dh)
    # terms that are rounded in binary32: seven operations on the first two
    # and the sum of 8 elements times up to 4 chunks a lane, 6 and 16 joins
    size = np.abs(r * g) + np.abs(h * r ** 3 * c / C) + (0 if dh is None else np.abs(dh))
    csize = np.abs(h) * r ** 3 / C * (np.abs(g * h).sum(1, keepdims=True))
    near = 12 * U32 * size + 64 * U32 * csize
    return dx, U16 * (np.abs(dx) + near) + near, (dy * h * r).sum(0), np.abs(dy * h * r).sum(0)


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 2048), (5, 2080), (70, 4128), (2, 8192), (3, 8224), (2, 16416),
                                       (1, 32768), (1025, 96), (2500, 320)])
@pytest.mark.parametrize("with_dh", [True, False])
def test_backward(rows, cols, with_dh):
    need_gpu()
    say("rmsnorm back", rows, cols, with_dh)
    rng = np.random.default_rng(rows + cols)
    x, r, w = inputs(rows, cols, rows * 5 + cols)
    h, rstd, _ = R.rmsnorm(x, r, w, 1e-5)
    dy = R.to_bf16(rng.standard_normal((rows, cols)) * 1e-3)
    dh = R.to_bf16(rng.standard_normal((rows, cols)) * 1e-3) if with_dh else None
    args = (bf(dy), bf(h), bf(w), torch.from_numpy(rstd).cuda())
    dx, dw = F.fp4_rmsnorm_backward(*args, None if dh is None else bf(dh))
    again = F.fp4_rmsnorm_backward(*args, None if dh is None else bf(dh))
    torch.cuda.synchronize()
    ref, near, dwref, dwsize = back_reference(dy, h, w, rstd, dh)
    assert (np.abs(dx.double().cpu().numpy() - ref) <= near).all()
    # dw: rows of a workgroup one after another, then 32 slices of the parts
    parts = F.fp4_rmsnorm_workspace_bytes(rows, cols) // (4 * cols)
    depth = -(-rows // parts) + -(-parts // 32) + 32 + 3
    assert (np.abs(dw.double().cpu().numpy() - dwref) <= depth * U32 * dwsize).all()
    assert torch.equal(dx.view(torch.int16), again[0].view(torch.int16)) and torch.equal(dw, again[1])


def test_backward_against_differences():
    """<dx, u> + <dw, v> against the central difference of sum(dy y) in 64 bits
    along (u, v), h perturbed; dx and dw carry their own roundings."""
    need_gpu()
    rows, cols, eps, step = 6, 160, 1e-5, 1e-4
    rng = np.random.default_rng(0)
    x, _, w = inputs(rows, cols, 21, residual=False)
    _, rstd, _ = R.rmsnorm(x, None, w, eps)
    dy = R.to_bf16(rng.standard_normal((rows, cols)))
    dx, dw = F.fp4_rmsnorm_backward(bf(dy), bf(x), bf(w), torch.from_numpy(rstd).cuda())
    torch.cuda.synchronize()
    u, v = rng.standard_normal(x.shape), rng.standard_normal(cols)

    def f(t):
        h, ww = x.astype(np.float64) + t * u, w.astype(np.float64) + t * v
        return (dy * (h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * ww)).sum()

    want = (f(step) - f(-step)) / (2 * step)
    got = (dx.double().cpu().numpy() * u).sum() + (dw.double().cpu().numpy() * v).sum()
    _, near, _, dwsize = back_reference(dy, x, w, rstd, None)
    # rstd itself is off by half a step of binary32 at most: within 4 U32 of each term
    bound = (near * np.abs(u)).sum() + (20 * U32 * dwsize * np.abs(v)).sum() + 1e-6 * abs(want)
    assert abs(got - want) <= bound


def test_backward_in_place_and_workspace():
    need_gpu()
    rows, cols = 40, 512
    rng = np.random.default_rng(5)
    x, _, w = inputs(rows, cols, 2, residual=False)
    _, rstd, _ = R.rmsnorm(x, None, w, 1e-5)
    dy, dh = (R.to_bf16(rng.standard_normal((rows, cols))) for _ in range(2))
    args = (bf(dy), bf(x), bf(w), torch.from_numpy(rstd).cuda())
    dx, dw = F.fp4_rmsnorm_backward(*args, bf(dh))
    g = bf(dh)
    ws = torch.empty(F.fp4_rmsnorm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    out = (g, torch.empty(cols, device="cuda"))
    got = F.fp4_rmsnorm_backward(*args, g, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert got[0] is g and torch.equal(g.view(torch.int16), dx.view(torch.int16)) and torch.equal(out[1], dw)
    with pytest.raises(F.Fp4Error) as e:
        F.fp4_rmsnorm_backward(*args, workspace=ws[:64])
    assert e.value.status == 6


def test_another_stream_and_a_captured_graph():
    """Forward and backward on a side stream, then captured and replayed with
    eager work between the replays: the same bits each time."""
    need_gpu()
    rows, cols = 64, 1024
    x, r, w = inputs(rows, cols, 8)
    gx, gr, gw = bf(x), bf(r), bf(w)
    dy = bf(np.random.default_rng(1).standard_normal((rows, cols)))

    def work():
        codes, scales, h, rstd = F.fp4_rmsnorm_quantize(gx, gw, gr, 1e-5, F.FMT_MXFP8)
        return (codes, scales, h, rstd) + F.fp4_rmsnorm_backward(dy, h, gw, rstd)

    want = work()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = work()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    given = F.fp4_rmsnorm_backward(dy, side[2], gw, side[3], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(given[0], want[4]) and torch.equal(given[1], want[5])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = work()
    for i in range(3):
        for t in caught:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(want, caught, side):
            assert torch.equal(a, b) and torch.equal(a, c), i
        work()


@pytest.mark.parametrize("scale", [1e-18, 1e18, 1e30])
def test_backward_of_rows_far_from_one(scale):
    """h so small or large that r^3, or c = sum g h, leaves binary32: dx is the
    gradient all the same (eps = 0)."""
    need_gpu()
    rows, cols = 7, 352
    rng = np.random.default_rng(12)
    h = R.to_bf16(rng.standard_normal((rows, cols)) * scale)
    w = R.to_bf16(1 + 0.1 * rng.standard_normal(cols))
    dy = R.to_bf16(rng.standard_normal((rows, cols)))
    h0, rstd, _ = R.rmsnorm(h, None, w, 0.0)
    assert np.array_equal(h0, h) and np.isfinite(rstd).all() and (rstd > 2.0 ** -126).all()
    dx, dw = F.fp4_rmsnorm_backward(bf(dy), bf(h), bf(w), torch.from_numpy(rstd).cuda())
    torch.cuda.synchronize()
    ref, near, dwref, dwsize = back_reference(dy, h, w, rstd, None)
    assert (np.abs(dx.double().cpu().numpy() - ref) <= near).all()
    assert (np.abs(dw.double().cpu().numpy() - dwref) <= 64 * U32 * dwsize).all()
