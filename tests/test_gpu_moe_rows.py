"""Slots sorted by expert, tokens gathered to rows and combined: whole numbers and
moved values exactly, sums within their roundings, untouched rows as they were."""
import numpy as np
import pytest
import torch

import fp4_precision_gemms_amd as F
from _moe import E24, sort
from _util import need_gpu, say

pytestmark = pytest.mark.gpu


def gpu(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def ids_of(rng, T, k, E, kind):
    if kind == "one":
        return np.full((T, k), E - 1)
    if kind == "none":
        return rng.choice([-1, E, 2 ** 31 - 1, -2 ** 31], (T, k))
    v = rng.integers(0, E, (T, k))
    if kind == "dropped":
        v = np.where(rng.random((T, k)) < 0.2, rng.choice([-1, -5, E, E + 1, 2 ** 31 - 1, -2 ** 31], (T, k)), v)
    return np.where(rng.random((T, k)) < 0.3, E // 2, v) if kind == "uneven" else v


@pytest.mark.parametrize("T,k", [(1, 1), (1, 7), (9, 7), (8, 8), (13, 5), (171, 3), (512, 1), (1023, 4), (1024, 4),
                                 (1366, 3), (4097, 1), (7000, 6), (40000, 8)])
@pytest.mark.parametrize("kind", ["any", "dropped", "uneven", "one", "none"])
def test_sort(T, k, kind):
    need_gpu()
    for E in (1, 2, 8, 63, 64, 65, 200, 1024):
        say("sort", T, k, E, kind)
        ids = ids_of(np.random.default_rng(T + E), T, k, E, kind)
        want = sort(ids, E)
        got = F.fp4_moe_sort(gpu(ids, torch.int32), E)
        torch.cuda.synchronize()
        for a, b, n in zip(got, want, ("offsets", "order", "position")):
            assert a.dtype == torch.int32 and np.array_equal(a.cpu().numpy(), b), n


@pytest.mark.parametrize("E", [3, 1024])
def test_sort_of_many_slots(E):
    """More slots than the workgroups' usual share."""
    need_gpu()
    ids = ids_of(np.random.default_rng(1), 300001, 5, E, "dropped")
    say("sort many", E)
    ws = torch.empty(F.fp4_moe_sort_workspace_bytes(ids.size, E), dtype=torch.uint8, device="cuda")
    got = F.fp4_moe_sort(gpu(ids, torch.int32), E, workspace=ws)
    torch.cuda.synchronize()
    for a, b in zip(got, sort(ids, E)):
        assert np.array_equal(a.cpu().numpy(), b)


COLS = [32, 96, 1024, 1056, 2080, 4096, 4128, 8224, 24608]
SHAPES = [(1, 1, 4), (5, 6, 64), (67, 3, 5), (40, 9, 16)]


def case(T, k, E, cols, kind="dropped", seed=0):
    rng = np.random.default_rng(T * cols + seed)
    ids = ids_of(rng, T, k, E, kind)
    _, order, position = sort(ids, E)
    return rng, order, position


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("T,k,E", SHAPES)
def test_gather(T, k, E, cols):
    need_gpu()
    rng, _, position = case(T, k, E, cols)
    say("gather", T, k, E, cols)
    p = gpu(position, torch.int32)
    x = torch.from_numpy(rng.integers(-2 ** 15, 2 ** 15, (T, cols), dtype=np.int16)).cuda()
    for rows in (T * k, T * k + 3, max(1, T * k // 2)):
        live = (position >= 0) & (position < rows)
        out = torch.full((rows, cols), 0x7A7A, dtype=torch.int16, device="cuda")
        want = out.cpu().numpy()
        want[position[live]] = x.cpu().numpy()[np.nonzero(live)[0]]
        got = F.fp4_moe_gather(x.view(torch.bfloat16), p, out=out.view(torch.bfloat16))
        torch.cuda.synchronize()
        assert np.array_equal(got.view(torch.int16).cpu().numpy(), want)
        q = torch.from_numpy(rng.integers(0, 256, (T, cols), dtype=np.uint8)).cuda()
        s = torch.from_numpy(rng.integers(0, 256, (T, cols // 32), dtype=np.uint8)).cuda()
        outs = [torch.full((rows, n), 0xCD, dtype=torch.uint8, device="cuda") for n in (cols, cols // 32)]
        wants = [o.cpu().numpy() for o in outs]
        for a, b in zip(wants, (q, s)):
            a[position[live]] = b.cpu().numpy()[np.nonzero(live)[0]]
        got = F.fp4_moe_gather(q, p, s, out=outs)
        torch.cuda.synchronize()
        for a, b in zip(got, wants):
            assert np.array_equal(a.cpu().numpy(), b)
    new = F.fp4_moe_gather(x.view(torch.bfloat16), p)
    assert new.shape == (T * k, cols) and new.dtype == torch.bfloat16


def test_positions_out_of_range_and_scales_off_alignment():
    need_gpu()
    x = torch.randn(3, 64, device="cuda").bfloat16()
    p = torch.tensor([[0, 6], [-2 ** 31, 2 ** 31 - 1], [5, -1]], dtype=torch.int32, device="cuda")
    out = torch.zeros(6, 64, device="cuda").bfloat16()
    F.fp4_moe_gather(x, p, out=out)
    assert torch.equal(out[0], x[0]) and torch.equal(out[5], x[2]) and not out[1:5].any()
    got = F.fp4_moe_combine(out, p)
    assert torch.equal(got[0], x[0]) and not got[1].any() and torch.equal(got[2], x[2])
    scales = torch.arange(1, 8, device="cuda").to(torch.uint8)[1:].view(3, 2)       # an odd address
    codes = torch.arange(3 * 64, device="cuda").to(torch.uint8).view(3, 64)
    q, s = F.fp4_moe_gather(codes, p[:, :1].contiguous(), scales)
    assert torch.equal(s[0], scales[0]) and torch.equal(q[0], codes[0])


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("T,k,E", SHAPES)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_and_its_gradient(T, k, E, cols, weighted):
    need_gpu()
    rng, _, position = case(T, k, E, cols)
    say("combine", T, k, E, cols, weighted)
    live = position >= 0
    y = torch.from_numpy(rng.standard_normal((T * k, cols)).astype(np.float32)).bfloat16()
    w = rng.standard_normal((T, k)).astype(np.float32)
    free = np.setdiff1d(np.arange(T * k), position[live])
    y[free] = float("nan")                               # rows of no slot hold anything
    w[~live] = np.nan
    p, wg = gpu(position, torch.int32), gpu(w)
    got = F.fp4_moe_combine(y.cuda(), p, wg if weighted else None)
    torch.cuda.synchronize()
    terms = y.double().numpy()[np.maximum(position, 0)] * (w.astype(np.float64) if weighted else np.ones_like(w))[..., None]
    terms[~live] = 0
    ref, size = terms.sum(1), np.abs(terms).sum(1)
    # k sums in binary32 (each product exact or within the same rounding), one rounding to bf16
    near = (k + 1) * E24 * size
    assert (np.abs(got.double().cpu().numpy() - ref) <= near + 2.0 ** -8 * (np.abs(ref) + near)).all()
    if not weighted:
        return
    d = torch.from_numpy(rng.standard_normal((T, cols)).astype(np.float32)).bfloat16()
    dy0 = torch.full((T * k, cols), 3.0).bfloat16()
    dy, dw = F.fp4_moe_combine_backward(d.cuda(), y.cuda(), p, wg, out=(dy0.cuda(), torch.full((T, k), 9.0, device="cuda")))
    torch.cuda.synchronize()
    want = dy0.clone()
    rows = position[live]
    want[rows] = (torch.from_numpy(w)[live][:, None] * d.float()[np.nonzero(live)[0]]).bfloat16()
    assert torch.equal(dy.cpu(), want)
    pairs = y.double().numpy()[np.maximum(position, 0)] * d.double().numpy()[:, None]
    pairs[~live] = 0
    # a lane's sum of 8 ceil(cols / 8 / 64) products at most, the lanes' and the waves'
    n = 8 * -(-cols // 512) + 12
    assert (np.abs(dw.double().cpu().numpy() - pairs.sum(2)) <= n * E24 * np.abs(pairs).sum(2)).all()
    # in place
    y2 = y.cuda()
    _, dw2 = F.fp4_moe_combine_backward(d.cuda(), y2, p, wg, out=(y2, torch.empty(T, k, device="cuda")))
    torch.cuda.synchronize()
    assert torch.equal(y2[rows].cpu(), want[rows]) and torch.equal(dw, dw2)
    assert torch.isnan(y2[free]).all()


@pytest.mark.parametrize("k,cols", [(70, 96), (64, 32), (130, 1056)])
def test_more_choices_than_lanes(k, cols):
    """Positions and weights come 64 at a time."""
    need_gpu()
    T = 5
    rng, _, position = case(T, k, 16, cols)
    say("many choices", k, cols)
    live = position >= 0
    p = gpu(position, torch.int32)
    x = torch.from_numpy(rng.integers(-4, 5, (T, cols)).astype(np.float32)).bfloat16()
    rows = torch.zeros(T * k, cols).bfloat16()
    got = F.fp4_moe_gather(x.cuda(), p, out=rows.cuda()).cpu()
    rows[position[live]] = x[np.nonzero(live)[0]]
    assert torch.equal(got, rows)
    # small whole numbers: every sum is exact in binary32
    y = torch.from_numpy(rng.integers(-2, 3, (T * k, cols)).astype(np.float32)).bfloat16()
    w = torch.from_numpy(rng.integers(-2, 3, (T, k)).astype(np.float32))
    terms = y.double().numpy()[np.maximum(position, 0)] * w.double().numpy()[..., None] * live[..., None]
    out = F.fp4_moe_combine(y.cuda(), p, w.cuda()).cpu()
    assert torch.equal(out, torch.from_numpy(terms.sum(1)).bfloat16())
    dy, dw = F.fp4_moe_combine_backward(x.cuda(), y.cuda(), p, w.cuda(), out=(torch.zeros_like(rows).cuda(), w.cuda()))
    want = torch.zeros_like(rows)
    want[position[live]] = (w[live][:, None] * x.float()[np.nonzero(live)[0]]).bfloat16()
    assert torch.equal(dy.cpu(), want)
    pairs = (y.double().numpy()[np.maximum(position, 0)] * x.double().numpy()[:, None] * live[..., None]).sum(2)
    assert np.array_equal(dw.double().cpu().numpy(), pairs)


@pytest.mark.parametrize("cols,rows", [(1024, 140000), (2080, 70000)])
def test_rows_beyond_the_last_level_cache(cols, rows):
    """Non-temporal reads: the same values as from a small copy of the rows."""
    need_gpu()
    say("far rows", cols, rows)
    T, k = 20, 3
    big = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    at = torch.randperm(rows, device="cuda")[:T * k].sort().values
    small = torch.randn(T * k, cols, device="cuda").bfloat16()
    big[at] = small
    p = torch.randperm(T * k, device="cuda").int().view(T, k)
    p[3, 1] = -1
    far = torch.where(p < 0, -1, at[p.clamp(min=0).long()]).int()
    w, d = torch.randn(T, k, device="cuda"), torch.randn(T, cols, device="cuda").bfloat16()
    for weights in (None, w):
        assert torch.equal(F.fp4_moe_combine(big, far, weights), F.fp4_moe_combine(small, p, weights))
    dy, dw = F.fp4_moe_combine_backward(d, small, p, w, out=(torch.zeros_like(small), torch.empty_like(w)))
    dbig, dwf = F.fp4_moe_combine_backward(d, big, far, w, out=(torch.zeros_like(big), torch.empty_like(w)))
    assert torch.equal(dwf, dw) and torch.equal(dbig[at], dy)
    assert int(torch.count_nonzero(dbig.any(1))) == int(torch.count_nonzero(dy.any(1)))


def test_combine_of_infinite_values():
    need_gpu()
    inf = float("inf")
    y = torch.zeros(4, 32, device="cuda").bfloat16()
    y[0], y[1], y[2, 5] = inf, -inf, float("nan")
    p = torch.tensor([[0, 3], [0, 1], [3, 2]], dtype=torch.int32, device="cuda")
    got = F.fp4_moe_combine(y, p, torch.ones(3, 2, device="cuda"))
    assert (got[0] == inf).all() and torch.isnan(got[1]).all() and torch.isnan(got[2, 5]) and got[2, :5].eq(0).all()


def test_gather_and_combine_are_each_others_gradient():
    """<gather(x), r> = <x, combine(r)> where each row has one token."""
    need_gpu()
    rng, _, position = case(50, 4, 8, 96)
    p = gpu(position, torch.int32)
    x = torch.randint(-4, 5, (50, 96), device="cuda").bfloat16()
    r = torch.randint(-4, 5, (200, 96), device="cuda").bfloat16()
    rows = torch.zeros(200, 96, device="cuda").bfloat16()
    F.fp4_moe_gather(x, p, out=rows)
    back = F.fp4_moe_combine(r, p)
    assert float((rows.double() * r.double()).sum()) == float((x.double() * back.double()).sum())


def test_beyond_32_bit_offsets():
    """Rows past 2^31 elements of the experts' tensor, few tokens."""
    need_gpu()
    cols, rows = 8192, 2 ** 18 + 40
    big = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(3, cols, device="cuda").bfloat16()
    p = torch.tensor([[rows - 1, 0], [2 ** 18 + 1, 7], [rows - 2, -1]], dtype=torch.int32, device="cuda")
    F.fp4_moe_gather(x, p, out=big)
    assert torch.equal(big[rows - 1], x[0]) and torch.equal(big[2 ** 18 + 1], x[1]) and torch.equal(big[rows - 2], x[2])
    w = torch.tensor([[1.0, 2.0], [0.5, 0.5], [1.0, 5.0]], device="cuda")
    out = F.fp4_moe_combine(big, p, w)
    assert torch.equal(out, (x.float() * torch.tensor([[3.0], [1.0], [1.0]], device="cuda")).bfloat16())
    _, dw = F.fp4_moe_combine_backward(x, big, p, w, out=(big, torch.empty_like(w)))
    want = (x.double() ** 2).sum(1)
    assert torch.allclose(dw[:, 0].double(), want, rtol=1e-4) and torch.allclose(dw[:2, 1].double(), want[:2], rtol=1e-4)
    assert dw[2, 1] == 0 and torch.equal(big[rows - 2], x[2]) and torch.equal(big[7], (0.5 * x[1].float()).bfloat16())
