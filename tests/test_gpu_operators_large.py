"""The norm, grouped and few-row operators where offsets pass 32 bits (tensors
of more than 2^31 elements or bytes), and with the largest number of experts.
What a call writes beyond 32 bits is compared with the same rows or the same
expert in a call of their own."""
import numpy as np
import pytest
import torch

import fp4_precision_gemms_amd as F
from _grouped import check, dev_offsets, grouped_operand, operand, random_mx4, values
from _util import need_gpu, say

pytestmark = pytest.mark.gpu


def normal(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, scale, generator=g)


def same(a, b):
    assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("fmt", [F.FMT_MXFP8, F.FMT_MXFP4])
def test_norm_beyond_32_bits(fmt):
    need_gpu()
    rows, cols = 65600, 32768                          # 2^31 elements are 65536 rows
    say("norm beyond 32 bits", fmt)
    x, w = normal(rows, cols), normal(cols, seed=1)
    codes, scales, h, rstd = F.fp4_rmsnorm_quantize(x, w, x, fmt=fmt)
    for lo in (0, 65536 - 32, rows - 32):
        c, s, hh, r = F.fp4_rmsnorm_quantize(x[lo:lo + 32], w, x[lo:lo + 32], fmt=fmt)
        same(h[lo:lo + 32], hh)
        same(rstd[lo:lo + 32], r)
        if fmt == F.FMT_MXFP8:
            same(codes[lo:lo + 32], c)
            same(scales[lo:lo + 32], s)
        else:
            same(codes[lo // 32:lo // 32 + 1], c)
            same(scales[:, lo:lo + 32], s)
    del codes, scales
    dx, dw = F.fp4_rmsnorm_backward(x, h, w, rstd)
    lo = rows - 40
    alone = F.fp4_rmsnorm_backward(x[lo:], h[lo:], w, rstd[lo:])[0]
    same(dx[lo:], alone)


@pytest.mark.parametrize("had", [F.HAD_NONE, F.HAD_DET])
def test_grouped_rows_beyond_32_bits(had):
    """An expert whose rows, codes and products begin past 2^31 elements of x
    and 2^31 bytes of its codes."""
    need_gpu()
    rows, cols, N = 140000, 32768, 64
    offsets = [0, 139000, 139333, 139990]
    say("grouped rows beyond 32 bits", had)
    x, off = normal(rows, cols), dev_offsets(offsets)
    cr, sr, cc, sc = F.fp4_quantize_grouped_dual(x, off, 32, had)
    wq, ws = zip(*(F.fp4_hadamard_quantize(normal(N, cols, seed=e + 1)) for e in range(3)))
    y = F.fp4_gemm_grouped(cc, sc, off, torch.stack(wq), torch.stack(ws), rows, out_dtype=F.OUT_F32)
    for e in (1, 2):
        lo, hi = offsets[e], offsets[e + 1]
        n, u, g = hi - lo, lo // 32 + e, lo // 256 + e
        one = dev_offsets([0, n])
        cr1, sr1, cc1, sc1 = F.fp4_quantize_grouped_dual(x[lo:hi], one, 32, had)
        stages = -(-n // 256)
        same(cc[u:u + n // 32], cc1[:n // 32])
        same(sc[:, 32 * u:32 * u + n], sc1[:, :n])
        same(cr[:, 8 * g:8 * (g + stages)], cr1[:, :8 * stages])
        same(sr[g:g + stages], sr1[:stages])
        alone = F.fp4_gemm_grouped(cc1, sc1, one, wq[e][None], ws[e][None], n, out_dtype=F.OUT_F32)
        # the two calls may take different kernels, each within 1e-5 sum |a w|
        # <= 1e-5 |a| |w|, and a rounded vector at most twice as long as its own
        near = 2e-5 * 4 * x[lo:hi].float().norm(dim=1)[:, None] * normal(N, cols, seed=e + 1).float().norm(dim=1)
        assert ((y[lo:hi] - alone).abs() <= near).all()


@pytest.mark.parametrize("each", [100, 700])
def test_weight_gradients_beyond_32_bits(each):
    """An output of more than 2^31 elements, on either kernel."""
    need_gpu()
    E, N, K = 40, 8192, 7168
    say("weight gradients beyond 32 bits", each)
    rows = E * each
    offsets = [e * each for e in range(E + 1)]
    dy, x, off = normal(rows, N), normal(rows, K, seed=1), dev_offsets(offsets)
    d, q = (F.fp4_quantize_grouped(t, off, F.AXIS_ROWS, 32, F.HAD_DET) for t in (dy, x))
    dw = F.fp4_gemm_grouped_wgrad(*d, *q, off, rows)
    assert dw.numel() > 2 ** 31
    for e in (0, E - 1):
        one = dev_offsets([0, each])
        d1, q1 = (F.fp4_quantize_grouped(t[e * each:(e + 1) * each], one, F.AXIS_ROWS, 32, F.HAD_DET) for t in (dy, x))
        same(dw[e], F.fp4_gemm_grouped_wgrad(*d1, *q1, one, each)[0])


@pytest.mark.parametrize("each", [30, 34])
def test_output_beyond_32_bits(each):
    """C of more than 2^31 elements, from the few-row kernel and the tiles."""
    need_gpu()
    E, N, K = 600, 122880, 64
    rows = E * each
    offsets = [e * each for e in range(E + 1)]
    say("outputs beyond 32 bits", each)
    x, off = normal(rows, K), dev_offsets(offsets)
    q, w = F.fp4_quantize_grouped(x, off), F.fp4_hadamard_quantize(normal(N, K, seed=1))
    wq, ws = (t[None].expand(E, *t.shape).contiguous() for t in w)
    y = F.fp4_gemm_grouped(*q, off, wq, ws, rows)
    assert y.numel() > 2 ** 31
    one = dev_offsets([0, each])
    for e in (0, E - 1):
        q1 = F.fp4_quantize_grouped(x[e * each:(e + 1) * each], one)
        alone = F.fp4_gemm_grouped(*q1, one, wq[:1], ws[:1], each)
        # one 64-element step: at most a rounding of the output apart
        err = (y[e * each:(e + 1) * each].float() - alone.float()).abs()
        assert (err <= 2.0 ** -7 * alone.float().abs() + 1e-4).all()


@pytest.mark.parametrize("rows", [2000, 40000])
def test_1024_experts(rows):
    """The most experts there may be, many without rows; few rows and tiles."""
    need_gpu()
    E, N, K = 1024, 40, 96
    say("1024 experts", rows)
    rng = np.random.default_rng(rows)
    offsets = [3] + sorted(int(v) for v in rng.integers(3, rows - 5, E - 1)) + [rows - 5]
    a, ws = random_mx4(rng, rows, K), [random_mx4(rng, N, K) for _ in range(5)]
    ops = [operand(*w) for w in ws]
    which = [e % 5 for e in range(E)]
    out = torch.full((rows, N), 77.0, device="cuda")
    F.fp4_gemm_grouped(*grouped_operand(*a, rows, offsets), dev_offsets(offsets), torch.stack([ops[i][0] for i in which]),
                       torch.stack([ops[i][1] for i in which]), rows, out=out, out_dtype=F.OUT_F32)
    torch.cuda.synchronize()
    av, wv = values(*a), [values(*w) for w in ws]
    ref, mag = np.full((rows, N), 77.0), np.zeros((rows, N))
    for i, lo, hi in zip(which, offsets, offsets[1:]):
        ref[lo:hi], mag[lo:hi] = av[lo:hi] @ wv[i].T, np.abs(av[lo:hi]) @ np.abs(wv[i]).T
    check(out, ref, mag)
    dy, x, off = normal(rows, 32), normal(rows, 64, seed=1), dev_offsets(offsets)
    d, q = (F.fp4_quantize_grouped(t, off, F.AXIS_ROWS, 32, F.HAD_DET) for t in (dy, x))
    dw = F.fp4_gemm_grouped_wgrad(*d, *q, off, rows, out_dtype=F.OUT_F32)
    for e in (0, 500, E - 1):
        lo, hi = offsets[e], offsets[e + 1]
        if lo == hi:
            assert (dw[e] == 0).all()
            continue
        one = dev_offsets([0, hi - lo])
        d1, q1 = (F.fp4_quantize_grouped(t[lo:hi], one, F.AXIS_ROWS, 32, F.HAD_DET) for t in (dy, x))
        same(dw[e], F.fp4_gemm_grouped_wgrad(*d1, *q1, one, hi - lo, out_dtype=F.OUT_F32)[0])
