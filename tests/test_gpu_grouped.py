"""Grouped products with many rows per expert and the grouped weight gradient
against 64-bit products of the dequantized operands, every byte that belongs
to no row poisoned; the autograd layer built on them."""
import numpy as np
import pytest
import torch

import fp4_precision_gemms_amd as F
import oracle as O
from _grouped import SPLITS, check, dev_offsets, grouped_operand, operand, random_mx4, staged_rows, values
from _mx_ref import mxfp4_values
from _util import bf16_bits, need_gpu, say, to_gpu_bf16

pytestmark = pytest.mark.gpu

# over 64 rows an expert on average: the large tiles
MANY = {"long": SPLITS["long"], "big": (1500, [0, 700, 701, 701, 1213, 1470]), "first": (600, [0, 600, 600]),
        "last": (1025, [0, 0, 0, 1025]), "exact": (1024, [0, 256, 768, 1024]), "uneven": (900, [3, 300, 812, 880]),
        "seventy": (2900, [0] + sorted(int(v) for v in np.random.default_rng(8).integers(0, 2901, 69)) + [2900])}
# enough tiles for 256 rows each, and over 512 rows an expert for the large
# tiles of the weight gradient: 0, 1, 3, 4, 6 and 8 stages
LARGE = {"two": (4000, [0, 2500, 3990]), "stages": (3700, [0, 1024, 1725, 2982, 3700]),
         "empty": (2600, [0, 1999, 1999, 2600]), "one more": (1200, [0, 1, 1200])}


@pytest.mark.parametrize("split", list(MANY))
@pytest.mark.parametrize("N,K", [(256, 1024), (512, 2048), (300, 512), (1030, 256), (96, 288), (258, 1056), (256, 1280)])
@pytest.mark.parametrize("out_dtype", [F.OUT_BF16, F.OUT_F32])
def test_many_rows(split, N, K, out_dtype):
    need_gpu()
    rows, offsets = MANY[split]
    E = len(offsets) - 1
    say("grouped large", split, N, K, out_dtype)
    rng = np.random.default_rng(rows + N + K)
    a, ws = random_mx4(rng, rows, K), [random_mx4(rng, N, K) for _ in range(E)]
    ops = [operand(*w) for w in ws]
    out = torch.full((rows, N), 77.0, dtype=torch.bfloat16 if out_dtype == F.OUT_BF16 else torch.float32, device="cuda")
    F.fp4_gemm_grouped(*grouped_operand(*a, rows, offsets), dev_offsets(offsets), torch.stack([o[0] for o in ops]),
                       torch.stack([o[1] for o in ops]), rows, out=out, out_dtype=out_dtype)
    torch.cuda.synchronize()
    av = values(*a)
    ref, mag = np.full((rows, N), 77.0), np.zeros((rows, N))
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        wv = values(*ws[e])
        ref[lo:hi], mag[lo:hi] = av[lo:hi] @ wv.T, np.abs(av[lo:hi]) @ np.abs(wv).T
    check(out, ref, mag)
    outside = np.r_[0:offsets[0], offsets[-1]:rows]
    assert (out.float().cpu().numpy()[outside] == 77.0).all()


@pytest.mark.parametrize("split", list(LARGE))
@pytest.mark.parametrize("N,K,out_dtype", [(2560, 288, F.OUT_BF16), (2568, 1056, F.OUT_F32), (2680, 1280, F.OUT_BF16)])
def test_many_rows_large_tiles(split, N, K, out_dtype):
    need_gpu()
    rows, offsets = LARGE[split]
    E = len(offsets) - 1
    say("grouped 256-row tiles", split, N, K, out_dtype)
    rng = np.random.default_rng(rows + N)
    a, ws = random_mx4(rng, rows, K), [random_mx4(rng, N, K) for _ in range(E)]
    ops = [operand(*w) for w in ws]
    out = torch.full((rows, N), 77.0, dtype=torch.bfloat16 if out_dtype == F.OUT_BF16 else torch.float32, device="cuda")
    F.fp4_gemm_grouped(*grouped_operand(*a, rows, offsets), dev_offsets(offsets), torch.stack([o[0] for o in ops]),
                       torch.stack([o[1] for o in ops]), rows, out=out, out_dtype=out_dtype)
    torch.cuda.synchronize()
    av = values(*a)
    ref, mag = np.full((rows, N), 77.0), np.zeros((rows, N))
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        wv = values(*ws[e])
        ref[lo:hi], mag[lo:hi] = av[lo:hi] @ wv.T, np.abs(av[lo:hi]) @ np.abs(wv).T
    check(out, ref, mag)


@pytest.mark.parametrize("split,N", [("uneven", 304), ("uneven", 1304), ("seventy", 304), ("empty", 2560)])
@pytest.mark.parametrize("K", [64, 480, 736, 1024, 1120, 1408, 1760, 2048, 2784])
def test_many_rows_of_each_contraction(split, N, K):
    """1 to 8 and 11 stages of 256 elements, in the few-row kernel, the 128-row
    tiles and the 256-row tiles."""
    need_gpu()
    rows, offsets = {**MANY, **LARGE}[split]
    E = len(offsets) - 1
    say("grouped contraction", split, N, K)
    rng = np.random.default_rng(rows + K)
    a, ws = random_mx4(rng, rows, K), [random_mx4(rng, N, K) for _ in range(min(E, 3))]
    ops = [operand(*w) for w in ws]
    which = [e % len(ws) for e in range(E)]
    out = F.fp4_gemm_grouped(*grouped_operand(*a, rows, offsets), dev_offsets(offsets),
                             torch.stack([ops[i][0] for i in which]), torch.stack([ops[i][1] for i in which]), rows,
                             out=torch.full((rows, N), 77.0, device="cuda"), out_dtype=F.OUT_F32)
    torch.cuda.synchronize()
    av, wv = values(*a), [values(*w) for w in ws]
    ref, mag = np.full((rows, N), 77.0), np.zeros((rows, N))
    for i, lo, hi in zip(which, offsets, offsets[1:]):
        ref[lo:hi], mag[lo:hi] = av[lo:hi] @ wv[i].T, np.abs(av[lo:hi]) @ np.abs(wv[i]).T
    check(out, ref, mag)


@pytest.mark.parametrize("split", ["odd", "uneven", "two"])
def test_nan_blocks_stay_in_their_rows(split):
    """A NaN scale in one row of A, in one weight row of one expert, and a NaN
    token in the weight gradient's operands reach their own outputs alone."""
    need_gpu()
    rows, offsets = {**SPLITS, **MANY, **LARGE}[split]
    E, N, K = len(offsets) - 1, 320, 544
    say("grouped NaN", split)
    rng = np.random.default_rng(1)
    a, ws = random_mx4(rng, rows, K), [random_mx4(rng, N, K) for _ in range(E)]
    first = next(e for e in range(E) if offsets[e + 1] > offsets[e])
    a[1][offsets[first], 16] = 255                           # the last block of a row
    ws[E - 1][1][33, 0] = 255
    ops = [operand(*w) for w in ws]
    out = torch.zeros(rows, N, device="cuda")
    F.fp4_gemm_grouped(*grouped_operand(*a, rows, offsets), dev_offsets(offsets), torch.stack([o[0] for o in ops]),
                       torch.stack([o[1] for o in ops]), rows, out=out, out_dtype=F.OUT_F32)
    torch.cuda.synchronize()
    av = values(*a)
    ref, mag = np.zeros((rows, N)), np.zeros((rows, N))
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        wv = values(*ws[e])
        ref[lo:hi], mag[lo:hi] = av[lo:hi] @ wv.T, np.abs(av[lo:hi]) @ np.abs(wv).T
    check(out, ref, mag)
    v = rng.standard_normal((rows, N)).astype(np.float32)
    v[offsets[first], 5], v[offsets[first + 1] - 1, 40] = np.nan, np.inf
    dy, x = bf16_bits(v), bf16_bits(rng.standard_normal((rows, K)))
    qdy, vdy = quantized_rows(dy, rows, offsets, 32, F.HAD_NONE, 0)
    qx, vx = quantized_rows(x, rows, offsets, 32, F.HAD_NONE, 0)
    got = F.fp4_gemm_grouped_wgrad(*qdy, *qx, dev_offsets(offsets), rows, out_dtype=F.OUT_F32)
    torch.cuda.synchronize()
    ref, mag = np.zeros((E, N, K)), np.zeros((E, N, K))
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        span = slice(256 * (lo // 256 + e), 256 * (lo // 256 + e) + hi - lo + (lo - hi) % 32)
        ref[e], mag[e] = vdy[:, span] @ vx[:, span].T, np.abs(vdy[:, span]) @ np.abs(vx[:, span]).T
    assert np.isnan(ref[first, 5]).all()
    check(got, ref, mag)


def quantized_rows(bits, rows, offsets, had_n, had, seed, rnd=F.RTN, sr=0):
    """(GPU codes and scales, with every byte that is not written 0xFF; the
    oracle's values [C, 256 stages])."""
    E = len(offsets) - 1
    out = [torch.full(s, 0xFF, dtype=torch.uint8, device="cuda")
           for s in F.grouped_shapes(rows, bits.shape[1], E, F.AXIS_ROWS)]
    q = F.fp4_quantize_grouped(to_gpu_bf16(bits), dev_offsets(offsets), F.AXIS_ROWS, had_n, had, seed, rnd, sr, out=out)
    at, stages, _ = staged_rows(rows, offsets)
    full = np.zeros((256 * stages, bits.shape[1]), np.uint16)
    full[at[at >= 0]] = bits[at >= 0]
    return q, mxfp4_values(*O.quant_mx(full, O.AXIS_ROWS, had_n, had, seed, rnd, sr))


@pytest.mark.parametrize("split", list(SPLITS) + ["big", "exact"] + list(LARGE))
@pytest.mark.parametrize("N,K", [(32, 64), (256, 256), (288, 512), (544, 320)])
@pytest.mark.parametrize("out_dtype", [F.OUT_BF16, F.OUT_F32])
def test_wgrad(split, N, K, out_dtype):
    need_gpu()
    rows, offsets = {**SPLITS, **MANY, **LARGE}[split]
    E = len(offsets) - 1
    say("grouped wgrad", split, N, K, out_dtype)
    rng = np.random.default_rng(rows + N + K)
    dy, x = bf16_bits(rng.standard_normal((rows, N)) * 1e-3), bf16_bits(rng.standard_normal((rows, K)))
    qdy, vdy = quantized_rows(dy, rows, offsets, 32, F.HAD_DET, 0)
    qx, vx = quantized_rows(x, rows, offsets, 32, F.HAD_DET, 0)
    got = F.fp4_gemm_grouped_wgrad(*qdy, *qx, dev_offsets(offsets), rows, out_dtype=out_dtype)
    torch.cuda.synchronize()
    ref, mag = np.zeros((E, N, K)), np.zeros((E, N, K))
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        span = slice(256 * (lo // 256 + e), 256 * (lo // 256 + e) + hi - lo + (lo - hi) % 32)
        ref[e], mag[e] = vdy[:, span] @ vx[:, span].T, np.abs(vdy[:, span]) @ np.abs(vx[:, span]).T
    check(got, ref, mag)
