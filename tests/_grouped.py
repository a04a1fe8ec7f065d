"""Shared by the grouped tests: splits of rows over experts, the padded
layout, operands with every padding byte poisoned."""
import numpy as np
import torch

import _mx_ref as R
from _util import group_scales, tile_codes

TOL = 1e-5     # the GEMMs' bound: |err| <= 1e-5 sum |a b|

# name -> (rows, offsets): empty experts first, last and between, one row,
# units that end inside a tile, rows of no expert before and behind
SPLITS = {
    "one": (1, [0, 1]),
    "one of four": (3, [0, 0, 3, 3, 3]),
    "odd": (200, [0, 1, 34, 34, 66, 130, 199, 200]),
    "aligned": (256, [0, 64, 96, 256]),
    "outside": (150, [5, 5, 40, 41, 120]),
    "none": (40, [7, 7, 7]),
    "long": (700, [0, 300, 301, 301, 633, 700]),
    "many": (333, sorted(int(v) for v in np.random.default_rng(4).integers(0, 334, 99))),
}
SPLITS["many"] = (333, [0] + SPLITS["many"][1] + [333])


def dev_offsets(offsets):
    return torch.tensor(offsets, dtype=torch.int32, device="cuda")


def padded_rows(rows, offsets):
    """Row of the padded layout of each row of x, -1 for rows of no expert;
    number of units."""
    at = np.full(rows, -1)
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        at[lo:hi] = 32 * (lo // 32 + e) + np.arange(hi - lo)
    return at, rows // 32 + len(offsets) - 1


def staged_rows(rows, offsets):
    """Element of the rows output's contraction of each row of x, -1 for rows
    of no expert; number of stages; the stages that are written."""
    at = np.full(rows, -1)
    used = []
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        first = lo // 256 + e
        at[lo:hi] = 256 * first + np.arange(hi - lo)
        used += range(first, first + (hi - lo + 255) // 256)
    return at, rows // 256 + len(offsets) - 1, used


def random_mx4(rng, rows, K, low=117, high=127):
    codes = rng.integers(0, 256, (rows, K // 2), dtype=np.uint8)
    return codes, rng.integers(low, high, (rows, K // 32), dtype=np.uint8)


def random_mx8(rng, rows, K, low=110, high=122):
    codes = rng.integers(0, 127, (rows, K), dtype=np.uint8) | (rng.integers(0, 2, (rows, K), dtype=np.uint8) << 7)
    return codes, rng.integers(low, high, (rows, K // 32), dtype=np.uint8)


def values(codes, scales):
    return R.mxfp8_values(codes, scales) if codes.shape[1] == 32 * scales.shape[1] else R.mxfp4_values(codes, scales)


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def operand(codes, scales):
    """On the GPU in the library's layout, padding rows 0xFF (-6) and padding
    scale bytes 0xFF (NaN)."""
    if codes.shape[1] == 32 * scales.shape[1]:
        return gpu(codes), gpu(scales)
    return gpu(tile_codes(codes, 0xFF)), gpu(group_scales(scales))


def grouped_operand(codes, scales, rows, offsets):
    """MXFP4 rows in the grouped layout along cols."""
    at, units = padded_rows(rows, offsets)
    c = np.full((32 * units, codes.shape[1]), 0xFF, np.uint8)
    s = np.full((32 * units, scales.shape[1]), 0xFF, np.uint8)
    c[at[at >= 0]], s[at[at >= 0]] = codes[at >= 0], scales[at >= 0]
    return operand(c, s)


def check(got, ref, mag):
    """got against the 64-bit product within the GEMM bound, and half a step
    more for bf16; NaN exactly where ref is NaN."""
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    g = got.double().cpu().numpy()
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(g), nan), "NaN pattern differs"
    near = TOL * mag
    near = near + half * (np.abs(ref) + near)
    bad = np.abs(g - ref)[~nan] > near[~nan]
    assert not bad.any(), "%d of %d out of bound" % (bad.sum(), bad.size)
