"""fp4_quantize_grouped bit for bit against the oracle on the padded layout:
the experts' rows at their units, zeros between them."""
import numpy as np
import pytest
import torch

import fp4_precision_gemms_amd as F
import oracle as O
from _grouped import SPLITS, dev_offsets, padded_rows, staged_rows
from _util import bf16_bits, need_gpu, say, sentinel_u8, to_gpu_bf16, ungroup_scales, untile_codes

pytestmark = pytest.mark.gpu

MODES = {"plain": (32, F.HAD_NONE, 0, F.RTN), "had32": (32, F.HAD_DET, 0, F.RTN),
         "had16 signed": (16, F.HAD_SIGNED, 99, F.RTN), "sr": (32, F.HAD_NONE, 0, F.SR),
         "had16 sr": (16, F.HAD_DET, 0, F.SR), "had32 sr": (32, F.HAD_SIGNED, 5, F.SR)}


def check_rows(codes, scales, bits, rows, offsets, mode, seed):
    """Every written byte of the rows output; every other byte still 0xCD."""
    had_n, had, sign_seed, rnd = mode
    at, stages, used = staged_rows(rows, offsets)
    C = bits.shape[1]
    full = np.zeros((256 * stages, C), np.uint16)
    full[at[at >= 0]] = bits[at >= 0]
    rc, rs = O.quant_mx(full, O.AXIS_ROWS, had_n, had, sign_seed, rnd, seed)
    want = np.full((C, stages, 128), 0xCD, np.uint8)
    want[:, used] = rc.reshape(C, stages, 128)[:, used]
    assert np.array_equal(untile_codes(codes.cpu().numpy(), C).reshape(C, stages, 128), want)
    ws = np.full((C, stages, 8), 0xCD, np.uint8)
    ws[:, used] = rs.reshape(C, stages, 8)[:, used]
    assert np.array_equal(scales.cpu().numpy(), ws.transpose(1, 0, 2))


def check_cols(codes, scales, bits, rows, offsets, mode, seed):
    had_n, had, sign_seed, rnd = mode
    at, units = padded_rows(rows, offsets)
    rc, rs = O.quant_mx(bits, O.AXIS_COLS, had_n, had, sign_seed, rnd, seed)
    nb = bits.shape[1] // 32
    want, ws = np.full((32 * units, 16 * nb), 0xCD, np.uint8), np.full((32 * units, nb), 0xCD, np.uint8)
    want[at[at >= 0]], ws[at[at >= 0]] = rc[at >= 0], rs[at >= 0]
    assert np.array_equal(untile_codes(codes.cpu().numpy(), 32 * units), want)
    assert np.array_equal(ungroup_scales(scales.cpu().numpy(), nb), ws)


def out(rows, cols, E, *axes):
    return [sentinel_u8(s) for a in axes for s in F.grouped_shapes(rows, cols, E, a)]


@pytest.mark.parametrize("split", list(SPLITS))
@pytest.mark.parametrize("mode", list(MODES))
def test_grouped_quantizers(split, mode):
    need_gpu()
    rows, offsets = SPLITS[split]
    E, m = len(offsets) - 1, MODES[mode]
    for cols in (32, 288):
        say("quantize grouped", split, mode, cols)
        rng = np.random.default_rng(rows + cols)
        bits = bf16_bits(rng.standard_t(4, (rows, cols)))
        x, off = to_gpu_bf16(bits), dev_offsets(offsets)
        got = F.fp4_quantize_grouped(x, off, F.AXIS_ROWS, *m, sr_seed=11, out=out(rows, cols, E, F.AXIS_ROWS))
        torch.cuda.synchronize()
        check_rows(*got, bits, rows, offsets, m, 11)
        got = F.fp4_quantize_grouped(x, off, F.AXIS_COLS, *m, sr_seed=12, out=out(rows, cols, E, F.AXIS_COLS))
        torch.cuda.synchronize()
        check_cols(*got, bits, rows, offsets, m, 12)
        got = F.fp4_quantize_grouped_dual(x, off, *m, sr_seed_rows=13, sr_seed_cols=14,
                                          out=out(rows, cols, E, F.AXIS_ROWS, F.AXIS_COLS))
        torch.cuda.synchronize()
        check_rows(*got[:2], bits, rows, offsets, m, 13)
        check_cols(*got[2:], bits, rows, offsets, (32, F.HAD_NONE, 0, m[3]), 14)


# two units per workgroup; with mostly short experts a stage per workgroup
WIDE = {"two units": (5000, [7, 7, 2600, 4991], 3104), "stages": (*SPLITS["many"], 1312),
        "stages of some": (400, [2] + [2 + 9 * i for i in range(30)] + [300] * 60 + [398], 1600)}


@pytest.mark.parametrize("split", list(WIDE))
@pytest.mark.parametrize("mode", ["had16 signed", "had32 sr"])
def test_grouped_quantizers_of_wide_tensors(split, mode):
    need_gpu()
    rows, offsets, cols = WIDE[split]
    E, m = len(offsets) - 1, MODES[mode]
    say("quantize grouped, wide", split, mode)
    bits = bf16_bits(np.random.default_rng(cols).standard_t(4, (rows, cols)))
    x, off = to_gpu_bf16(bits), dev_offsets(offsets)
    got = F.fp4_quantize_grouped(x, off, F.AXIS_ROWS, *m, sr_seed=11, out=out(rows, cols, E, F.AXIS_ROWS))
    both = F.fp4_quantize_grouped_dual(x, off, *m, sr_seed_rows=11, sr_seed_cols=14,
                                       out=out(rows, cols, E, F.AXIS_ROWS, F.AXIS_COLS))
    cols_only = F.fp4_quantize_grouped(x, off, F.AXIS_COLS, 32, F.HAD_NONE, 0, m[3], sr_seed=14,
                                       out=out(rows, cols, E, F.AXIS_COLS))
    torch.cuda.synchronize()
    check_rows(*got, bits, rows, offsets, m, 11)
    check_cols(*cols_only, bits, rows, offsets, (32, F.HAD_NONE, 0, m[3]), 14)
    for a, b in zip(both, (*got, *cols_only)):
        assert torch.equal(a, b)


def test_non_finite_values():
    need_gpu()
    rows, offsets = SPLITS["odd"]
    rng = np.random.default_rng(0)
    v = rng.standard_normal((rows, 64)).astype(np.float32)
    v[3, 5], v[40, 33], v[150] = np.nan, np.inf, 0
    bits = bf16_bits(v)
    m = MODES["plain"]
    got = F.fp4_quantize_grouped_dual(to_gpu_bf16(bits), dev_offsets(offsets),
                                      out=out(rows, 64, len(offsets) - 1, F.AXIS_ROWS, F.AXIS_COLS))
    torch.cuda.synchronize()
    check_rows(*got[:2], bits, rows, offsets, m, 0)
    check_cols(*got[2:], bits, rows, offsets, m, 0)
