"""The norm and the grouped quantizer on so many rows that a launch has 2^32
threads or more: rows from all over against a call of their own."""
import pytest
import torch

import fp4_precision_gemms_amd as F
from _grouped import dev_offsets
from _util import need_gpu, say

pytestmark = pytest.mark.gpu


def repeated(rows, cols, period, seed):
    """bf16 [rows, cols], normal values that come again every `period` rows."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    one = torch.randn(period, cols, device="cuda", generator=g).bfloat16()
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    whole = rows // period * period
    x[:whole].view(-1, period, cols).copy_(one.expand(whole // period, period, cols))
    x[whole:] = one[:rows - whole]
    return x


def blocks(scales, cols):
    """The scale bytes of the blocks there are, [rows, cols / 32]."""
    return scales.transpose(0, 1).flatten(1)[:, :cols // 32]


def same(a, b):
    assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("fmt", [F.FMT_MXFP8, F.FMT_MXFP4])
@pytest.mark.parametrize("rows,cols", [(2 ** 26 + 37, 32), (2 ** 25 + 37, 1056)])
def test_norm(fmt, rows, cols):
    """64 threads a row of up to 1024 columns, 128 of up to 2048."""
    need_gpu()
    say("norm of many rows", fmt, rows, cols)
    x, w = repeated(rows, cols, 4096, 0), repeated(1, cols, 1, 1)[0]
    codes, scales, h, rstd = F.fp4_rmsnorm_quantize(x, w, fmt=fmt)
    torch.cuda.synchronize()
    for lo in (0, rows // 2 // 32 * 32, (rows - 40) // 32 * 32):
        hi = min(lo + 64, rows)
        c, s, _, r = F.fp4_rmsnorm_quantize(x[lo:hi], w, fmt=fmt)
        same(rstd[lo:hi], r)
        if fmt == F.FMT_MXFP8:
            same(codes[lo:hi], c)
            same(scales[lo:hi], s)
        else:
            full = (hi - lo) // 32
            same(codes[lo // 32:lo // 32 + full], c[:full])
            same(blocks(scales[:, lo:hi], cols), blocks(s, cols))
    # each row gives what the first one of its kind gives
    whole = rows // 4096 * 4096
    assert (rstd[:whole].view(-1, 4096) == rstd[:4096]).all()


def test_quantize_grouped():
    need_gpu()
    rows, cols = 2 ** 30 + 4096, 32
    say("grouped quantizer of many rows")
    offsets = [0, 5, 2 ** 30 + 1000, rows - 3]
    x = repeated(rows, cols, 4096, 2)
    q, s = F.fp4_quantize_grouped(x, dev_offsets(offsets))
    torch.cuda.synchronize()
    for e, lo, hi in ((0, 0, 5), (1, 5 + 2 ** 29, 5 + 2 ** 29 + 64), (2, offsets[2], offsets[3])):
        q1, s1 = F.fp4_quantize_grouped(x[lo:hi], dev_offsets([0, hi - lo]))
        u = offsets[e] // 32 + e + (lo - offsets[e]) // 32
        n = (hi - lo) // 32
        same(q[u:u + n], q1[:n])
        same(blocks(s[:, 32 * u:32 * u + hi - lo], cols), blocks(s1[:, :hi - lo], cols))
