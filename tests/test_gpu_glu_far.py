"""The gated activation on inputs beyond the last-level cache, whose kernels access
memory non-temporally: the same bits as the same rows in a small call, rows of no
expert as they were."""
import pytest
import torch

import fp4_precision_gemms_amd as F
from _util import need_gpu, say

pytestmark = pytest.mark.gpu

# a wave a row of the gradient (by width, by rows), 256 threads, 1024
SIZES = [(70000, 1024), (40000, 1760), (17000, 4096), (8200, 8224)]
SOME = 1100                    # as many rows that the small call shares the threads of a row


def tiled_rows(codes, rows):
    """MXFP4 codes [ceil(R/32), C/32, 512] as [R, C/32, 16]."""
    n, nb, _ = codes.shape
    return codes.view(n, nb, 32, 16).permute(0, 2, 1, 3).reshape(n * 32, nb, 16)[:rows]


def grouped_scales(scales, rows, nb):
    return scales.permute(1, 0, 2).reshape(rows, -1)[:, :nb]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("act", [F.ACT_SILU, F.ACT_GELU])
def test_far_rows_as_near_ones(rows, cols, act):
    need_gpu()
    say("glu far", rows, cols, act)
    assert 4 * rows * cols >= 2 ** 28 > 4 * SOME * cols
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, 2 * cols, device="cuda", generator=g).bfloat16()
    w = torch.randn(rows, device="cuda", generator=g)
    order = torch.randperm(rows, device="cuda", generator=g).int()
    lo, hi = 5, rows - 37
    off = torch.tensor([lo, rows // 3, rows // 3, hi], dtype=torch.int32, device="cuda")
    at = (lo + torch.randperm(hi - lo, device="cuda", generator=g)[:SOME - 2]).tolist() + [lo, hi - 1]
    at = torch.tensor(sorted(set(at)), device="cuda")
    dead = torch.ones(rows, dtype=torch.bool, device="cuda")
    dead[lo:hi] = False
    small, by_row = x[at].contiguous(), w[order[at].long()].contiguous()
    nb, n = cols // 32, len(at)

    def kept(outs):
        return [torch.full_like(t, 7) for t in outs]

    # bf16 with the checkpoint, and without weights
    want = F.fp4_glu(small, act, by_row, checkpoint=True)
    got = kept(F.fp4_glu(x, act, checkpoint=True))
    assert torch.equal(F.fp4_glu(x, act)[at], F.fp4_glu(small, act))
    F.fp4_glu(x, act, w, order, off, checkpoint=True, out=got)
    for a, b in zip(got, want):
        assert torch.equal(a[at], b) and (a[dead] == 7).all()
    # MXFP8
    want8 = F.fp4_glu_quantize(small, act, by_row)
    got8 = kept(F.fp4_glu_quantize(x, act))
    F.fp4_glu_quantize(x, act, w, order, off, out=got8)
    for a, b in zip(got8, want8):
        assert torch.equal(a[at], b) and (a[dead] == 7).all()
    # MXFP4
    want4 = F.fp4_glu_quantize(small, act, by_row, fmt=F.FMT_MXFP4)
    got4 = kept(F.fp4_glu_quantize(x, act, fmt=F.FMT_MXFP4))
    F.fp4_glu_quantize(x, act, w, order, off, F.FMT_MXFP4, out=got4)
    codes = tiled_rows(got4[0], rows)
    assert torch.equal(codes[at], tiled_rows(want4[0], n)) and (codes[dead] == 7).all()
    scales = grouped_scales(got4[1], rows, nb)
    assert torch.equal(scales[at], grouped_scales(want4[1], n, nb)) and (scales[dead] == 7).all()
    # the gradient, with the weights' and without
    _, xq, xs = F.fp4_glu(x, act, checkpoint=True)
    dy = torch.randn(rows, cols, device="cuda", generator=g).bfloat16()
    dy_small, q, s = dy[at].contiguous(), xq[at].contiguous(), xs[at].contiguous()
    dx, dw = F.fp4_glu_backward(dy_small, q, s, act, by_row)
    out = kept((x, w))
    F.fp4_glu_backward(dy, xq, xs, act, w, order, off, out=out)
    assert torch.equal(out[0][at], dx) and (out[0][dead] == 7).all()
    assert torch.equal(out[1][order[at].long()], dw) and not out[1][order[dead].long()].any()
    assert torch.equal(F.fp4_glu_backward(dy, xq, xs, act)[at], F.fp4_glu_backward(dy_small, q, s, act))
