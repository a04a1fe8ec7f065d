"""The few-row kernel where an expert has more rows than a row tile: tiles that
several workgroups share, and experts with more of them than the average."""
import numpy as np
import pytest
import torch

import fp4_precision_gemms_amd as F
from _grouped import check, dev_offsets, grouped_operand, operand, random_mx4, random_mx8, values
from _util import need_gpu, say

pytestmark = pytest.mark.gpu

# one row tile past the end, the rows of all but one expert few, rows outside
SPLITS = {"one": (700, [0, 700]), "one more": (513, [0, 513]), "skewed": (650, [0, 3, 3, 640, 645, 650]),
          "first": (1300, [0, 1290, 1295, 1300]), "outside": (400, [30, 30, 385, 390])}


@pytest.mark.parametrize("split", list(SPLITS))
@pytest.mark.parametrize("fmt", [F.FMT_MXFP8, F.FMT_MXFP4])
@pytest.mark.parametrize("N,K,out_dtype", [(35, 352, F.OUT_F32), (64, 2112, F.OUT_BF16), (130, 4160, F.OUT_F32)])
def test_grouped(split, fmt, N, K, out_dtype):
    need_gpu()
    rows, offsets = SPLITS[split]
    say("few-row kernel, many rows", split, fmt, N, K)
    rng = np.random.default_rng(rows + N)
    E = len(offsets) - 1
    a, ws = (random_mx8 if fmt == F.FMT_MXFP8 else random_mx4)(rng, rows, K), [random_mx4(rng, N, K) for _ in range(E)]
    ga = operand(*a) if fmt == F.FMT_MXFP8 else grouped_operand(*a, rows, offsets)
    ops = [operand(*w) for w in ws]
    out = torch.full((rows, N), 77.0, dtype=torch.bfloat16 if out_dtype == F.OUT_BF16 else torch.float32, device="cuda")
    F.fp4_gemm_grouped(*ga, dev_offsets(offsets), torch.stack([o[0] for o in ops]), torch.stack([o[1] for o in ops]),
                       rows, out=out, out_dtype=out_dtype)
    torch.cuda.synchronize()
    av = values(*a)
    ref, mag = np.full((rows, N), 77.0), np.zeros((rows, N))
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        wv = values(*ws[e])
        ref[lo:hi], mag[lo:hi] = av[lo:hi] @ wv.T, np.abs(av[lo:hi]) @ np.abs(wv).T
    check(out, ref, mag)


@pytest.mark.parametrize("fmt", [F.FMT_MXFP8, F.FMT_MXFP4])
@pytest.mark.parametrize("M,N,K", [(300, 20, 2080), (1000, 96, 4128), (129, 4104, 96)])
def test_decode(M, N, K, fmt):
    need_gpu()
    say("few-row kernel, many rows", M, N, K, fmt)
    rng = np.random.default_rng(M)
    a, w = (random_mx8 if fmt == F.FMT_MXFP8 else random_mx4)(rng, M, K), random_mx4(rng, N, K)
    got = F.fp4_gemm_decode(*operand(*a), *operand(*w), out_dtype=F.OUT_F32)
    torch.cuda.synchronize()
    av, wv = values(*a), values(*w)
    check(got, av @ wv.T, np.abs(av) @ np.abs(wv).T)
