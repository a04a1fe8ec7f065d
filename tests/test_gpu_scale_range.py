"""MXFP8 activations times MXFP4 weights with scale bytes from one end of E8M0
to the other: elements that leave bf16's range although their products do not."""
import numpy as np
import pytest
import torch

import fp4_precision_gemms_amd as F
from _grouped import SPLITS, check, dev_offsets, operand, random_mx4, random_mx8, values
from _util import need_gpu, say

pytestmark = pytest.mark.gpu


def opposite(rng, a, w, low, high):
    """Scale bytes of each block of the contraction: the activations' next to a
    byte of [low, high], the weights' next to its opposite, so that every
    product is of the order of one."""
    nb = a[1].shape[1]
    mid = rng.integers(low, high + 1, nb)
    a[1][:] = np.clip(mid + rng.integers(-2, 3, a[1].shape), 0, 254)
    w[1][:] = np.clip(254 - mid + rng.integers(-2, 3, w[1].shape), 0, 254)


# every launch shape: 1, 2 and 4 row tiles, 1 and 2 weight tiles, 2, 4 and 8
# waves, a second pass over the rows, contractions that end inside a k-group
SHAPES = [(1, 40, 96), (16, 33, 256), (20, 48, 2080), (50, 35, 4128), (5, 16, 4096), (3, 8192, 288), (17, 8200, 2080),
          (40, 8192, 64), (70, 16, 512), (30, 24, 736)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("low,high", [(0, 4), (245, 254), (0, 254)])
@pytest.mark.parametrize("out_dtype", [F.OUT_BF16, F.OUT_F32])
def test_decode_over_the_whole_range_of_scales(M, N, K, low, high, out_dtype):
    need_gpu()
    say("scale range", M, N, K, low, high, out_dtype)
    rng = np.random.default_rng(M + N + K + low)
    a, w = random_mx8(rng, M, K), random_mx4(rng, N, K)
    opposite(rng, a, w, low, high)
    got = F.fp4_gemm_decode(*operand(*a), *operand(*w), out_dtype=out_dtype)
    torch.cuda.synchronize()
    av, wv = values(*a), values(*w)
    check(got, av @ wv.T, np.abs(av) @ np.abs(wv).T)


@pytest.mark.parametrize("split", ["odd", "outside", "long"])
def test_grouped_over_the_whole_range_of_scales(split):
    need_gpu()
    say("scale range grouped", split)
    rows, offsets = SPLITS[split]
    N, K, E = 72, 352, len(offsets) - 1
    rng = np.random.default_rng(rows)
    a, ws = random_mx8(rng, rows, K), [random_mx4(rng, N, K) for _ in range(E)]
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        opposite(rng, (a[0][lo:hi], a[1][lo:hi]), ws[e], 0, 254)
    ops = [operand(*w) for w in ws]
    out = torch.full((rows, N), 77.0, device="cuda")
    F.fp4_gemm_grouped(*operand(*a), dev_offsets(offsets), torch.stack([o[0] for o in ops]),
                       torch.stack([o[1] for o in ops]), rows, out=out, out_dtype=F.OUT_F32)
    torch.cuda.synchronize()
    av = values(*a)
    ref, mag = np.full((rows, N), 77.0), np.zeros((rows, N))
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        wv = values(*ws[e])
        ref[lo:hi], mag[lo:hi] = av[lo:hi] @ wv.T, np.abs(av[lo:hi]) @ np.abs(wv).T
    check(out, ref, mag)


@pytest.mark.parametrize("M,N,K", [(20, 33, 320), (3, 8192, 2080)])
def test_nan_scales_beside_scales_at_the_ends(M, N, K):
    """A NaN byte reaches its own row or column alone, zero blocks stay zero
    under any byte, and a sum that passes binary32 is infinite."""
    need_gpu()
    rng = np.random.default_rng(5)
    a, w = random_mx8(rng, M, K), random_mx4(rng, N, K)
    opposite(rng, a, w, 0, 254)
    a[1][0, 4] = 255
    w[1][7, 9] = 255
    a[0][1, :32] = 0
    a[1][1, 0], w[1][:, 0] = 254, 254
    got = F.fp4_gemm_decode(*operand(*a), *operand(*w), out_dtype=F.OUT_F32)
    torch.cuda.synchronize()
    g, av, wv = got.double().cpu().numpy(), values(*a), values(*w)
    ref, mag = av @ wv.T, np.abs(av) @ np.abs(wv).T
    assert np.isnan(g[0]).all() and np.isnan(g[:, 7]).all()
    keep = np.arange(N) != 7
    check(got[1:2, keep], ref[1:2, keep], mag[1:2, keep])
    large = np.abs(ref[2:, keep]) > 2.0 ** 130
    assert large.any() and np.isinf(g[2:, keep][large]).all()


@pytest.mark.parametrize("fmt", [F.FMT_MXFP8, F.FMT_MXFP4])
def test_nan_blocks_as_the_quantizers_write_them(fmt):
    """A NaN activation or weight leaves a block of zero codes under scale byte
    255: NaN in its row or column, nothing elsewhere."""
    need_gpu()
    M, N, K = 6, 96, 320
    g = torch.Generator(device="cuda").manual_seed(0)
    x, w = (torch.randn(n, K, device="cuda", generator=g).bfloat16() for n in (M, N))
    x[4, 77] = float("nan")
    w[33, 300] = float("-inf")
    a = F.fp4_rmsnorm_quantize(x, torch.ones(K, device="cuda").bfloat16(), fmt=fmt)[:2]
    y = F.fp4_gemm_decode(*a, *F.fp4_hadamard_quantize(w))
    torch.cuda.synchronize()
    want = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    want[4] = True
    want[:, 33] = True
    assert torch.equal(y.isnan(), want)
