"""fp4_gemm_decode and fp4_gemm_grouped of few rows against the 64-bit product
of the dequantized operands."""
import numpy as np
import pytest
import torch

import fp4_precision_gemms_amd as F
from _grouped import (SPLITS, check, dev_offsets, gpu, grouped_operand, operand, random_mx4, random_mx8, values)
from _util import need_gpu, say

pytestmark = pytest.mark.gpu

RANDOM = {F.FMT_MXFP8: random_mx8, F.FMT_MXFP4: random_mx4}


@pytest.mark.parametrize("fmt", [F.FMT_MXFP8, F.FMT_MXFP4])
@pytest.mark.parametrize("out_dtype", [F.OUT_BF16, F.OUT_F32])
@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 4096, 4096), (2, 3, 64), (5, 16, 96), (15, 30, 256), (16, 64, 288),
                                   (17, 100, 1024), (31, 258, 224), (32, 48, 2080), (33, 72, 2336), (48, 515, 512),
                                   (64, 112, 4128), (65, 40, 160), (130, 96, 8224), (3, 32, 16416)])
def test_decode(M, N, K, fmt, out_dtype):
    need_gpu()
    say("decode", M, N, K, fmt, out_dtype)
    rng = np.random.default_rng(M + 3 * N + 5 * K)
    a, w = RANDOM[fmt](rng, M, K), random_mx4(rng, N, K)
    got = F.fp4_gemm_decode(*operand(*a), *operand(*w), out_dtype=out_dtype)
    torch.cuda.synchronize()
    av, wv = values(*a), values(*w)
    check(got, av @ wv.T, np.abs(av) @ np.abs(wv).T)


def test_decode_element_by_element():
    """One nonzero element of A and of W at a time, at every k of two k-groups:
    each product lands alone, so a wrong position in k shows."""
    need_gpu()
    K = 512
    rng = np.random.default_rng(0)
    wc = rng.integers(1, 8, (K, K // 2), dtype=np.uint8) * 0                # W = identity: 1.0 is code 2
    wc[np.arange(K), np.arange(K) // 2] = np.where(np.arange(K) % 2, 0x20, 0x02)
    ws = rng.integers(120, 135, (K, K // 32), dtype=np.uint8)
    a = random_mx8(rng, 16, K)
    got = F.fp4_gemm_decode(*operand(*a), *operand(wc, ws), out_dtype=F.OUT_F32)
    b = random_mx4(rng, 16, K)
    got4 = F.fp4_gemm_decode(*operand(*b), *operand(wc, ws), out_dtype=F.OUT_F32)
    torch.cuda.synchronize()
    diag = values(wc, ws).diagonal()
    assert np.array_equal(got.double().cpu().numpy(), values(*a) * diag)
    assert np.array_equal(got4.double().cpu().numpy(), values(*b) * diag)


@pytest.mark.parametrize("fmt", [F.FMT_MXFP8, F.FMT_MXFP4])
def test_decode_nan_scales_and_zero_rows(fmt):
    need_gpu()
    M, N, K = 20, 33, 320
    rng = np.random.default_rng(2)
    a, w = RANDOM[fmt](rng, M, K), random_mx4(rng, N, K)
    a[1][3, 4] = 255
    w[1][7, 9] = 255
    a[0][5] = 0
    got = F.fp4_gemm_decode(*operand(*a), *operand(*w), out_dtype=F.OUT_F32)
    torch.cuda.synchronize()
    av, wv = values(*a), values(*w)
    check(got, av @ wv.T, np.abs(av) @ np.abs(wv).T)
    assert not got[5].nan_to_num().any()


def test_decode_agrees_with_the_large_product():
    """The same MXFP4 operands through fp4_gemm_mx."""
    need_gpu()
    rng = np.random.default_rng(9)
    a, w = random_mx4(rng, 48, 1024), random_mx4(rng, 320, 1024)
    ga, gw = operand(*a), operand(*w)
    one, two = F.fp4_gemm_decode(*ga, *gw, out_dtype=F.OUT_F32), F.fp4_gemm_mx(*ga, *gw)
    torch.cuda.synchronize()
    mag = np.abs(values(*a)) @ np.abs(values(*w)).T
    assert (np.abs((one - two).double().cpu().numpy()) <= 2e-5 * mag).all()


def stack(ws):
    ops = [operand(*w) for w in ws]
    return torch.stack([o[0] for o in ops]), torch.stack([o[1] for o in ops])


@pytest.mark.parametrize("split", list(SPLITS))
@pytest.mark.parametrize("fmt", [F.FMT_MXFP8, F.FMT_MXFP4])
@pytest.mark.parametrize("N,K,out_dtype", [(48, 256, F.OUT_BF16), (35, 352, F.OUT_F32)])
def test_grouped(split, fmt, N, K, out_dtype):
    need_gpu()
    rows, offsets = SPLITS[split]
    say("grouped", split, fmt, N, K)
    rng = np.random.default_rng(rows + N)
    E = len(offsets) - 1
    a, ws = RANDOM[fmt](rng, rows, K), [random_mx4(rng, N, K) for _ in range(E)]
    ga = operand(*a) if fmt == F.FMT_MXFP8 else grouped_operand(*a, rows, offsets)
    out = torch.full((rows, N), 77.0, dtype=torch.bfloat16 if out_dtype == F.OUT_BF16 else torch.float32, device="cuda")
    got = F.fp4_gemm_grouped(*ga, dev_offsets(offsets), *stack(ws), rows, out=out, out_dtype=out_dtype)
    torch.cuda.synchronize()
    assert got is out
    av = values(*a)
    ref, mag = np.full((rows, N), 77.0), np.zeros((rows, N))
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        wv = values(*ws[e])
        ref[lo:hi], mag[lo:hi] = av[lo:hi] @ wv.T, np.abs(av[lo:hi]) @ np.abs(wv).T
    check(got, ref, mag)
    outside = np.r_[0:offsets[0], offsets[-1]:rows]
    assert (got.float().cpu().numpy()[outside] == 77.0).all()


def test_decode_on_a_side_stream_and_in_a_graph():
    """A captured decode step (norm, product) replayed with new inputs in the
    same buffers, eager work between the replays."""
    need_gpu()
    from _mx_ref import to_bf16
    rows, K, N = 3, 1024, 512
    rng = np.random.default_rng(6)
    w = operand(*random_mx4(rng, N, K))
    x, r = (torch.from_numpy(to_bf16(rng.standard_normal((rows, K)))).bfloat16().cuda() for _ in range(2))
    g = torch.ones(K, dtype=torch.bfloat16, device="cuda")

    def step():
        codes, scales, h, _ = F.fp4_rmsnorm_quantize(x, g, r)
        return h, F.fp4_gemm_decode(codes, scales, *w)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = step()
    for i in range(3):
        x.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(caught, want):
            assert torch.equal(a, b), i


def test_two_streams_at_once():
    """Two grouped products on two streams share no state."""
    need_gpu()
    rows, offsets = SPLITS["odd"]
    rng = np.random.default_rng(1)
    N, K = 64, 512
    a = random_mx8(rng, rows, K)
    st = stack([random_mx4(rng, N, K) for _ in range(len(offsets) - 1)])
    ga, off = operand(*a), dev_offsets(offsets)
    want = F.fp4_gemm_grouped(*ga, off, *st, rows)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(want) for _ in range(2)]
    for _ in range(5):
        for s, o in zip(streams, outs):
            F.fp4_gemm_grouped(*ga, off, *st, rows, out=o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
