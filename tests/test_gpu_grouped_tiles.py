"""The tile kernels of the grouped product and of the weight gradient against
64-bit products: several tiles a workgroup (the next tile's first stages load
while the last one's output is stored), small outputs, NaN blocks, and a
captured graph replayed with other offsets."""
import numpy as np
import pytest
import torch

import fp4_precision_gemms_amd as F
from _grouped import TOL, dev_offsets, grouped_operand, operand, random_mx4, values
from _util import bf16_bits, need_gpu, say
from test_gpu_grouped import MANY, quantized_rows

pytestmark = pytest.mark.gpu


def ragged(rows, experts, seed):
    """Offsets of experts of uneven length, the second and the last empty."""
    c = sorted(int(v) for v in np.random.default_rng(seed).integers(0, rows + 1, experts - 3))
    c = [0] + c + [rows]
    return c[:2] + c[1:] + [rows]


def close(got, a, b):
    """got within the GEMMs' bound of a b^T, a and b float64 on the GPU; half a
    step more for bf16."""
    ref, mag = a @ b.T, a.abs() @ b.abs().T
    near = TOL * mag
    if got.dtype == torch.bfloat16:
        near = near + 2.0 ** -8 * (ref.abs() + near)
    assert ((got.double() - ref).abs() <= near).all()


def product(rows, offsets, N, K, out_dtype, kinds=3):
    """The grouped product of random operands, checked expert by expert."""
    E = len(offsets) - 1
    rng = np.random.default_rng(rows + N + K)
    a, ws = random_mx4(rng, rows, K), [random_mx4(rng, N, K) for _ in range(min(E, kinds))]
    ops = [operand(*w) for w in ws]
    which = [e % len(ws) for e in range(E)]
    dt = torch.bfloat16 if out_dtype == F.OUT_BF16 else torch.float32
    out = torch.full((rows, N), 77.0, dtype=dt, device="cuda")
    F.fp4_gemm_grouped(*grouped_operand(*a, rows, offsets), dev_offsets(offsets), torch.stack([ops[i][0] for i in which]),
                       torch.stack([ops[i][1] for i in which]), rows, out=out, out_dtype=out_dtype)
    torch.cuda.synchronize()
    av, wv = torch.from_numpy(values(*a)).cuda(), [torch.from_numpy(values(*w)).cuda() for w in ws]
    for i, lo, hi in zip(which, offsets, offsets[1:]):
        if hi > lo:
            close(out[lo:hi], av[lo:hi], wv[i])
    assert (out[:offsets[0]] == 77.0).all() and (out[offsets[-1]:] == 77.0).all()


# rows, experts, N: 128-row tiles (360 and 800 for 256 workgroups), 256-row tiles
# (about 500, 800); by the rounds that launch_gemm_row_groups counts
SEVERAL = {"128": (6000, 40, 1408), "128 more": (9000, 100, 1408), "256": (12000, 4, 2560), "256 more": (20000, 5, 2560)}


@pytest.mark.parametrize("size", list(SEVERAL))
@pytest.mark.parametrize("K", [96, 480, 736, 1024, 1152, 2176])
@pytest.mark.parametrize("out_dtype", [F.OUT_BF16, F.OUT_F32])
def test_several_tiles_a_workgroup(size, K, out_dtype):
    need_gpu()
    rows, E, N = SEVERAL[size]
    say("grouped, several tiles", size, K, out_dtype)
    product(rows, ragged(rows, E, K), N, K, out_dtype)


@pytest.mark.parametrize("split", list(MANY))
@pytest.mark.parametrize("N,K", [(256, 1024), (512, 2048), (304, 512), (1032, 256), (96, 288), (8, 1056), (264, 1280)])
@pytest.mark.parametrize("out_dtype", [F.OUT_BF16, F.OUT_F32])
def test_small_outputs(split, N, K, out_dtype):
    """17 experts or more take the tiles whatever the output's size: the splits
    of test_many_rows with experts that are empty."""
    need_gpu()
    rows, offsets = MANY[split]
    say("grouped tiles, small output", split, N, K, out_dtype)
    offsets = [offsets[0]] * 5 + offsets + [offsets[-1]] * max(0, 13 - len(offsets))
    assert len(offsets) > 17 and rows > 32 * (len(offsets) - 1)
    product(rows, offsets, N, K, out_dtype, kinds=8)


@pytest.mark.parametrize("size", ["128", "256"])
def test_nan_blocks_of_later_tiles(size):
    """A NaN scale in the last row of A, and in one weight row of the last expert
    with rows, reach their own outputs alone."""
    need_gpu()
    rows, E, N = SEVERAL[size]
    K, offsets = 544, ragged(rows, E, 1)
    say("grouped tiles NaN", size)
    rng = np.random.default_rng(3)
    a, w = random_mx4(rng, rows, K), [random_mx4(rng, N, K) for _ in range(2)]
    last = max(e for e in range(E) if offsets[e + 1] > offsets[e])
    a[1][rows - 1, 16] = 255
    w[1][1][33, 0] = 255
    ops = [operand(*v) for v in w]
    which = [int(e == last) for e in range(E)]
    out = torch.zeros(rows, N, device="cuda")
    F.fp4_gemm_grouped(*grouped_operand(*a, rows, offsets), dev_offsets(offsets), torch.stack([ops[i][0] for i in which]),
                       torch.stack([ops[i][1] for i in which]), rows, out=out, out_dtype=F.OUT_F32)
    torch.cuda.synchronize()
    nan = torch.zeros_like(out, dtype=torch.bool)
    nan[rows - 1] = True
    nan[offsets[last]:offsets[last + 1], 33] = True
    assert torch.equal(out.isnan(), nan)


# more than 512 rows an expert, more than 256 tiles; 0 to 3 stages over a multiple
# of four, one expert of one row
DEPTH = {"two rounds": (3900, [0, 1, 1200, 1200, 2400, 3900], 2048, 1856),
         "three rounds": (6700, [7, 1300, 2070, 2400, 4000, 4257, 5790, 6690], 1824, 1536),
         "one column of tiles": (9000, [0, 2100, 2101, 5000, 8999], 24000, 64)}


@pytest.mark.parametrize("size", list(DEPTH))
@pytest.mark.parametrize("out_dtype", [F.OUT_BF16, F.OUT_F32])
def test_several_tiles_of_long_weight_gradients(size, out_dtype):
    need_gpu()
    rows, offsets, N, K = DEPTH[size]
    E = len(offsets) - 1
    assert rows > 512 * E and E * -(-N // 256) * -(-K // 256) > 256
    say("grouped wgrad, several tiles", size, out_dtype)
    rng = np.random.default_rng(rows)
    dy, x = bf16_bits(rng.standard_normal((rows, N)) * 1e-3), bf16_bits(rng.standard_normal((rows, K)))
    qdy, vdy = quantized_rows(dy, rows, offsets, 32, F.HAD_DET, 0)
    qx, vx = quantized_rows(x, rows, offsets, 32, F.HAD_DET, 0)
    got = F.fp4_gemm_grouped_wgrad(*qdy, *qx, dev_offsets(offsets), rows, out_dtype=out_dtype)
    torch.cuda.synchronize()
    vdy, vx = torch.from_numpy(vdy).cuda(), torch.from_numpy(vx).cuda()
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        span = slice(256 * (lo // 256 + e), 256 * (lo // 256 + e) + hi - lo + (lo - hi) % 32)
        close(got[e], vdy[:, span].contiguous(), vx[:, span].contiguous())


@pytest.mark.parametrize("rows,E,N,K", [(6000, 40, 1408, 480), (12000, 4, 2560, 736)])
def test_tiles_captured_and_replayed_with_other_offsets(rows, E, N, K):
    """Quantizers, product and weight gradient on the tile kernels as one graph:
    on each replay the eager calls' bits, for splits from even to one expert
    with all rows, eager work between."""
    need_gpu()
    say("grouped tiles in a graph", rows, E, N, K)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, dy = (torch.randn(rows, c, device="cuda", generator=g).bfloat16() for c in (K, N))
    wq, ws = zip(*(F.fp4_hadamard_quantize(torch.randn(N, K, device="cuda", generator=g).bfloat16()) for _ in range(E)))
    wq, ws = torch.stack(wq), torch.stack(ws)
    even = [rows * e // E for e in range(E + 1)]
    off = dev_offsets(even)

    def step():
        xt, xts, xq, xs = F.fp4_quantize_grouped_dual(x, off, 32, F.HAD_DET)
        d = F.fp4_quantize_grouped(dy, off, F.AXIS_ROWS, 32, F.HAD_DET)
        y = F.fp4_gemm_grouped(xq, xs, off, wq, ws, rows, out=torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda"))
        return y, F.fp4_gemm_grouped_wgrad(*d, xt, xts, off, rows)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = step()
    splits = [even, ragged(rows, E, 5), [0] + [rows] * E, [0] * E + [rows], [3] * E + [700], even]
    for i, split in enumerate(splits):
        off.copy_(torch.tensor(split, dtype=torch.int32))
        x.mul_(1.25)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(caught, step()):
            assert torch.equal(a, b), i
        torch.cuda.synchronize()
