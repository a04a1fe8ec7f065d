"""The norm, grouped and few-row operators on a stream given to the call: the
current stream's results, outputs from that stream's memory pool."""
import pytest
import torch

import fp4_precision_gemms_amd as F
from _util import need_gpu, say

pytestmark = pytest.mark.gpu

T, K, N, E = 160, 256, 128, 5


def pool_of(t):
    """The stream whose pool t's memory came from."""
    p = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= p < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no segment holds the tensor")


@pytest.mark.parametrize("kind", ["stream", "integer"])
def test_every_operator_on_a_given_stream(kind):
    need_gpu()
    say("operators on a given stream", kind)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r, dh = (torch.randn(T, K, device="cuda", generator=g).bfloat16() for _ in range(3))
    dy = torch.randn(T, N, device="cuda", generator=g).bfloat16()
    w = torch.randn(K, device="cuda", generator=g).bfloat16()
    off = torch.tensor([0, 30, 30, 100, 150, 160], dtype=torch.int32, device="cuda")
    wtq, wts, wq, ws = F.linear.quantize_experts((torch.randn(E, N, K, device="cuda", generator=g) * 0.05).bfloat16())

    def work(stream):
        q, s, h, rstd = norm = F.fp4_rmsnorm_quantize(x, w, r, stream=stream)
        back = F.fp4_rmsnorm_backward(x, h, w, rstd, dh, stream=stream)
        y = F.fp4_gemm_decode(q, s, wq[0], ws[0], stream=stream)
        y8 = F.fp4_gemm_grouped(q, s, off, wq, ws, T, stream=stream)
        xtq, xts, xq, xs = both = F.fp4_quantize_grouped_dual(x, off, 32, F.HAD_DET, stream=stream)
        d = F.fp4_quantize_grouped(dy, off, F.AXIS_ROWS, 32, F.HAD_DET, stream=stream)
        y4 = F.fp4_gemm_grouped(xq, xs, off, wq, ws, T, stream=stream)
        dw = F.fp4_gemm_grouped_wgrad(*d, xtq, xts, off, T, stream=stream)
        return (*norm, *back, y, y8, y4, dw), (*both, *d)

    want, _ = work(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, codes = work(s if kind == "stream" else s.cuda_stream)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()
    assert all(pool_of(t) == s.cuda_stream for t in (*got, *codes))
    assert all(pool_of(t) != s.cuda_stream for t in want)


def test_outputs_of_a_given_stream_outlive_their_readers():
    """An output that is freed while the current stream still reads it is not
    handed out again before that is done."""
    need_gpu()
    x, w = torch.ones(64, 4096, device="cuda").bfloat16(), torch.ones(4096, device="cuda").bfloat16()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = F.fp4_rmsnorm_quantize(x, w, x, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(20_000_000)                    # the reader below waits behind this
    kept = out[2].clone()
    p = out[2].data_ptr()
    del out
    again = F.fp4_rmsnorm_quantize(x, w, stream=s, y=None)
    more = F.fp4_rmsnorm_quantize(x, w, x, stream=s)
    assert more[2].data_ptr() != p
    torch.cuda.synchronize()
    assert (kept == 2).all() and again[2] is x


def test_stream_zero_is_the_default_stream():
    need_gpu()
    x, w = torch.ones(64, 64, device="cuda").bfloat16(), torch.ones(64, device="cuda").bfloat16()
    want = F.fp4_rmsnorm_backward(x, x, w, torch.ones(64, device="cuda"))
    got = F.fp4_rmsnorm_backward(x, x, w, torch.ones(64, device="cuda"), stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_a_given_stream_inside_a_captured_graph():
    """The norm on the capturing stream, its gradient and a product on a stream
    that forks from it, replayed with other inputs and eager work between."""
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(3)
    x, dy = (torch.randn(T, K, device="cuda", generator=g).bfloat16() for _ in range(2))
    w = torch.randn(K, device="cuda", generator=g).bfloat16()
    wq, ws = F.fp4_hadamard_quantize(torch.randn(N, K, device="cuda", generator=g).bfloat16())
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        q, s, h, rstd = F.fp4_rmsnorm_quantize(x, w, x, stream=here)
        side.wait_stream(here)
        y = F.fp4_gemm_decode(q, s, wq, ws, stream=side)
        back = F.fp4_rmsnorm_backward(dy, h, w, rstd, stream=side.cuda_stream)
        here.wait_stream(side)
        return (h, y + 1) + back

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = step()
    for i in range(4):
        x.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(caught, step()):
            assert torch.equal(a, b), i
        torch.cuda.synchronize()
