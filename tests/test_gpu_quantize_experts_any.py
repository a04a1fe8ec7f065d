"""linear.quantize_experts takes any number of experts of any size."""
import pytest
import torch

import fp4_precision_gemms_amd as F
from _util import need_gpu, say

pytestmark = pytest.mark.gpu


def each_by_itself(w, got, experts):
    """Each axis of some experts by a call of its own."""
    for e in experts:
        wq, ws = F.fp4_hadamard_quantize(w[e], F.AXIS_COLS)
        wtq, wts = F.fp4_hadamard_quantize(w[e], F.AXIS_ROWS)
        nb, nbt = w.shape[2] // 32, w.shape[1] // 32
        assert torch.equal(got[0][e], wtq) and torch.equal(got[2][e], wq)
        for a, b, n in ((got[1][e], wts, nbt), (got[3][e], ws, nb)):     # without the last group's padding
            pick = [t.permute(1, 0, 2).flatten(1)[:, :n] for t in (a, b)]
            assert torch.equal(*pick)


@pytest.mark.parametrize("E,N,K", [(1025, 32, 64), (2600, 64, 32), (2, 2 ** 22, 32), (2, 32, 2 ** 24)])
def test_more_than_one_call_takes(E, N, K):
    need_gpu()
    say("quantize experts in several calls", E, N, K)
    g = torch.Generator(device="cuda").manual_seed(E)
    w = torch.randn(E, N, K, device="cuda", generator=g, dtype=torch.bfloat16)
    w[0, 3, 5], w[-1, N - 1, K - 1] = float("nan"), float("inf")
    got = F.linear.quantize_experts(w)
    torch.cuda.synchronize()
    each_by_itself(w, got, {0, 1, E // 2, min(1023, E - 1), min(1024, E - 1), E - 1})


def test_no_experts():
    need_gpu()
    got = F.linear.quantize_experts(torch.empty(0, 64, 96, dtype=torch.bfloat16, device="cuda"))
    want = (F.code_shape(96, 64), F.scale_shape(96, 64), F.code_shape(64, 96), F.scale_shape(64, 96))
    assert [tuple(t.shape) for t in got] == [(0, *s) for s in want]
    assert all(t.dtype == torch.uint8 and t.is_cuda for t in got)


def test_experts_beyond_two_gib():
    """A launch an expert, on offsets past 32 bits."""
    need_gpu()
    E, N, K = 2, 32768, 32800
    say("experts beyond 2 GiB", E, N, K)
    w = torch.zeros(E, N, K, device="cuda", dtype=torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(1)
    for e in range(E):
        w[e, -64:] = torch.randn(64, K, device="cuda", generator=g, dtype=torch.bfloat16)
        w[e, :, -64:] = torch.randn(N, 64, device="cuda", generator=g, dtype=torch.bfloat16)
        w[e, 7] = torch.randn(K, device="cuda", generator=g, dtype=torch.bfloat16)
    got = F.fp4_quantize_experts(w)
    torch.cuda.synchronize()
    # the last rows, as a small matrix (the blocks along K are each row's own)
    for e in range(E):
        last = w[e, -64:].contiguous()
        q, s = F.fp4_hadamard_quantize(last, F.AXIS_COLS)
        assert torch.equal(got[2][e, -2:], q)
        assert torch.equal(got[3][e, :, -64:].permute(1, 0, 2).flatten(1)[:, :K // 32],
                           s.permute(1, 0, 2).flatten(1)[:, :K // 32])
        right = w[e, :, -64:].contiguous()                 # the last columns: W^T's last rows
        q, s = F.fp4_hadamard_quantize(right, F.AXIS_ROWS)
        assert torch.equal(got[0][e, -2:], q)
        assert torch.equal(got[1][e, :, -64:], s)
        assert not got[2][e, 1:-2, :K // 32 - 2].any()     # zeros between
