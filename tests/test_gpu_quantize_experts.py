"""fp4_quantize_experts bit for bit against a call an expert, and what it refuses."""
import pytest
import torch

import fp4_precision_gemms_amd as F
from _util import need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,N,K", [(1, 32, 32), (1, 4096, 96), (3, 96, 160), (2, 288, 1120), (5, 736, 1120), (40, 64, 288),
                                   (1024, 32, 64), (8, 2048, 2080)])
def test_every_expert_as_by_itself(E, N, K):
    need_gpu()
    say("quantize experts", E, N, K)
    g = torch.Generator(device="cuda").manual_seed(N + K)
    w = (torch.randn(E, N, K, device="cuda", generator=g) * torch.exp2(torch.randint(-20, 20, (E, N, 1), device="cuda", generator=g).float())).bfloat16()
    w[0, 3, 5], w[-1, N - 1, K - 1], w[E // 2, 0] = float("nan"), float("inf"), 0
    shapes = (F.code_shape(K, N), F.scale_shape(K, N), F.code_shape(N, K), F.scale_shape(N, K))
    out = [torch.full((E, *s), 0xCD, dtype=torch.uint8, device="cuda") for s in shapes]
    want = [t.clone() for t in out]
    got = F.fp4_quantize_experts(w, out=out)
    for e in range(E):
        F.fp4_hadamard_quantize_dual(w[e], out=[t[e] for t in want])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    new = F.linear.quantize_experts(w)
    assert all(t.shape == (E, *s) for t, s in zip(new, shapes))
    assert torch.equal(new[0], want[0]) and torch.equal(new[2], want[2])


def test_weights_that_are_not_contiguous():
    need_gpu()
    w = torch.randn(3, 256, 512, device="cuda").bfloat16()       # whole scale groups: every byte is written
    for a, b in zip(F.linear.quantize_experts(w.transpose(1, 2)), F.linear.quantize_experts(w.transpose(1, 2).contiguous())):
        assert torch.equal(a, b)
    with pytest.raises(ValueError, match="contiguous"):
        F.fp4_quantize_experts(w.transpose(1, 2))


def test_refusals_and_streams():
    need_gpu()
    w = torch.randn(3, 64, 96, device="cuda").bfloat16()
    out = F.fp4_quantize_experts(w)
    with pytest.raises(ValueError, match="output of shape"):
        F.fp4_quantize_experts(w, out=(out[1], out[1], out[2], out[3]))
    with pytest.raises(ValueError, match="out must be"):
        F.fp4_quantize_experts(w, out=out[:3])
    with pytest.raises(TypeError, match="torch.bfloat16"):
        F.fp4_quantize_experts(w.float())
    with pytest.raises(F.Fp4Error) as e:
        F.fp4_quantize_experts(w[:, :40].contiguous())
    assert e.value.status == 2
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = F.fp4_quantize_experts(w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], out[0]) and torch.equal(got[2], out[2])
