"""What the binding of the norm, grouped and few-row operators refuses on GPU
tensors, and that a refused call leaves the outputs alone."""
import pytest
import torch

import fp4_precision_gemms_amd as F
from _util import need_gpu

pytestmark = pytest.mark.gpu


def u8(shape):
    return torch.full(tuple(shape), 0x22, dtype=torch.uint8, device="cuda")


@pytest.fixture
def t():
    need_gpu()

    class T:
        x = torch.ones(64, 96, device="cuda").bfloat16()
        w = torch.ones(96, device="cuda").bfloat16()
        off = torch.tensor([0, 40, 64], dtype=torch.int32, device="cuda")
        wq, ws = u8((2, *F.code_shape(32, 96))), u8((2, *F.scale_shape(32, 96)))
        aq, as_ = u8(F.grouped_shapes(64, 96, 2, F.AXIS_COLS)[0]), u8(F.grouped_shapes(64, 96, 2, F.AXIS_COLS)[1])
    return T


def test_norm(t):
    for bad, what in ((t.x.t(), "shape|contiguous"), (t.x[:, :64], "shape|contiguous"), (t.x[0], "two dimensions")):
        with pytest.raises(ValueError, match=what):
            F.fp4_rmsnorm_quantize(bad, t.w)
    with pytest.raises(ValueError, match="contiguous"):
        F.fp4_rmsnorm_quantize(t.x[:, ::1].t().contiguous().t(), t.w)
    with pytest.raises(TypeError, match="weight must be torch.bfloat16"):
        F.fp4_rmsnorm_quantize(t.x, t.w.float())
    with pytest.raises(ValueError, match="weight must have shape"):
        F.fp4_rmsnorm_quantize(t.x, t.w[:64])
    with pytest.raises(ValueError, match="residual must be a GPU tensor"):
        F.fp4_rmsnorm_quantize(t.x, t.w, t.x.cpu())
    with pytest.raises(TypeError, match="weight must be a tensor"):
        F.fp4_rmsnorm_quantize(t.x, None)
    with pytest.raises(ValueError, match="4 tensors"):
        F.fp4_rmsnorm_quantize(t.x, t.w, out=(t.x,))
    for kw in (dict(fmt=7), dict(eps=-1.0)):
        with pytest.raises(F.Fp4Error) as e:
            F.fp4_rmsnorm_quantize(t.x, t.w, **kw)
        assert e.value.status == 4
    with pytest.raises(F.Fp4Error) as e:
        F.fp4_rmsnorm_quantize(t.x[:, :80].contiguous(), t.w[:80])
    assert e.value.status == 2
    with pytest.raises(F.Fp4Error) as e:
        F.fp4_rmsnorm_quantize(t.x[:0], t.w)
    assert e.value.status == 2
    rstd = torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="dh must have shape"):
        F.fp4_rmsnorm_backward(t.x, t.x, t.w, rstd, t.x[:32])
    with pytest.raises(TypeError, match="rstd must be torch.float32"):
        F.fp4_rmsnorm_backward(t.x, t.x, t.w, rstd.bfloat16())
    # outputs from any iterable
    out = F.fp4_rmsnorm_quantize(t.x, t.w)
    again = F.fp4_rmsnorm_quantize(t.x, t.w, out=(v for v in [o.clone() for o in out]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, again))


def test_offsets(t):
    for bad, error, what in ((t.off.long(), TypeError, "torch.int32"), (t.off.cpu(), ValueError, "GPU tensor"),
                             (t.off[:1], ValueError, "experts"), (t.off.view(3, 1), ValueError, "experts"),
                             (torch.stack((t.off, t.off), 1)[:, 0], ValueError, "contiguous")):
        with pytest.raises(error, match=what):
            F.fp4_quantize_grouped(t.x, bad)
        with pytest.raises(error, match=what):
            F.fp4_gemm_grouped(t.aq, t.as_, bad, t.wq, t.ws, 64)


def test_grouped(t):
    with pytest.raises(ValueError, match="axis"):
        F.fp4_quantize_grouped(t.x, t.off, 2)
    with pytest.raises(F.Fp4Error) as e:
        F.fp4_quantize_grouped(t.x, t.off, F.AXIS_ROWS, 8, F.HAD_DET)
    assert e.value.status == 4
    with pytest.raises(F.Fp4Error) as e:
        F.fp4_quantize_grouped(t.x[:, :80].contiguous(), t.off)
    assert e.value.status == 2
    with pytest.raises(ValueError, match="2 experts"):
        F.fp4_gemm_grouped(t.aq, t.as_, t.off, t.wq[:1], t.ws[:1], 64)
    with pytest.raises(ValueError, match="a codes must have shape"):
        F.fp4_gemm_grouped(t.aq, t.as_, t.off, t.wq, t.ws, 96)
    with pytest.raises(ValueError, match="out must have shape"):
        F.fp4_gemm_grouped(t.aq, t.as_, t.off, t.wq, t.ws, 64, out=torch.empty(64, 33, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError, match="out must be torch.bfloat16"):
        F.fp4_gemm_grouped(t.aq, t.as_, t.off, t.wq, t.ws, 64, out=torch.empty(64, 32, device="cuda"))
    with pytest.raises(F.Fp4Error) as e:
        F.fp4_gemm_grouped(t.aq, t.as_, t.off, t.wq, t.ws, 64, out_dtype=5)
    assert e.value.status == 4
    rows = [u8(s) for s in F.grouped_shapes(64, 96, 2, F.AXIS_ROWS)]
    with pytest.raises(ValueError, match="X codes must have shape"):
        F.fp4_gemm_grouped_wgrad(*rows, rows[0][:1], rows[1], t.off, 64)
    with pytest.raises(ValueError, match="dY codes must have shape"):
        F.fp4_gemm_grouped_wgrad(*rows, *rows, t.off, 600)


def test_decode(t):
    q, s = F.fp4_hadamard_quantize(t.x)
    with pytest.raises(ValueError, match="contraction"):
        F.fp4_gemm_decode(q, s, u8(F.code_shape(32, 128)), u8(F.scale_shape(32, 128)))
    with pytest.raises(ValueError, match="one operand"):
        F.fp4_gemm_decode(q, s[:, :32].contiguous(), t.wq[0], t.ws[0])
    with pytest.raises(ValueError, match="three dimensions"):
        F.fp4_gemm_decode(q, s, t.wq, t.ws)
    with pytest.raises(TypeError, match="a codes must be torch.uint8"):
        F.fp4_gemm_decode(torch.zeros(4, 96, device="cuda", dtype=torch.int8), u8((4, 3)), t.wq[0], t.ws[0])
