"""The norm, grouped and few-row entry points without a GPU: arguments are
refused with the documented status codes before any HIP call, and by the
binding before the library is reached."""
import os

import pytest
import torch

import fp4_precision_gemms_amd as F

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_ENUM, ERR_LAUNCH, ERR_WORKSPACE = range(7)
A = 0x10000          # a fake 16-byte aligned device address (never dereferenced)
MIS = 0x10008        # misaligned


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(F.LIB_PATH):
        pytest.skip("libfp4.so not built")
    return F.lib()


def test_rmsnorm_quantize_errors(L):
    def call(x=A, res=A, w=A, eps=1e-5, rows=4, cols=64, fmt=1, h=A, rstd=A, y=None, codes=A, scales=A):
        return L.fp4_rmsnorm_quantize(x, res, w, eps, rows, cols, fmt, h, rstd, y, codes, scales, None)

    assert call(fmt=2) == ERR_ENUM and call(fmt=-1) == ERR_ENUM
    assert call(eps=-1e-9) == ERR_ENUM and call(eps=float("nan")) == ERR_ENUM
    for name in ("x", "w", "codes", "scales", "h"):
        assert call(**{name: None}) == ERR_NULL, name
    assert call(rows=0) == ERR_SHAPE and call(rows=-3) == ERR_SHAPE and call(rows=2 ** 31) == ERR_SHAPE
    assert call(cols=0) == ERR_SHAPE and call(cols=48) == ERR_SHAPE and call(cols=32800) == ERR_SHAPE
    for name in ("x", "res", "w", "h", "y", "codes", "scales"):
        assert call(**{name: MIS}) == ERR_ALIGN, name
    assert call(rstd=A + 2) == ERR_ALIGN


def test_rmsnorm_backward_errors(L):
    def call(dy=A, h=A, w=A, rstd=A, dh=None, rows=4, cols=64, dx=A, dw=A, ws=A, wsb=4 * 64 * 4):
        return L.fp4_rmsnorm_backward(dy, h, w, rstd, dh, rows, cols, dx, dw, ws, wsb, None)

    for name in ("dy", "h", "w", "rstd", "dx", "dw"):
        assert call(**{name: None}) == ERR_NULL, name
    assert call(rows=0) == ERR_SHAPE and call(cols=72) == ERR_SHAPE and call(cols=65536) == ERR_SHAPE
    assert call(ws=None) == ERR_WORKSPACE and call(wsb=4 * 64 * 4 - 1) == ERR_WORKSPACE
    for name in ("dy", "h", "w", "dh", "dx", "dw", "ws"):
        assert call(**{name: MIS}) == ERR_ALIGN, name
    assert L.fp4_rmsnorm_workspace_bytes(4, 64) == 4 * 64 * 4
    assert L.fp4_rmsnorm_workspace_bytes(0, 64) == 0 and L.fp4_rmsnorm_workspace_bytes(4, 40) == 0


def test_norm_binding_refuses():
    if not os.path.exists(F.LIB_PATH):
        pytest.skip("libfp4.so not built")
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        F.fp4_rmsnorm_quantize(x, w)
    with pytest.raises(TypeError, match="x must be"):
        F.fp4_rmsnorm_quantize(x.float(), w)
    with pytest.raises(ValueError, match="GPU"):
        F.fp4_rmsnorm_backward(x, x, w, torch.zeros(4))
    with pytest.raises(TypeError, match="dy must be"):
        F.fp4_rmsnorm_backward(x.float(), x, w, torch.zeros(4))
