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


def test_gemm_decode_errors(L):
    def call(p=(A, A, A, A), fmt=1, dims=(4, 64, 64), c=A, out=1):
        return L.fp4_gemm_decode(p[0], p[1], fmt, p[2], p[3], *dims, c, out, None)

    assert call(fmt=2) == ERR_ENUM and call(out=2) == ERR_ENUM
    for i in range(4):
        assert call(p=tuple(None if j == i else A for j in range(4))) == ERR_NULL
        assert call(p=tuple(MIS if j == i else A for j in range(4))) == ERR_ALIGN
    assert call(c=None) == ERR_NULL and call(c=MIS) == ERR_ALIGN
    for dims in ((0, 64, 64), (4, -1, 64), (4, 64, 0), (4, 64, 48), (4, 64, 2 ** 24), (2 ** 31, 64, 64), (4, 2 ** 31, 64)):
        assert call(dims=dims) == ERR_SHAPE, dims


def test_quantize_grouped_errors(L):
    def call(x=A, off=A, E=4, rows=64, cols=64, hn=32, had=1, rnd=0, p=(A, A, A, A)):
        return L.fp4_quantize_grouped(x, off, E, rows, cols, hn, had, 0, rnd, 0, 0, *p, None)

    assert call(had=3) == ERR_ENUM and call(hn=8) == ERR_ENUM and call(rnd=2) == ERR_ENUM
    assert call(x=None) == ERR_NULL and call(off=None) == ERR_NULL
    for p in ((None, None, None, None), (A, None, A, A), (None, A, A, A), (A, A, None, A), (A, A, A, None)):
        assert call(p=p) == ERR_NULL, p
    assert call(E=0) == ERR_SHAPE and call(E=1025) == ERR_SHAPE
    assert call(rows=0) == ERR_SHAPE and call(cols=48) == ERR_SHAPE and call(cols=2 ** 24) == ERR_SHAPE
    assert call(rows=2 ** 31) == ERR_SHAPE
    assert call(x=MIS) == ERR_ALIGN and call(off=A + 2) == ERR_ALIGN
    for i in range(4):
        assert call(p=tuple(MIS if j == i else A for j in range(4))) == ERR_ALIGN


def test_gemm_grouped_errors(L):
    def call(a=A, s=A, fmt=0, off=A, E=4, rows=64, w=A, ws=A, N=64, K=64, c=A, out=1):
        return L.fp4_gemm_grouped(a, s, fmt, off, E, rows, w, ws, N, K, c, out, None)

    assert call(fmt=3) == ERR_ENUM and call(out=-1) == ERR_ENUM
    for name in ("a", "s", "off", "w", "ws", "c"):
        assert call(**{name: None}) == ERR_NULL, name
    for name in ("a", "s", "w", "ws", "c"):
        assert call(**{name: MIS}) == ERR_ALIGN, name
    assert call(off=A + 2) == ERR_ALIGN
    for bad in (dict(E=0), dict(E=2000), dict(rows=0), dict(N=0), dict(K=40), dict(K=2 ** 24), dict(rows=2 ** 31),
                dict(E=1024, rows=2 ** 20, N=2 ** 20)):
        assert call(**bad) == ERR_SHAPE, bad


def test_grouped_binding_refuses():
    if not os.path.exists(F.LIB_PATH):
        pytest.skip("libfp4.so not built")
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    x, off = torch.zeros(64, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        F.fp4_quantize_grouped(x, off)
    # activations that do not fit the weights, weights of another number of experts
    with pytest.raises(ValueError, match="contraction"):
        F.fp4_gemm_decode(u8(4, 64), u8(4, 2), u8(*F.code_shape(32, 96)), u8(*F.scale_shape(32, 96)))
    with pytest.raises(ValueError, match="one operand"):
        F.fp4_gemm_decode(u8(4, 64), u8(4, 3), u8(*F.code_shape(32, 64)), u8(*F.scale_shape(32, 64)))
    assert F.grouped_shapes(100, 64, 5, F.AXIS_COLS) == ((8, 2, 512), (1, 256, 8))
    assert F.grouped_shapes(1000, 64, 5, F.AXIS_ROWS) == ((2, 64, 512), (8, 64, 8))


def test_units_of_the_grouped_layout_never_meet():
    """Expert e's units start at offsets[e] // U + e: for any split they end
    before the next expert's first one and inside the layout."""
    import random
    rng = random.Random(1)
    for _ in range(500):
        rows, E = rng.randint(1, 2000), rng.randint(1, 40)
        off = sorted(rng.randint(0, rows) for _ in range(E + 1))
        for U in (32, 256):
            for e in range(E):
                end = off[e] // U + e + (off[e + 1] - off[e] + U - 1) // U
                assert end <= (off[e + 1] // U + e + 1 if e + 1 < E else rows // U + E)


def test_gemm_grouped_wgrad_errors(L):
    def call(p=(A, A, A, A), off=A, E=4, rows=64, N=64, K=64, c=A, out=1):
        return L.fp4_gemm_grouped_wgrad(*p, off, E, rows, N, K, c, out, None)

    assert call(out=2) == ERR_ENUM
    for i in range(4):
        assert call(p=tuple(None if j == i else A for j in range(4))) == ERR_NULL
        assert call(p=tuple(MIS if j == i else A for j in range(4))) == ERR_ALIGN
    assert call(off=None) == ERR_NULL and call(c=None) == ERR_NULL
    assert call(off=A + 2) == ERR_ALIGN and call(c=MIS) == ERR_ALIGN
    for bad in (dict(E=0), dict(E=1025), dict(rows=0), dict(rows=2 ** 24), dict(N=48), dict(K=16), dict(N=0),
                dict(N=2 ** 20, K=2 ** 20), dict(K=2 ** 21), dict(rows=2 ** 23, N=2 ** 14)):
        assert call(**bad) == ERR_SHAPE, bad
