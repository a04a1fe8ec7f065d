"""Python binding of libfp4.so, the MXFP4 / NVFP4 block-quantized linear layer
for AMD Instinct MI355X (gfx950).

The functions below carry the names of the C entry points (include/fp4.h)
and only marshal arguments: shapes and pointers of torch tensors in, status
codes out (through ctypes; the operators from the norm on, whose calls are
short, through the CPython functions of csrc/torch_binding*.cpp).  Every step of the computation runs in the HIP kernels of the
library.  torch supplies device memory and the current HIP stream.

A call runs on the current stream of its tensors' device, or on `stream` (a
torch stream or a hipStream_t as an integer), which the caller orders against
the streams that make the inputs and read the outputs; inputs that are freed
before that stream is done are recorded on it (Tensor.record_stream), as for any
torch operator on a side stream.

Where a call makes its outputs itself, small ones of one call, and codes with their
scales, may share an allocation, which lives as long as any of them.

If the libraries have not been built (``python -m fp4_precision_gemms_amd.build``)
every call raises; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

AXIS_COLS, AXIS_ROWS = 0, 1
HAD_NONE, HAD_DET, HAD_SIGNED = 0, 1, 2
RTN, SR = 0, 1
OUT_F32, OUT_BF16 = 0, 1
FMT_MXFP4, FMT_MXFP8 = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
ACT_SILU, ACT_GELU = 0, 1

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp4.so")
_lib = None


class Fp4Error(RuntimeError):
    """A nonzero fp4_status returned by the library."""

    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded libfp4.so with argument types set; raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libfp4.so is not built: run `python -m fp4_precision_gemms_amd.build` "
                           "(expected at %s)" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    i64, u64, i32, vp = ctypes.c_int64, ctypes.c_uint64, ctypes.c_int, ctypes.c_void_p
    L.fp4_hadamard_quantize.argtypes = [vp, i64, i64, i32, i32, i32, u64, i32, u64, vp, vp, vp]
    L.fp4_hadamard_quantize.restype = i32
    for name in ("fp4_gemm_fprop", "fp4_gemm_dgrad", "fp4_gemm_wgrad"):
        fn = getattr(L, name)
        fn.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, vp]
        fn.restype = i32
    L.fp4_hadamard_quantize_dual.argtypes = [vp, i64, i64, i32, i32, u64, i32, u64, vp, vp,
                                             i32, i32, u64, i32, u64, vp, vp, vp]
    L.fp4_hadamard_quantize_dual.restype = i32
    L.fp4_wgrad_quantize.argtypes = [vp, vp, i64, i64, i64, i32, i32, u64, i32, u64, u64,
                                     vp, vp, vp, vp, vp]
    L.fp4_wgrad_quantize.restype = i32
    L.fp4_gemm_mx.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, i32, i32, vp]
    L.fp4_gemm_mx.restype = i32
    L.nvfp4_quantize.argtypes = [vp, i64, i64, i32, u64, i32, u64, vp, vp, vp, vp, vp,
                                 ctypes.c_size_t, vp]
    L.nvfp4_quantize.restype = i32
    L.nvfp4_quantize_noalloc.argtypes = [vp, i64, i64, i32, u64, i32, u64, vp, vp, vp, vp, vp]
    L.nvfp4_quantize_noalloc.restype = i32
    L.nvfp4_workspace_bytes.argtypes = [i64, i64]
    L.nvfp4_workspace_bytes.restype = ctypes.c_size_t
    L.fp4_rmsnorm_quantize.argtypes = [vp, vp, vp, ctypes.c_double, i64, i64, i32, vp, vp, vp, vp, vp, vp]
    L.fp4_rmsnorm_quantize.restype = i32
    L.fp4_rmsnorm_backward.argtypes = [vp, vp, vp, vp, vp, i64, i64, vp, vp, vp, ctypes.c_size_t, vp]
    L.fp4_rmsnorm_backward.restype = i32
    L.fp4_rmsnorm_workspace_bytes.argtypes = [i64, i64]
    L.fp4_rmsnorm_workspace_bytes.restype = ctypes.c_size_t
    L.fp4_gemm_decode.argtypes = [vp, vp, i32, vp, vp, i64, i64, i64, vp, i32, vp]
    L.fp4_gemm_decode.restype = i32
    L.fp4_quantize_grouped.argtypes = [vp, vp, i64, i64, i64, i32, i32, u64, i32, u64, u64, vp, vp, vp, vp, vp]
    L.fp4_quantize_grouped.restype = i32
    L.fp4_gemm_grouped.argtypes = [vp, vp, i32, vp, i64, i64, vp, vp, i64, i64, vp, i32, vp]
    L.fp4_gemm_grouped.restype = i32
    L.fp4_gemm_grouped_wgrad.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, i32, vp]
    L.fp4_gemm_grouped_wgrad.restype = i32
    L.fp4_moe_route.argtypes = [vp, i32, i64, i64, i64, i32, i32, vp, vp, vp]
    L.fp4_moe_route.restype = i32
    L.fp4_moe_route_backward.argtypes = [vp, vp, i32, vp, i64, i64, i64, i32, i32, vp, vp]
    L.fp4_moe_route_backward.restype = i32
    L.fp4_moe_sort.argtypes = [vp, i64, i64, vp, vp, vp, vp, ctypes.c_size_t, vp]
    L.fp4_moe_sort.restype = i32
    L.fp4_moe_sort_workspace_bytes.argtypes = [i64, i64]
    L.fp4_moe_sort_workspace_bytes.restype = ctypes.c_size_t
    L.fp4_moe_gather.argtypes = [vp, vp, vp, i64, i64, i64, i64, vp, vp, vp]
    L.fp4_moe_gather.restype = i32
    L.fp4_moe_combine.argtypes = [vp, vp, vp, i64, i64, i64, i64, vp, vp]
    L.fp4_moe_combine.restype = i32
    L.fp4_moe_combine_backward.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, vp, vp, vp]
    L.fp4_moe_combine_backward.restype = i32
    L.fp4_quantize_experts.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, vp]
    L.fp4_quantize_experts.restype = i32
    L.fp4_glu.argtypes = [vp, vp, vp, vp, i64, i32, i64, i64, vp, i32, vp, vp, vp, vp, vp]
    L.fp4_glu.restype = i32
    L.fp4_glu_backward.argtypes = [vp, vp, vp, vp, vp, vp, i64, i32, i64, i64, vp, vp, vp]
    L.fp4_glu_backward.restype = i32
    L.fp4_status_string.argtypes = [i32]
    L.fp4_status_string.restype = ctypes.c_char_p
    _lib = L
    return L


def fp4_status_string(status: int) -> str:
    return lib().fp4_status_string(int(status)).decode()


def _check(status: int) -> None:
    if status != 0:
        raise Fp4Error(status, fp4_status_string(status))


def _stream_ptr(stream, device) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, dtype, name: str) -> None:
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


_binding = None


def _native():
    """The functions of csrc/torch_binding.cpp; raises if they are not built."""
    global _binding
    if _binding is None:
        lib()
        try:
            from . import _torch_binding
        except ImportError as e:
            raise RuntimeError("_torch_binding.so is not built: run `python -m fp4_precision_gemms_amd.build`") from e
        _torch_binding.set_error(Fp4Error)
        _binding = _torch_binding
    return _binding


def _as_stream(stream, device) -> torch.cuda.Stream:
    """A torch stream of `stream`: one already, or a hipStream_t as an integer
    (or as the `cuda_stream` of another library's object)."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    p = int(getattr(stream, "cuda_stream", stream))
    return torch.cuda.ExternalStream(p, device) if p else torch.cuda.default_stream(device)


def _call(function, like, stream, *args):
    """function(*args, stream) of the native binding, on `stream` or by default
    on the current stream of like's device.  What the function allocates
    (outputs, a workspace) comes from the pool of the stream that it runs on:
    a block of the current stream's pool may still be in use by work queued
    there, which `stream` does not wait for.  Outputs are recorded on the current
    stream, whose work may read them after it has waited for `stream`."""
    if stream is None:
        return function(*args, None)               # which takes the current one
    if not getattr(like, "is_cuda", False):
        return function(*args, 0)                  # refuses it
    here, there = torch.cuda.current_stream(like.device), _as_stream(stream, like.device)
    with torch.cuda.stream(there):
        out = function(*args, there.cuda_stream)
    if here.cuda_stream != there.cuda_stream:
        for t in out if isinstance(out, tuple) else (out,):
            t.record_stream(here)
    return out


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """An output or workspace of a call on `stream` that the library makes itself:
    from the stream's pool, recorded on the current stream (as _call does)."""
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    here, there = torch.cuda.current_stream(device), _as_stream(stream, device)
    with torch.cuda.stream(there):
        t = torch.empty(shape, dtype=dtype, device=device)
    if here.cuda_stream != there.cuda_stream:
        t.record_stream(here)
    return t


def code_shape(R: int, C: int):
    """Shape of the MXFP4 codes of R rows of C contraction elements in the
    library's 32-row tiled layout: for each group of 32 rows and each
    32-element block, the 32 rows' 16 code bytes are one 512-byte chunk
    ([ceil(R/32), C/32, 512]; row r at bytes 16 (r mod 32) of its chunk)."""
    return ((R + 31) // 32, C // 32, 512)


def scale_shape(R: int, C: int):
    """k-grouped E8M0 scale shape of R rows of C contraction elements:
    [ceil(C/256), R, 8], block b of row r at [b // 8, r, b % 8]."""
    return ((C // 32 + 7) // 8, R, 8)


def mx_shapes(rows: int, cols: int, axis: int):
    """(codes shape, scales shape) of fp4_hadamard_quantize's outputs for
    x[rows, cols] along `axis` (the logical operand has R rows of C
    contraction elements: (rows, cols) along cols, (cols, rows) along rows)."""
    R, C = (rows, cols) if axis == AXIS_COLS else (cols, rows)
    return code_shape(R, C), scale_shape(R, C)


def mx_dims(codes: torch.Tensor, scales: torch.Tensor):
    """(R, C) of an MXFP4 operand from its codes and scales, checking that
    the two agree."""
    if codes.dim() != 3 or scales.dim() != 3:
        raise ValueError("MXFP4 operands are codes [ceil(R/32), C/32, 512] and scales [ceil(C/256), R, 8]")
    R, C = scales.shape[1], codes.shape[1] * 32
    if tuple(codes.shape) != code_shape(R, C) or tuple(scales.shape) != scale_shape(R, C):
        raise ValueError("codes %s and scales %s do not describe one operand"
                         % (tuple(codes.shape), tuple(scales.shape)))
    return R, C


def fp4_hadamard_quantize(x: torch.Tensor, axis: int = AXIS_COLS, had_n: int = 32,
                          had: int = HAD_NONE, sign_seed: int = 0, rnd: int = RTN,
                          sr_seed: int = 0, codes: torch.Tensor | None = None,
                          scales: torch.Tensor | None = None, stream=None):
    """MXFP4 codes and E8M0 scales of bf16 x[rows, cols] (see include/fp4.h)."""
    _need(x, torch.bfloat16, "x")
    rows, cols = x.shape
    if axis not in (AXIS_COLS, AXIS_ROWS):         # ctypes would pass its low bits, the shapes go by all of it
        _check(4)
    cshape, sshape = mx_shapes(rows, cols, axis)
    if codes is None:
        codes = _empty(cshape, torch.uint8, x.device, stream)
    if scales is None:
        scales = _empty(sshape, torch.uint8, x.device, stream)
    _need(codes, torch.uint8, "codes")
    _need(scales, torch.uint8, "scales")
    if tuple(codes.shape) != cshape or tuple(scales.shape) != sshape:
        raise ValueError("output shapes must be %s and %s" % (cshape, sshape))
    _check(lib().fp4_hadamard_quantize(x.data_ptr(), rows, cols, axis, had_n, had,
                                       sign_seed & (2 ** 64 - 1), rnd, sr_seed & (2 ** 64 - 1),
                                       codes.data_ptr(), scales.data_ptr(),
                                       _stream_ptr(stream, x.device)))
    return codes, scales


def fp4_hadamard_quantize_dual(x: torch.Tensor, had_n_rows: int = 32, had_rows: int = HAD_NONE,
                               sign_seed_rows: int = 0, rnd_rows: int = RTN, sr_seed_rows: int = 0,
                               had_n_cols: int = 32, had_cols: int = HAD_NONE, sign_seed_cols: int = 0,
                               rnd_cols: int = RTN, sr_seed_cols: int = 0, out=None, stream=None):
    """Both quantizations of bf16 x[rows, cols] from one read: (codes, scales)
    along rows (as AXIS_ROWS) and along cols (as AXIS_COLS), each with its own
    rotation and rounding (see include/fp4.h).  `out`: optional preallocated
    (codes_rows, scales_rows, codes_cols, scales_cols)."""
    _need(x, torch.bfloat16, "x")
    rows, cols = x.shape
    (cr, sr), (cc, sc) = mx_shapes(rows, cols, AXIS_ROWS), mx_shapes(rows, cols, AXIS_COLS)
    dev = x.device
    if out is None:
        out = [_empty(sh, torch.uint8, dev, stream) for sh in (cr, sr, cc, sc)]
    for t, sh in zip(out, (cr, sr, cc, sc)):
        _need(t, torch.uint8, "output")
        if tuple(t.shape) != tuple(sh):
            raise ValueError("output of shape %s expected, got %s" % (sh, tuple(t.shape)))
    m = 2 ** 64 - 1
    _check(lib().fp4_hadamard_quantize_dual(
        x.data_ptr(), rows, cols, had_n_rows, had_rows, sign_seed_rows & m, rnd_rows, sr_seed_rows & m,
        out[0].data_ptr(), out[1].data_ptr(), had_n_cols, had_cols, sign_seed_cols & m, rnd_cols,
        sr_seed_cols & m, out[2].data_ptr(), out[3].data_ptr(), _stream_ptr(stream, dev)))
    return tuple(out)


def fp4_wgrad_quantize(dy: torch.Tensor, x: torch.Tensor, had_n: int = 32, had: int = HAD_DET,
                       sign_seed: int = 0, rnd: int = RTN, sr_seed_dy: int = 0, sr_seed_x: int = 0,
                       out=None, stream=None):
    """The Wgrad operand pair: dY[T, N] and X[T, K] quantized along T with one
    rotation; returns (dytq, dyts, xtq, xts) (see include/fp4.h)."""
    T, N = dy.shape
    if x.shape[0] != T:
        raise ValueError("dy and x must have the same number of rows")
    K = x.shape[1]
    (a, b), (c, d) = mx_shapes(T, N, AXIS_ROWS), mx_shapes(T, K, AXIS_ROWS)
    if out is not None:
        # the kernels write exactly these extents: a smaller buffer would be
        # written past its end
        if len(out) != 4:
            raise ValueError("out must be (dytq, dyts, xtq, xts)")
        for t, sh, n in zip(out, (a, b, c, d), ("dytq", "dyts", "xtq", "xts")):
            if tuple(t.shape) != tuple(sh):
                raise ValueError("%s must have shape %s, got %s" % (n, tuple(sh), tuple(t.shape)))
    _need(dy, torch.bfloat16, "dy")
    _need(x, torch.bfloat16, "x")
    if out is None:
        out = tuple(_empty(sh, torch.uint8, dy.device, stream) for sh in (a, b, c, d))
    for t in out:
        _need(t, torch.uint8, "output")
    m = 2 ** 64 - 1
    _check(lib().fp4_wgrad_quantize(dy.data_ptr(), x.data_ptr(), T, N, K, had_n, had, sign_seed & m, rnd,
                                    sr_seed_dy & m, sr_seed_x & m, *(t.data_ptr() for t in out),
                                    _stream_ptr(stream, dy.device)))
    return out


def _gemm(fn, aq, as_, bq, bs, T, N, K, out_shape, out, stream):
    for t, n in ((aq, "a codes"), (as_, "a scales"), (bq, "b codes"), (bs, "b scales")):
        _need(t, torch.uint8, n)
    if out is None:
        out = _empty(out_shape, torch.float32, aq.device, stream)
    _need(out, torch.float32, "out")
    if tuple(out.shape) != tuple(out_shape):
        raise ValueError("out must have shape %s" % (out_shape,))
    _check(fn(aq.data_ptr(), as_.data_ptr(), bq.data_ptr(), bs.data_ptr(), T, N, K,
              out.data_ptr(), _stream_ptr(stream, aq.device)))
    return out


def _operands(aq, as_, bq, bs, what):
    M, Ka = mx_dims(aq, as_)
    N, Kb = mx_dims(bq, bs)
    if Ka != Kb:
        raise ValueError("%s operands have different contraction sizes (%d, %d)" % (what, Ka, Kb))
    return M, N, Ka


def fp4_gemm_fprop(xq, xs, wq, ws, out=None, stream=None):
    """y[T, N] = X W^T from X and W quantized along K."""
    T, N, K = _operands(xq, xs, wq, ws, "fprop")
    return _gemm(lib().fp4_gemm_fprop, xq, xs, wq, ws, T, N, K, (T, N), out, stream)


def fp4_gemm_dgrad(dyq, dys, wtq, wts, out=None, stream=None):
    """dx[T, K] = dY W from dY quantized along N and W^T (W along its rows)."""
    T, K, N = _operands(dyq, dys, wtq, wts, "dgrad")
    return _gemm(lib().fp4_gemm_dgrad, dyq, dys, wtq, wts, T, N, K, (T, K), out, stream)


def fp4_gemm_wgrad(dytq, dyts, xtq, xts, out=None, stream=None):
    """dw[N, K] = dY^T X from dY^T and X^T (both quantized along T)."""
    N, K, T = _operands(dytq, dyts, xtq, xts, "wgrad")
    return _gemm(lib().fp4_gemm_wgrad, dytq, dyts, xtq, xts, T, N, K, (N, K), out, stream)


def fp4_gemm_mx(aq, as_, bq, bs, out=None, out_dtype: int = OUT_F32, accumulate: bool = False,
                stream=None):
    """C[M, N] = A B^T (+ C when accumulate) from MXFP4 operands A [M, Kc] and
    B [N, Kc] (codes and scales as the quantizers write them); C fp32 or
    bf16 (see include/fp4.h)."""
    M, N, Kc = _operands(aq, as_, bq, bs, "gemm")
    for t, n in ((aq, "a codes"), (as_, "a scales"), (bq, "b codes"), (bs, "b scales")):
        _need(t, torch.uint8, n)
    dt = {OUT_F32: torch.float32, OUT_BF16: torch.bfloat16}[out_dtype]
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an existing out")
        out = _empty((M, N), dt, aq.device, stream)
    _need(out, dt, "out")
    if tuple(out.shape) != (M, N):
        raise ValueError("out must have shape %s" % ((M, N),))
    _check(lib().fp4_gemm_mx(aq.data_ptr(), as_.data_ptr(), bq.data_ptr(), bs.data_ptr(), M, N, Kc,
                             out.data_ptr(), out_dtype, int(bool(accumulate)),
                             _stream_ptr(stream, aq.device)))
    return out


def nvfp4_workspace_bytes(rows: int, cols: int) -> int:
    return int(lib().nvfp4_workspace_bytes(rows, cols))


NV_RTN, NV_RENORM_SR, NV_ELEMENT_SR = 0, 1, 2   # nvfp4_mode


def nvfp4_quantize(x: torch.Tensor, had: int = HAD_SIGNED, sign_seed: int = 0, mode: int = NV_RENORM_SR,
                   sr_seed: int = 0, amax_in: torch.Tensor | None = None,
                   codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                   tensor_scale: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None):
    """NVFP4 codes [rows, cols/2], E4M3 scales [rows, cols/16] and the fp32
    tensor scale (a 1-element device tensor) of bf16 x (see include/fp4.h)."""
    rows, cols = x.shape
    for t, sh, n in ((codes, (rows, cols // 2), "codes"), (scales, (rows, cols // 16), "scales"),
                     (tensor_scale, (1,), "tensor_scale")):
        if t is not None and tuple(t.shape) != sh:
            raise ValueError("%s must have shape %s, got %s" % (n, sh, tuple(t.shape)))
    if amax_in is not None and amax_in.numel() != 1:
        raise ValueError("amax_in must hold one float")
    _need(x, torch.bfloat16, "x")
    dev = x.device
    codes = _empty((rows, cols // 2), torch.uint8, dev, stream) if codes is None else codes
    scales = _empty((rows, cols // 16), torch.uint8, dev, stream) if scales is None else scales
    tensor_scale = _empty(1, torch.float32, dev, stream) if tensor_scale is None else tensor_scale
    for t, dt, n in ((codes, torch.uint8, "codes"), (scales, torch.uint8, "scales"),
                     (tensor_scale, torch.float32, "tensor_scale")):
        _need(t, dt, n)
    if amax_in is not None:
        _need(amax_in, torch.float32, "amax_in")
    if workspace is not None:
        _need(workspace, torch.uint8, "workspace")
    if amax_in is None and workspace is None:
        workspace = _empty(nvfp4_workspace_bytes(rows, cols), torch.uint8, dev, stream)
    _check(lib().nvfp4_quantize(x.data_ptr(), rows, cols, had, sign_seed & (2 ** 64 - 1), mode,
                                sr_seed & (2 ** 64 - 1), _ptr(amax_in), codes.data_ptr(),
                                scales.data_ptr(), tensor_scale.data_ptr(), _ptr(workspace),
                                0 if workspace is None else workspace.numel() * workspace.element_size(),
                                _stream_ptr(stream, dev)))
    return codes, scales, tensor_scale


def nvfp4_quantize_noalloc(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                           tensor_scale: torch.Tensor, had: int = HAD_SIGNED, sign_seed: int = 0,
                           mode: int = NV_RENORM_SR, sr_seed: int = 0,
                           amax_in: torch.Tensor | None = None, stream=None):
    """nvfp4_quantize into caller-provided outputs, with the in-library amax
    in the library's own device scratch instead of a workspace (see
    include/fp4.h: calls that overlap on one GPU race on it)."""
    rows, cols = x.shape
    for t, sh, dt, n in ((codes, (rows, cols // 2), torch.uint8, "codes"),
                         (scales, (rows, cols // 16), torch.uint8, "scales"),
                         (tensor_scale, (1,), torch.float32, "tensor_scale")):
        if tuple(t.shape) != sh:
            raise ValueError("%s must have shape %s, got %s" % (n, sh, tuple(t.shape)))
        _need(t, dt, n)
    _need(x, torch.bfloat16, "x")
    if amax_in is not None:
        if amax_in.numel() != 1:
            raise ValueError("amax_in must hold one float")
        _need(amax_in, torch.float32, "amax_in")
    _check(lib().nvfp4_quantize_noalloc(x.data_ptr(), rows, cols, had, sign_seed & (2 ** 64 - 1), mode,
                                        sr_seed & (2 ** 64 - 1), _ptr(amax_in), codes.data_ptr(),
                                        scales.data_ptr(), tensor_scale.data_ptr(),
                                        _stream_ptr(stream, x.device)))
    return codes, scales, tensor_scale


def mx8_shapes(R: int, C: int):
    """(codes shape, scales shape) of an MXFP8 operand of R rows of C
    contraction elements: row-major E4M3 bytes and E8M0 scale bytes."""
    return (R, C), (R, C // 32)


def fp4_rmsnorm_quantize(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                         eps: float = 1e-5, fmt: int = FMT_MXFP8, out=None, y: torch.Tensor | None = None,
                         stream=None):
    """h = x + residual and its root-mean-square norm times `weight`, quantized
    along cols: (codes, scales, h, rstd) of bf16 x[rows, cols] (see
    include/fp4.h).  fmt FMT_MXFP8: codes (E4M3) and scales in the shapes of
    mx8_shapes(rows, cols); FMT_MXFP4: of mx_shapes(rows, cols, AXIS_COLS), all
    uint8.  h is x itself without a residual, rstd
    fp32 [rows].  `out`: optional preallocated (codes, scales, h, rstd); h may
    be x or residual.  `y`: optional bf16 [rows, cols] that receives the norm
    before its quantization, rounded to bf16."""
    return _call(_native().rmsnorm_quantize, x, stream, x, weight, residual, eps, fmt, out, y)


def fp4_rmsnorm_workspace_bytes(rows: int, cols: int) -> int:
    return int(lib().fp4_rmsnorm_workspace_bytes(rows, cols))


def fp4_rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                         dh: torch.Tensor | None = None, out=None, workspace: torch.Tensor | None = None,
                         stream=None):
    """(dx bf16 [rows, cols], dw fp32 [cols]) of the norm from dy and the h and
    rstd of the forward pass; `dh`: the gradient that reaches h past the norm
    (see include/fp4.h).  `out`: optional preallocated (dx, dw); dx may be dh."""
    return _call(_native().rmsnorm_backward, dy, stream, dy, h, weight, rstd, dh, out, workspace)


def fp4_gemm_decode(aq: torch.Tensor, as_: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor,
                    out: torch.Tensor | None = None, out_dtype: int = OUT_BF16, stream=None):
    """c[M, N] = A W^T for few rows: A MXFP8 (codes and scales of mx8_shapes(M,
    K)) or MXFP4 (of mx_shapes(M, K, AXIS_COLS)), W [N, K] MXFP4 (see
    include/fp4.h)."""
    return _call(_native().gemm_decode, aq, stream, aq, as_, wq, ws, out, out_dtype)


def grouped_shapes(rows: int, cols: int, experts: int, axis: int):
    """(codes shape, scales shape) of fp4_quantize_grouped's outputs for
    x[rows, cols] along `axis`."""
    units = rows // 32 + experts
    if axis == AXIS_COLS:
        return (units, cols // 32, 512), scale_shape(32 * units, cols)
    return (cols // 32, 8 * (rows // 256 + experts), 512), (rows // 256 + experts, cols, 8)


def fp4_quantize_grouped(x: torch.Tensor, offsets: torch.Tensor, axis: int = AXIS_COLS, had_n: int = 32,
                         had: int = HAD_NONE, sign_seed: int = 0, rnd: int = RTN, sr_seed: int = 0, out=None,
                         stream=None):
    """(codes, scales) of bf16 x[rows, cols] with rows grouped by expert
    (offsets int32 [experts + 1], on the GPU), along `axis`, in the shapes of
    grouped_shapes (see include/fp4.h)."""
    if axis not in (AXIS_COLS, AXIS_ROWS):
        raise ValueError("axis must be AXIS_COLS or AXIS_ROWS")
    return _call(_native().quantize_grouped, x, stream, x, offsets, 1 + axis, had_n, had, sign_seed, rnd, sr_seed,
                 sr_seed, out)


def fp4_quantize_grouped_dual(x: torch.Tensor, offsets: torch.Tensor, had_n: int = 32, had: int = HAD_NONE,
                              sign_seed: int = 0, rnd: int = RTN, sr_seed_rows: int = 0, sr_seed_cols: int = 0,
                              out=None, stream=None):
    """Both quantizations of x from one read: (codes, scales) along rows,
    rotated, and (codes, scales) along cols, not rotated."""
    return _call(_native().quantize_grouped, x, stream, x, offsets, 3, had_n, had, sign_seed, rnd, sr_seed_rows,
                 sr_seed_cols, out)


def fp4_gemm_grouped(aq: torch.Tensor, as_: torch.Tensor, offsets: torch.Tensor, wq: torch.Tensor,
                     ws: torch.Tensor, rows: int, out: torch.Tensor | None = None, out_dtype: int = OUT_BF16,
                     stream=None):
    """c[rows, N]: each expert's rows times its weight (see include/fp4.h).
    aq, as_: MXFP4 of fp4_quantize_grouped(x, offsets) or MXFP8 row-major; wq
    [experts, ceil(N/32), K/32, 512] and ws [experts, ceil(K/256), N, 8]: the
    experts' weights, each quantized along its contraction.  Rows of no expert
    are left as they were (in a new tensor: not set)."""
    return _call(_native().gemm_grouped, aq, stream, aq, as_, offsets, wq, ws, rows, out, out_dtype)


def fp4_gemm_grouped_wgrad(dytq: torch.Tensor, dyts: torch.Tensor, xtq: torch.Tensor, xts: torch.Tensor,
                           offsets: torch.Tensor, rows: int, out: torch.Tensor | None = None,
                           out_dtype: int = OUT_BF16, stream=None):
    """dw[experts, N, K] = each expert's dY^T X from dY [rows, N] and X
    [rows, K] quantized along rows by fp4_quantize_grouped with these offsets
    (see include/fp4.h)."""
    return _call(_native().gemm_grouped_wgrad, dytq, stream, dytq, dyts, xtq, xts, offsets, rows, out, out_dtype)


def fp4_quantize_experts(w: torch.Tensor, out=None, stream=None):
    """The weights w bf16 [E, N, K] of a mixture of experts (N and K multiples of
    32) quantized both ways, as fp4_gemm_grouped takes them: (wtq, wts) of W^T for
    Dgrad, (wq, ws) for the forward product, each [E, ...] (see include/fp4.h).
    `out`: optional preallocated (wtq, wts, wq, ws)."""
    if w.dim() != 3:
        raise ValueError("w must be [experts, N, K], got shape %s" % (tuple(w.shape),))
    _need(w, torch.bfloat16, "w")
    E, N, K = w.shape
    shapes = [(E, *s) for s in (code_shape(K, N), scale_shape(K, N), code_shape(N, K), scale_shape(N, K))]
    out = [_empty(s, torch.uint8, w.device, stream) for s in shapes] if out is None else list(out)
    if len(out) != 4:
        raise ValueError("out must be (wtq, wts, wq, ws)")
    for t, s in zip(out, shapes):
        _need(t, torch.uint8, "output")
        if tuple(t.shape) != s or t.device != w.device:
            raise ValueError("output of shape %s on %s expected, got %s on %s" % (s, w.device, tuple(t.shape), t.device))
    with torch.cuda.device(w.device):
        _check(lib().fp4_quantize_experts(w.data_ptr(), E, N, K, *(t.data_ptr() for t in out),
                                          _stream_ptr(stream, w.device)))
    return tuple(out)


def fp4_moe_route(logits: torch.Tensor, k: int, score: int = SCORE_SOFTMAX, normalize: bool = True, out=None,
                  stream=None):
    """(ids int32 [T, k], weights fp32 [T, k]): the k experts of the largest
    logits [T, E] (fp32 or bf16) of each token, largest first, equal ones by
    their index, and their scores, over their sum if `normalize` (see
    include/fp4.h).  Logits of -infinity or NaN are no choice (id -1, weight 0
    where nothing else is left).  `out`: optional preallocated (ids, weights)."""
    return _call(_native().moe_route, logits, stream, logits, k, score, normalize, out)


def fp4_moe_route_backward(dweights: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor,
                           score: int = SCORE_SOFTMAX, normalize: bool = True, out: torch.Tensor | None = None,
                           stream=None):
    """dlogits [T, E] in the type of the logits, from the gradient of
    fp4_moe_route's weights for its ids (see include/fp4.h)."""
    return _call(_native().moe_route_backward, logits, stream, dweights, logits, ids, score, normalize, out)


def fp4_moe_sort_workspace_bytes(slots: int, experts: int) -> int:
    return int(lib().fp4_moe_sort_workspace_bytes(slots, experts))


def fp4_moe_sort(ids: torch.Tensor, experts: int, out=None, workspace: torch.Tensor | None = None, stream=None):
    """Slots sorted by expert from ids int32 [T, k]: (offsets [experts + 1] as the
    grouped operators take them, order [T k] the slot t k + j of each row, position
    [T, k] the row of each slot), int32.  A slot whose id is outside of [0,
    experts) has position -1, and its place in order is behind the last expert's rows.
    `out`: optional preallocated (offsets, order, position)."""
    return _call(_native().moe_sort, ids, stream, ids, experts, out, workspace)


def fp4_moe_gather(x: torch.Tensor, position: torch.Tensor, scales: torch.Tensor | None = None, out=None, stream=None):
    """Tokens to their experts' rows: out[position[t, j]] = x[t] for x bf16
    [T, cols], or MXFP8 codes uint8 [T, cols] with `scales` [T, cols / 32], giving
    (codes, scales).  Rows of no slot are left as they were (in a new tensor of
    T k rows: not set).  `out`: optional tensor, or pair, of any number of rows;
    positions beyond them are no slot's.  The gradient is fp4_moe_combine without
    weights."""
    return _call(_native().moe_gather, x, stream, x, position, scales, out)


def fp4_moe_combine(y: torch.Tensor, position: torch.Tensor, weights: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, stream=None):
    """out[t] = sum over j of weights[t, j] y[position[t, j]]: bf16 [T, cols] of
    the experts' rows y bf16 [rows, cols]; weights fp32 [T, k], all 1 if None (the
    gradient is then fp4_moe_gather)."""
    return _call(_native().moe_combine, y, stream, y, position, weights, out)


def fp4_moe_combine_backward(dout: torch.Tensor, y: torch.Tensor, position: torch.Tensor, weights: torch.Tensor,
                             out=None, stream=None):
    """(dy bf16 [rows, cols], dweights fp32 [T, k]) of fp4_moe_combine with
    weights from dout bf16 [T, cols].  Rows of no slot are left as they were (in
    a new dy: not set).  `out`: optional preallocated (dy, dweights); dy may be y."""
    return _call(_native().moe_combine_backward, y, stream, dout, y, position, weights, out)


def fp4_glu(x: torch.Tensor, act: int = ACT_SILU, weights: torch.Tensor | None = None,
            order: torch.Tensor | None = None, offsets: torch.Tensor | None = None, checkpoint: bool = False, out=None,
            stream=None):
    """The gated activation y[r, c] = w_r act(x[r, c]) x[r, cols + c] of x bf16
    [rows, 2 cols], gate and up side by side (see include/fp4.h): y bf16
    [rows, cols], with `checkpoint` (y, xq, xs), x in MXFP8 (mx8_shapes(rows, 2
    cols)) for fp4_glu_backward.  weights (fp32, one a row in any shape) and order
    (int32, fp4_moe_sort's): w_r = weights[order[r]], or weights[r] without an order.
    offsets (fp4_moe_sort's): rows of no expert are left as they were (in a new
    tensor: not set).  `out`: optional preallocated y, or (y, xq, xs)."""
    return _call(_native().glu, x, stream, x, act, weights, order, offsets, checkpoint, out)


def fp4_glu_quantize(x: torch.Tensor, act: int = ACT_SILU, weights: torch.Tensor | None = None,
                     order: torch.Tensor | None = None, offsets: torch.Tensor | None = None, fmt: int = FMT_MXFP8,
                     out=None, stream=None):
    """fp4_glu with its output quantized along cols: (codes, scales) in `fmt`, as
    fp4_rmsnorm_quantize gives them, for fp4_gemm_decode and fp4_gemm_grouped."""
    return _call(_native().glu_quantize, x, stream, x, act, weights, order, offsets, fmt, out)


def fp4_glu_backward(dy: torch.Tensor, xq: torch.Tensor, xs: torch.Tensor, act: int = ACT_SILU,
                     weights: torch.Tensor | None = None, order: torch.Tensor | None = None,
                     offsets: torch.Tensor | None = None, out=None, stream=None):
    """dx bf16 [rows, 2 cols] of fp4_glu from dy bf16 [rows, cols] and its
    checkpoint, and with weights (dx, dweights fp32 in the shape of weights).  Rows
    of no expert leave dx as it was (in a new tensor: not set) and give 0 in
    dweights.  `out`: optional preallocated dx, or (dx, dweights)."""
    return _call(_native().glu_backward, dy, stream, dy, xq, xs, act, weights, order, offsets, out)


from . import linear, moe  # noqa: E402  (the autograd layers built on the calls above)
