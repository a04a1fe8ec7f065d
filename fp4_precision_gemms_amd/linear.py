"""An MXFP4 linear layer as a torch autograd Function: Fprop, Dgrad and
Wgrad on the scaled FP4 matrix cores, wired the way the pages describe.

[AMD-MXFP4] "Pretraining large language models with MXFP4 on Native FP4
Hardware", section "Поисковая экспериментальная работа: корень
нестабильности": the three GEMMs of a linear layer run in MXFP4 --

    Fprop  Y  = X W^T      X along K, W along K      (no rotation)
    Dgrad  dX = dY W       dY along N, W^T along N   (no rotation)
    Wgrad  dW = dY^T X     dY^T, X^T along T         (block Hadamard on both)

-- and the rotation is applied only to the Wgrad operands, the same
transform on both so that it cancels in dY^T X.

Every operand is quantized once per direction by the dual quantizer (one
read of X, of W and of dY each); forward keeps only the quantized operands
backward needs (X^T and W^T codes), not the bf16 tensors.  Inputs and the
weight are bf16; Y, dX and dW are returned in bf16 (each the fp32 GEMM
result rounded to nearest even by the GEMM kernel).  This module only
sequences library calls; all arithmetic runs in libfp4.so.

MXFP4NormLinear puts the norm that feeds such a layer in front of it (residual
added, output quantized without a pass of its own), MXFP4GroupedLinear is the
layer of a mixture of experts: rows sorted by expert, one weight each.

Captured into a HIP graph, a layer's forward and backward pass go into the same
capture, after a warm-up on the capturing stream and with no eager graph of its
parameters alive (torch's gradient accumulation would wait for the stream of
that one).

The gradients have none of their own: torch refuses a backward pass that reaches a
layer's gradient (once_differentiable).
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (AXIS_ROWS, FMT_MXFP4, HAD_DET, HAD_NONE, OUT_BF16, RTN, code_shape, fp4_gemm_grouped,
               fp4_gemm_grouped_wgrad, fp4_gemm_mx, fp4_hadamard_quantize, fp4_hadamard_quantize_dual,
               fp4_quantize_experts, fp4_quantize_grouped_dual, fp4_rmsnorm_backward, fp4_rmsnorm_quantize, scale_shape)

_SR_COLS = 0x9E3779B97F4A7C15      # tells the SR stream of the Dgrad operand from the Wgrad one's


class MXFP4LinearFunction(torch.autograd.Function):
    """y = x w^T with x [T, K], w [N, K] (both bf16, T and K multiples of 32,
    N a multiple of 32), all three GEMMs in MXFP4."""

    @staticmethod
    def forward(ctx, x, w, had: int = HAD_DET, had_n: int = 32, sign_seed: int = 0,
                grad_rounding: int = RTN, sr_seed: int = 0):
        x = x.contiguous()
        w = w.contiguous()
        # X: along rows (X^T, Wgrad, rotated) and along cols (Fprop)
        xtq, xts, xq, xs = fp4_hadamard_quantize_dual(x, had_n, had, sign_seed, RTN, 0,
                                                      32, HAD_NONE, 0, RTN, 0)
        # W [N, K]: along rows (W^T, Dgrad) and along cols (Fprop)
        wtq, wts, wq, ws = fp4_hadamard_quantize_dual(w, 32, HAD_NONE, 0, RTN, 0,
                                                      32, HAD_NONE, 0, RTN, 0)
        y = fp4_gemm_mx(xq, xs, wq, ws, out_dtype=OUT_BF16)
        ctx.save_for_backward(xtq, xts, wtq, wts)
        ctx.cfg = (had, had_n, sign_seed, grad_rounding, sr_seed)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        xtq, xts, wtq, wts = ctx.saved_tensors
        had, had_n, sign_seed, grad_rounding, sr_seed = ctx.cfg
        dy = dy.to(torch.bfloat16).contiguous()
        # dY: along rows (dY^T, Wgrad, the same rotation as X^T) and along cols
        # (Dgrad); the gradient may be rounded stochastically
        dytq, dyts, dyq, dys = fp4_hadamard_quantize_dual(dy, had_n, had, sign_seed, grad_rounding,
                                                          sr_seed, 32, HAD_NONE, 0, grad_rounding,
                                                          sr_seed ^ _SR_COLS)
        dx = fp4_gemm_mx(dyq, dys, wtq, wts, out_dtype=OUT_BF16)       # [T, K]
        dw = fp4_gemm_mx(dytq, dyts, xtq, xts, out_dtype=OUT_BF16)     # [N, K]
        return dx, dw, None, None, None, None, None


class MXFP4Linear(torch.nn.Module):
    """A bias-free linear layer whose three GEMMs run in MXFP4.  `sign_seed`
    selects the random-sign Hadamard when had = HAD_SIGNED (change it per
    step for a per-step random rotation)."""

    def __init__(self, in_features: int, out_features: int, had: int = HAD_DET, had_n: int = 32,
                 grad_rounding: int = RTN, device=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.empty(out_features, in_features,
                                                     dtype=torch.bfloat16, device=device))
        self.had, self.had_n, self.grad_rounding = had, had_n, grad_rounding
        self.sign_seed = 0
        self.sr_seed = 0

    def forward(self, x):
        return MXFP4LinearFunction.apply(x, self.weight, self.had, self.had_n, self.sign_seed,
                                         self.grad_rounding, self.sr_seed)


class MXFP4NormLinearFunction(torch.autograd.Function):
    """(y, h) with h = x + residual and y = rmsnorm(h) w^T: x and residual
    [T, K], norm weight [K], w [N, K] (all bf16, T, K and N multiples of 32).
    The norm leaves its output quantized for Fprop; Wgrad's operand is
    quantized from the norm rounded to bf16, rotated.  Both roundings are
    passed straight through to the norm's gradient."""

    @staticmethod
    def forward(ctx, x, residual, norm_weight, w, eps: float = 1e-5, had: int = HAD_DET, had_n: int = 32,
                sign_seed: int = 0, grad_rounding: int = RTN, sr_seed: int = 0):
        ctx.set_materialize_grads(False)
        x, w = x.contiguous(), w.contiguous()
        residual = None if residual is None else residual.contiguous()
        n = torch.empty_like(x)
        nq, ns, h, rstd = fp4_rmsnorm_quantize(x, norm_weight, residual, eps, FMT_MXFP4, y=n)
        ntq, nts = fp4_hadamard_quantize(n, AXIS_ROWS, had_n, had, sign_seed)
        wtq, wts, wq, ws = fp4_hadamard_quantize_dual(w)
        y = fp4_gemm_mx(nq, ns, wq, ws, out_dtype=OUT_BF16)
        ctx.save_for_backward(h, rstd, norm_weight, ntq, nts, wtq, wts)
        ctx.cfg = (residual is not None, had, had_n, sign_seed, grad_rounding, sr_seed)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        h, rstd, norm_weight, ntq, nts, wtq, wts = ctx.saved_tensors
        added, had, had_n, sign_seed, grad_rounding, sr_seed = ctx.cfg
        dh = None if dh is None else dh.to(torch.bfloat16).contiguous()
        if dy is None:                 # y took no part
            return (dh, dh if added else None) + (None,) * 8
        dy = dy.to(torch.bfloat16).contiguous()
        dytq, dyts, dyq, dys = fp4_hadamard_quantize_dual(dy, had_n, had, sign_seed, grad_rounding, sr_seed,
                                                          rnd_cols=grad_rounding, sr_seed_cols=sr_seed ^ _SR_COLS)
        dn = fp4_gemm_mx(dyq, dys, wtq, wts, out_dtype=OUT_BF16)
        dw = fp4_gemm_mx(dytq, dyts, ntq, nts, out_dtype=OUT_BF16)
        dx, dnorm = fp4_rmsnorm_backward(dn, h, norm_weight, rstd, dh)
        return (dx, dx if added else None, dnorm.to(norm_weight.dtype), dw) + (None,) * 6


class MXFP4NormLinear(torch.nn.Module):
    """Residual addition, root-mean-square norm and a bias-free MXFP4 linear
    layer: forward(x, residual) gives (y, h), h the new residual stream."""

    def __init__(self, in_features: int, out_features: int, eps: float = 1e-5, had: int = HAD_DET, had_n: int = 32,
                 grad_rounding: int = RTN, device=None):
        super().__init__()
        self.norm_weight = torch.nn.Parameter(torch.ones(in_features, dtype=torch.bfloat16, device=device))
        self.weight = torch.nn.Parameter(torch.empty(out_features, in_features, dtype=torch.bfloat16, device=device))
        self.eps, self.had, self.had_n, self.grad_rounding = eps, had, had_n, grad_rounding
        self.sign_seed = 0
        self.sr_seed = 0

    def forward(self, x, residual=None):
        return MXFP4NormLinearFunction.apply(x, residual, self.norm_weight, self.weight, self.eps, self.had,
                                             self.had_n, self.sign_seed, self.grad_rounding, self.sr_seed)


def quantize_experts(w: torch.Tensor):
    """Both operands of each of the experts' weights w [E, N, K] (bf16, N and K
    multiples of 32), as fp4_gemm_grouped takes them: (wtq, wts) for Dgrad,
    (wq, ws) for the forward product.  Any number of experts of any size: what
    one fp4_quantize_experts does not take goes in several calls."""
    w = w.contiguous()
    E, N, K = w.shape
    whole = N < 2 ** 22 and K < 2 ** 24
    if whole and 1 <= E <= 1024:
        return fp4_quantize_experts(w)
    shapes = (code_shape(K, N), scale_shape(K, N), code_shape(N, K), scale_shape(N, K))
    out = tuple(torch.empty((E, *s), dtype=torch.uint8, device=w.device) for s in shapes)
    for e in range(0, E, 1024 if whole else 1):
        if whole:
            fp4_quantize_experts(w[e:e + 1024], out=[t[e:e + 1024] for t in out])
        else:
            fp4_hadamard_quantize_dual(w[e], out=[t[e] for t in out])
    return out


class MXFP4GroupedLinearFunction(torch.autograd.Function):
    """y[r] = x[r] w[e]^T for the rows r of expert e: x [T, K] with rows sorted
    by expert, offsets int32 [E + 1], w [E, N, K] (bf16, N and K multiples of
    32).  Rows of no expert give zero rows of y and of x's gradient if `padded`
    (else those are not set), and reach no weight."""

    @staticmethod
    def forward(ctx, x, offsets, w, padded: bool = False, had: int = HAD_DET, had_n: int = 32, sign_seed: int = 0,
                grad_rounding: int = RTN, sr_seed: int = 0):
        x, w = x.contiguous(), w.contiguous()
        xtq, xts, xq, xs = fp4_quantize_grouped_dual(x, offsets, had_n, had, sign_seed)
        wtq, wts, wq, ws = quantize_experts(w)
        y = fp4_gemm_grouped(xq, xs, offsets, wq, ws, x.shape[0], out=_rows(x, w.shape[1], padded))
        ctx.save_for_backward(offsets, xtq, xts, wtq, wts)
        ctx.cfg = (x.shape[0], w.shape[2], padded, had, had_n, sign_seed, grad_rounding, sr_seed)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        offsets, xtq, xts, wtq, wts = ctx.saved_tensors
        rows, K, padded, had, had_n, sign_seed, grad_rounding, sr_seed = ctx.cfg
        dy = dy.to(torch.bfloat16).contiguous()
        dytq, dyts, dyq, dys = fp4_quantize_grouped_dual(dy, offsets, had_n, had, sign_seed, grad_rounding, sr_seed,
                                                         sr_seed ^ _SR_COLS)
        dx = fp4_gemm_grouped(dyq, dys, offsets, wtq, wts, rows, out=_rows(dy, K, padded))
        dw = fp4_gemm_grouped_wgrad(dytq, dyts, xtq, xts, offsets, rows)
        return dx, None, dw, None, None, None, None, None, None


def _rows(like: torch.Tensor, cols: int, padded: bool) -> torch.Tensor:
    return (like.new_zeros if padded else like.new_empty)((like.shape[0], cols))


class MXFP4GroupedLinear(torch.nn.Module):
    """The bias-free linear layers of `experts` experts, whose products run in
    MXFP4: forward(x, offsets) with the rows of x sorted by expert.  `padded`:
    x may hold rows of no expert (see MXFP4GroupedLinearFunction)."""

    def __init__(self, experts: int, in_features: int, out_features: int, padded: bool = False, had: int = HAD_DET,
                 had_n: int = 32, grad_rounding: int = RTN, device=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.empty(experts, out_features, in_features, dtype=torch.bfloat16,
                                                     device=device))
        self.padded, self.had, self.had_n, self.grad_rounding = padded, had, had_n, grad_rounding
        self.sign_seed = 0
        self.sr_seed = 0

    def forward(self, x, offsets):
        return MXFP4GroupedLinearFunction.apply(x, offsets, self.weight, self.padded, self.had, self.had_n,
                                                self.sign_seed, self.grad_rounding, self.sr_seed)
