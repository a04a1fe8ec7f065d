"""A mixture of experts with a gated activation on the library's calls: router,
tokens sorted by expert, the experts' two MXFP4 products with the activation
between them, and the way back to the tokens.

Training (MXFP4MoE): out[t] = sum over token t's experts e of
w[t, e] W2_e (act(G_e x[t]) * (U_e x[t])), W1_e = [G_e; U_e].  All six products run in
MXFP4 as in MXFP4GroupedLinear.  The weights are applied to the activation, not
to the second product's rows: since that product is linear the output is the
same, and the weights' gradient, sum_c dy[c] act(g)[c] u[c], needs none of its
rows.  Kept for the backward pass: the products' operands in 4 bits and the
activation's input in 8 (MXFP8), no tensor of the experts' rows in bf16.

Serving (moe_decode): the same from 8-bit rows, as fp4_rmsnorm_quantize leaves
them, through the few-row products.

Captured into a HIP graph, forward and backward pass go into the same capture,
after a warm-up on the capturing stream and with no eager graph of its parameters
alive, as for the layers of linear.py.  The gradients have none of their own, as there.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (ACT_SILU, HAD_DET, RTN, SCORE_SOFTMAX, fp4_gemm_grouped, fp4_gemm_grouped_wgrad, fp4_glu,
               fp4_glu_backward, fp4_glu_quantize, fp4_moe_combine, fp4_moe_gather, fp4_moe_route,
               fp4_moe_route_backward, fp4_moe_sort, fp4_quantize_grouped_dual)
from .linear import _SR_COLS, quantize_experts

_SR_SECOND = 0xD1B54A32D192ED03     # tells the SR streams of the second product from the first one's


class RouteFunction(torch.autograd.Function):
    """(ids, weights) of fp4_moe_route, differentiable in the logits by the weights."""

    @staticmethod
    def forward(ctx, logits, k: int, score: int = SCORE_SOFTMAX, normalize: bool = True):
        logits = logits.contiguous()
        ids, weights = fp4_moe_route(logits, k, score, normalize)
        ctx.save_for_backward(logits, ids)
        ctx.cfg = (score, normalize)
        ctx.mark_non_differentiable(ids)
        return ids, weights

    @staticmethod
    @once_differentiable
    def backward(ctx, _, dweights):
        logits, ids = ctx.saved_tensors
        return fp4_moe_route_backward(dweights.float().contiguous(), logits, ids, *ctx.cfg), None, None, None


class MXFP4MoEFunction(torch.autograd.Function):
    """out [T, C] of x [T, C] (bf16), ids int32 [T, k], weights fp32 [T, k], w1
    [E, 2 I, C] (gate rows, then up rows) and w2 [E, C, I] (bf16; C and I multiples
    of 32).  A slot whose id is outside of [0, E) adds nothing."""

    @staticmethod
    def forward(ctx, x, ids, weights, w1, w2, act: int = ACT_SILU, had: int = HAD_DET, had_n: int = 32,
                sign_seed: int = 0, grad_rounding: int = RTN, sr_seed: int = 0):
        x, ids, weights, w1, w2 = (t.contiguous() for t in (x, ids, weights, w1, w2))
        offsets, order, position = fp4_moe_sort(ids, w1.shape[0])
        slots = order.shape[0]
        xtq, xts, xq, xs = fp4_quantize_grouped_dual(fp4_moe_gather(x, position), offsets, had_n, had, sign_seed)
        w1tq, w1ts, w1q, w1s = quantize_experts(w1)
        gate_up = fp4_gemm_grouped(xq, xs, offsets, w1q, w1s, slots)
        y, kept, kept_scales = fp4_glu(gate_up, act, weights, order, offsets, checkpoint=True)
        ytq, yts, yq, ys = fp4_quantize_grouped_dual(y, offsets, had_n, had, sign_seed)
        w2tq, w2ts, w2q, w2s = quantize_experts(w2)
        out = fp4_moe_combine(fp4_gemm_grouped(yq, ys, offsets, w2q, w2s, slots), position)
        ctx.save_for_backward(weights, offsets, order, position, xtq, xts, w1tq, w1ts, kept, kept_scales, ytq, yts,
                              w2tq, w2ts)
        ctx.cfg = (act, had, had_n, sign_seed, grad_rounding, sr_seed)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        (weights, offsets, order, position, xtq, xts, w1tq, w1ts, kept, kept_scales, ytq, yts, w2tq,
         w2ts) = ctx.saved_tensors
        act, had, had_n, sign_seed, grad_rounding, sr_seed = ctx.cfg
        slots = order.shape[0]

        def operands(d, seed):
            """A gradient's rows for Wgrad (rotated) and for Dgrad."""
            return fp4_quantize_grouped_dual(d, offsets, had_n, had, sign_seed, grad_rounding, seed, seed ^ _SR_COLS)

        dztq, dzts, dzq, dzs = operands(fp4_moe_gather(dout.to(torch.bfloat16).contiguous(), position),
                                        sr_seed ^ _SR_SECOND)
        dw2 = fp4_gemm_grouped_wgrad(dztq, dzts, ytq, yts, offsets, slots)
        dy = fp4_gemm_grouped(dzq, dzs, offsets, w2tq, w2ts, slots)
        dgate_up, dweights = fp4_glu_backward(dy, kept, kept_scales, act, weights, order, offsets)
        dtq, dts, dq, ds = operands(dgate_up, sr_seed)
        dw1 = fp4_gemm_grouped_wgrad(dtq, dts, xtq, xts, offsets, slots)
        dx = fp4_moe_combine(fp4_gemm_grouped(dq, ds, offsets, w1tq, w1ts, slots), position)
        return (dx, None, dweights, dw1, dw2) + (None,) * 6


class MXFP4MoE(torch.nn.Module):
    """`experts` experts of a gated activation, k of them a token: forward(x,
    logits) with x [T, in_features] (bf16) and the router's logits [T, experts]
    (fp32 or bf16).  T is at least 1: a batch without tokens is refused
    (FP4_ERR_SHAPE), as a size of 0 is by every call."""

    def __init__(self, experts: int, k: int, in_features: int, inner: int, act: int = ACT_SILU,
                 score: int = SCORE_SOFTMAX, normalize: bool = True, had: int = HAD_DET, had_n: int = 32,
                 grad_rounding: int = RTN, device=None):
        super().__init__()
        bf = dict(dtype=torch.bfloat16, device=device)
        self.gate_up = torch.nn.Parameter(torch.empty(experts, 2 * inner, in_features, **bf))
        self.down = torch.nn.Parameter(torch.empty(experts, in_features, inner, **bf))
        self.k, self.act, self.score, self.normalize = k, act, score, normalize
        self.had, self.had_n, self.grad_rounding = had, had_n, grad_rounding
        self.sign_seed = 0
        self.sr_seed = 0

    def forward(self, x, logits):
        ids, weights = RouteFunction.apply(logits, self.k, self.score, self.normalize)
        return MXFP4MoEFunction.apply(x, ids, weights, self.gate_up, self.down, self.act, self.had, self.had_n,
                                      self.sign_seed, self.grad_rounding, self.sr_seed)


def moe_decode(codes: torch.Tensor, scales: torch.Tensor, logits: torch.Tensor, k: int, w1q: torch.Tensor,
               w1s: torch.Tensor, w2q: torch.Tensor, w2s: torch.Tensor, act: int = ACT_SILU,
               score: int = SCORE_SOFTMAX, normalize: bool = True) -> torch.Tensor:
    """The layer for a few tokens: MXFP8 rows (codes [T, C], scales [T, C / 32], as
    fp4_rmsnorm_quantize writes them) to bf16 [T, C].  w1q, w1s / w2q, w2s: the
    experts' weights [E, 2 I, C] and [E, C, I] as fp4_gemm_grouped takes them (the
    last two of quantize_experts).  The weights go to the second product's rows
    here, in binary32.  At least one token, as for the layer."""
    ids, weights = fp4_moe_route(logits, k, score, normalize)
    offsets, _, position = fp4_moe_sort(ids, w1q.shape[0])
    aq, as_ = fp4_moe_gather(codes, position, scales)
    rows = aq.shape[0]
    bq, bs = fp4_glu_quantize(fp4_gemm_grouped(aq, as_, offsets, w1q, w1s, rows), act, offsets=offsets)
    return fp4_moe_combine(fp4_gemm_grouped(bq, bs, offsets, w2q, w2s, rows), position, weights)
