"""The autograd layers on the norm and the grouped products: outputs and every
gradient against the oracle-quantized operands in 64 bits, within the bounds of
their bf16 outputs."""
import numpy as np
import pytest
import torch

import _mx_ref as R
import fp4_precision_gemms_amd as F
import oracle as O
from _grouped import check
from _util import bf16_bits, bits_to_f32, need_gpu, say, to_gpu_bf16

pytestmark = pytest.mark.gpu

SR_COLS = 0x9E3779B97F4A7C15
MODES = {"det_rtn": (F.HAD_DET, 0, F.RTN, 0), "signed_sr": (F.HAD_SIGNED, 1234, F.SR, 77)}


def cols(bits, rnd=F.RTN, seed=0):
    return R.mxfp4_values(*O.quant_mx(bits, O.AXIS_COLS, 32, O.HAD_NONE, 0, rnd, seed))


def rows(bits, had=F.HAD_NONE, sign=0, rnd=F.RTN, seed=0):
    return R.mxfp4_values(*O.quant_mx(bits, O.AXIS_ROWS, 32, had, sign, rnd, seed))


def product(a, b):
    return a @ b.T, np.abs(a) @ np.abs(b).T


def bits_of(t):
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("residual", [True, False])
def test_norm_linear(mode, residual):
    need_gpu()
    T, K, N = 96, 320, 160
    had, sign, rnd, sr = MODES[mode]
    say("norm linear", mode, residual)
    rng = np.random.default_rng(3)
    xb, rb = bf16_bits(rng.standard_normal((T, K))), bf16_bits(rng.standard_normal((T, K)))
    gb, wb = bf16_bits(1 + 0.1 * rng.standard_normal(K)), bf16_bits(rng.standard_normal((N, K)) * 0.02)
    dyb, dhb = bf16_bits(rng.standard_normal((T, N)) * 1e-2), bf16_bits(rng.standard_normal((T, K)) * 1e-2)
    leaves = [to_gpu_bf16(b).requires_grad_(True) for b in (xb, rb, gb, wb)]
    x, r, g, w = leaves
    y, h = F.linear.MXFP4NormLinearFunction.apply(x, r if residual else None, g, w, 1e-5, had, 32, sign, rnd, sr)
    torch.autograd.backward((y, h), (to_gpu_bf16(dyb), to_gpu_bf16(dhb)))
    torch.cuda.synchronize()

    href, rstd, norm = R.rmsnorm(bits_to_f32(xb), bits_to_f32(rb) if residual else None, bits_to_f32(gb), 1e-5)
    assert np.array_equal(h.detach().float().cpu().numpy(), href)
    check(y.detach(), *product(R.mxfp4_values(*R.mxfp4(norm)), cols(wb)))
    normb = bf16_bits(norm)
    check(w.grad, *product(rows(dyb, had, sign, rnd, sr), rows(normb, had, sign)))
    # the gradient at the norm's output, rounded to bf16 as the layer has it,
    # through the norm in 64 bits
    dn, dn_mag = product(cols(dyb, rnd, sr ^ SR_COLS), rows(wb))
    near = 1e-5 * dn_mag
    near = near + 2.0 ** -8 * (np.abs(dn) + near)            # of dn as the layer holds it
    gw, hh, rr = bits_to_f32(gb).astype(np.float64), href.astype(np.float64), rstd.astype(np.float64)[:, None]

    def through(d):
        e = d * gw
        return rr * e - hh * rr ** 3 * (e * hh).mean(1, keepdims=True)

    ref = through(dn) + bits_to_f32(dhb)
    worst = rr * near * np.abs(gw) + np.abs(hh) * rr ** 3 * (near * np.abs(gw * hh)).mean(1, keepdims=True)
    worst = worst + 100 * 2.0 ** -24 * (np.abs(ref) + np.abs(bits_to_f32(dhb)) + rr * np.abs(dn * gw)
                                        + np.abs(hh) * rr ** 3 * np.abs(dn * gw * hh).mean(1, keepdims=True))
    worst = worst + 2.0 ** -8 * (np.abs(ref) + worst)
    assert (np.abs(x.grad.double().cpu().numpy() - ref) <= worst).all()
    if residual:
        assert torch.equal(x.grad, r.grad) and x.grad.data_ptr() != r.grad.data_ptr()
    else:
        assert r.grad is None
    gref = (dn * hh * rr).sum(0)
    gnear = (near * np.abs(hh * rr)).sum(0) + 100 * 2.0 ** -24 * np.abs(dn * hh * rr).sum(0)
    gnear = gnear + 2.0 ** -8 * (np.abs(gref) + gnear)
    assert (np.abs(g.grad.double().cpu().numpy() - gref) <= gnear).all()


def test_norm_linear_without_one_of_its_gradients():
    need_gpu()
    torch.manual_seed(0)
    layer = F.linear.MXFP4NormLinear(64, 96, device="cuda")
    with torch.no_grad():
        layer.weight.normal_(0, 0.05)
    x, r = (torch.randn(32, 64, device="cuda").bfloat16().requires_grad_(True) for _ in range(2))
    y, h = layer(x, r)
    h.float().sum().backward()
    assert torch.equal(x.grad, torch.ones_like(x)) and torch.equal(r.grad, x.grad) and layer.weight.grad is None
    x.grad = r.grad = None
    y, h = layer(x, r)
    y.float().square().sum().backward()
    assert torch.equal(x.grad, r.grad) and torch.isfinite(x.grad).all() and x.grad.abs().max() > 0
    assert layer.norm_weight.grad.shape == (64,) and layer.weight.grad.shape == (96, 64)


@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("T,offsets", [(200, [0, 70, 70, 199, 200]), (416, [0, 400, 416]), (90, [10, 40, 41, 60])])
def test_grouped_linear(mode, T, offsets):
    need_gpu()
    K, N, E = 288, 160, len(offsets) - 1
    had, sign, rnd, sr = MODES[mode]
    say("grouped linear", mode, T, offsets)
    rng = np.random.default_rng(T)
    xb, wb = bf16_bits(rng.standard_normal((T, K))), bf16_bits(rng.standard_normal((E * N, K)) * 0.02)
    dyb = bf16_bits(rng.standard_normal((T, N)) * 1e-2)
    x = to_gpu_bf16(xb).requires_grad_(True)
    w = to_gpu_bf16(wb).view(E, N, K).requires_grad_(True)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    y = F.linear.MXFP4GroupedLinearFunction.apply(x, off, w, True, had, 32, sign, rnd, sr)
    y.backward(to_gpu_bf16(dyb))
    torch.cuda.synchronize()

    stages = T // 256 + E
    def staged(bits, seed=0, rounding=F.RTN):
        full = np.zeros((256 * stages, bits.shape[1]), np.uint16)
        for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
            full[256 * (lo // 256 + e):][:hi - lo] = bits[lo:hi]
        return rows(full, had, sign, rounding, seed)

    xc, dc = cols(xb), cols(dyb, rnd, sr ^ SR_COLS)
    dr, xr = staged(dyb, sr, rnd), staged(xb)
    yref, ymag = np.zeros((T, N)), np.zeros((T, N))
    dref, dmag = np.zeros((T, K)), np.zeros((T, K))
    wref, wmag = np.zeros((E, N, K)), np.zeros((E, N, K))
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        we = wb[e * N:(e + 1) * N]
        yref[lo:hi], ymag[lo:hi] = product(xc[lo:hi], cols(we))
        dref[lo:hi], dmag[lo:hi] = product(dc[lo:hi], rows(we))
        span = slice(256 * (lo // 256 + e), 256 * (lo // 256 + e) + (hi - lo + 31) // 32 * 32)
        wref[e], wmag[e] = product(dr[:, span], xr[:, span])
    check(y.detach(), yref, ymag)
    check(x.grad, dref, dmag)
    check(w.grad, wref, wmag)


def test_grouped_linear_approximates_the_unquantized_layers():
    need_gpu()
    torch.manual_seed(1)
    E, K, N, T = 3, 128, 96, 128
    layer = F.linear.MXFP4GroupedLinear(E, K, N, device="cuda")
    with torch.no_grad():
        layer.weight.normal_(0, 0.05)
    x = torch.randn(T, K, device="cuda").bfloat16().requires_grad_(True)
    off = torch.tensor([0, 50, 50, T], dtype=torch.int32, device="cuda")
    y = layer(x, off)
    y.float().square().sum().backward()
    exact = torch.cat([x[:50].detach().double() @ layer.weight[0].detach().double().T,
                       x[50:].detach().double() @ layer.weight[2].detach().double().T])
    assert float((y.detach().double() - exact).norm() / exact.norm()) < 0.2
    assert not layer.weight.grad[1].any() and layer.weight.grad[0].any() and torch.isfinite(x.grad).all()


def test_a_block_of_experts_captured_and_replayed():
    """norm to MXFP4 and MXFP8, grouped quantizers, products and gradients as
    one graph, replayed with other inputs and other splits in the same
    buffers, eager work between: the same bits as the eager calls."""
    need_gpu()
    T, K, N, E = 160, 256, 128, 5
    torch.manual_seed(2)
    x, r, dy = (torch.randn(T, n, device="cuda").bfloat16() for n in (K, K, N))
    g = torch.ones(K, device="cuda").bfloat16()
    w = (torch.randn(E, N, K, device="cuda") * 0.05).bfloat16()
    off = torch.tensor([0, 30, 30, 100, 150, 160], dtype=torch.int32, device="cuda")
    wtq, wts, wq, ws = F.linear.quantize_experts(w)

    def step():
        n = torch.empty_like(x)
        q8, s8, h, rstd = F.fp4_rmsnorm_quantize(x, g, r, y=n)
        y8 = F.fp4_gemm_grouped(q8, s8, off, wq, ws, T)
        xtq, xts, xq, xs = F.fp4_quantize_grouped_dual(n, off, 32, F.HAD_DET)
        y = F.fp4_gemm_grouped(xq, xs, off, wq, ws, T)
        dytq, dyts, dyq, dys = F.fp4_quantize_grouped_dual(dy, off, 32, F.HAD_DET)
        dn = F.fp4_gemm_grouped(dyq, dys, off, wtq, wts, T)
        dw = F.fp4_gemm_grouped_wgrad(dytq, dyts, xtq, xts, off, T)
        return (h, y8, y, dn, dw) + F.fp4_rmsnorm_backward(dn, h, g, rstd)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = step()
    for i, split in enumerate(([0, 30, 30, 100, 150, 160], [0, 0, 0, 1, 159, 160], [0, 160, 160, 160, 160, 160])):
        off.copy_(torch.tensor(split, dtype=torch.int32))
        x.mul_(1.25)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(caught, step()):
            assert torch.equal(a, b), i
