"""The mixture of experts as a layer and as a decode step: the public calls one
after another, near the unquantized layer, captured and replayed, on other
streams and while the caller's tensors are not contiguous."""
import pytest
import torch

import fp4_precision_gemms_amd as F
from _util import need_gpu, say

pytestmark = pytest.mark.gpu

T, E, K, C, I = 150, 6, 3, 96, 160


def leaves(seed=0, tokens=T, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, C, device="cuda", generator=g).bfloat16()
    logits = torch.randn(tokens, E, device="cuda", generator=g)
    w1 = (torch.randn(E, 2 * I, C, device="cuda", generator=g) * 0.1 * scale).bfloat16()
    w2 = (torch.randn(E, C, I, device="cuda", generator=g) * 0.08 * scale).bfloat16()
    return [t.requires_grad_(True) for t in (x, logits, w1, w2)], g


def dense(x, logits, w1, w2, act, score, normalize):
    """The unquantized layer in 64 bits, every expert on every token."""
    x, logits, w1, w2 = (t.detach().double().cpu().requires_grad_(True) for t in (x, logits, w1, w2))
    a = torch.softmax(logits, 1) if score == F.SCORE_SOFTMAX else torch.sigmoid(logits)
    top, ids = torch.topk(a, K, 1)
    w = top / top.sum(1, keepdim=True) if normalize else top
    full = torch.zeros_like(a).scatter(1, ids, w)
    h = torch.einsum("tc,enc->ten", x, w1)
    gate = h[..., :I]
    y = (torch.nn.functional.silu(gate) if act == F.ACT_SILU else torch.nn.functional.gelu(gate, approximate="tanh")) * h[..., I:]
    return (x, logits, w1, w2), torch.einsum("ten,ecn,te->tc", y, w2, full)


@pytest.mark.parametrize("act", [F.ACT_SILU, F.ACT_GELU])
@pytest.mark.parametrize("score,normalize", [(F.SCORE_SOFTMAX, True), (F.SCORE_SOFTMAX, False), (F.SCORE_SIGMOID, True)])
def test_layer_is_near_the_unquantized_one(act, score, normalize):
    """A 4-bit operand is off by about 12 % of its norm (its scale to a power of
    two, a quarter step's rounding), a product of two by 17 %.  The output has two
    products one after another and the gate's product twice: sqrt(4) 17 %; the
    gradients one or two more: sqrt(6) 17 %.  A wrong wiring is off by 100 %."""
    need_gpu()
    say("moe layer", act, score, normalize)
    (x, logits, w1, w2), g = leaves()
    layer = F.moe.MXFP4MoE(E, K, C, I, act, score, normalize, device="cuda")
    with torch.no_grad():
        layer.gate_up.copy_(w1)
        layer.down.copy_(w2)
    out = layer(x, logits)
    d = torch.randn(out.shape, device="cuda", generator=g).bfloat16()
    out.backward(d)
    ref, want = dense(x, logits, w1, w2, act, score, normalize)
    want.backward(d.double().cpu())
    want = want.detach()
    off = float((out.detach().double().cpu() - want).norm() / want.norm())
    assert off < 0.34, off
    for name, got, r in zip(("x", "logits", "w1", "w2"), (x.grad, logits.grad, layer.gate_up.grad, layer.down.grad), ref):
        assert got.dtype == (torch.float32 if name == "logits" else torch.bfloat16)
        off = float((got.double().cpu() - r.grad).norm() / r.grad.norm())
        assert off < 0.42, (name, off)


@pytest.mark.parametrize("rnd,seed", [(F.RTN, 0), (F.SR, 77)])
def test_layer_is_its_calls_one_after_another(rnd, seed):
    """Bit for bit, some slots of no expert."""
    need_gpu()
    (x, logits, w1, w2), g = leaves(1)
    with torch.no_grad():
        logits[::9] = -float("inf")
        logits[1::9, :E - 1] = -float("inf")
    d = torch.randn(T, C, device="cuda", generator=g).bfloat16()
    ids, w = F.moe.RouteFunction.apply(logits, K)
    out = F.moe.MXFP4MoEFunction.apply(x, ids, w, w1, w2, F.ACT_SILU, F.HAD_SIGNED, 32, 5, rnd, seed)
    out.backward(d)
    with torch.no_grad():
        off, order, pos = F.fp4_moe_sort(ids, E)
        n = order.numel()
        assert int(off[-1]) < n
        q1, q2 = F.linear.quantize_experts(w1), F.linear.quantize_experts(w2)
        a = F.fp4_quantize_grouped_dual(F.fp4_moe_gather(x, pos), off, 32, F.HAD_SIGNED, 5)
        h = F.fp4_gemm_grouped(*a[2:], off, *q1[2:], n)
        y, hq, hs = F.fp4_glu(h, F.ACT_SILU, w, order, off, checkpoint=True)
        b = F.fp4_quantize_grouped_dual(y, off, 32, F.HAD_SIGNED, 5)
        z = F.fp4_gemm_grouped(*b[2:], off, *q2[2:], n)
        assert torch.equal(out, F.fp4_moe_combine(z, pos))
        s2 = seed ^ 0xD1B54A32D192ED03
        dz = F.fp4_quantize_grouped_dual(F.fp4_moe_gather(d, pos), off, 32, F.HAD_SIGNED, 5, rnd, s2, s2 ^ 0x9E3779B97F4A7C15)
        assert torch.equal(w2.grad, F.fp4_gemm_grouped_wgrad(*dz[:2], *b[:2], off, n))
        dh, dw = F.fp4_glu_backward(F.fp4_gemm_grouped(*dz[2:], off, *q2[:2], n), hq, hs, F.ACT_SILU, w, order, off)
        dq = F.fp4_quantize_grouped_dual(dh, off, 32, F.HAD_SIGNED, 5, rnd, seed, seed ^ 0x9E3779B97F4A7C15)
        assert torch.equal(w1.grad, F.fp4_gemm_grouped_wgrad(*dq[:2], *a[:2], off, n))
        assert torch.equal(x.grad, F.fp4_moe_combine(F.fp4_gemm_grouped(*dq[2:], off, *q1[:2], n), pos))
        assert torch.equal(logits.grad, F.fp4_moe_route_backward(dw, logits, ids))
        assert not out[::9].any() and not x.grad[::9].any() and not logits.grad[::9].any() and not dw[ids < 0].any()


def test_weights_here_or_at_the_combination():
    """The weights at the activation or at the second product's rows: the same
    layer, apart from the roundings of bf16 and of the 4-bit operand, which a
    power of two does not change."""
    need_gpu()
    (x, logits, w1, w2), _ = leaves(2)
    with torch.no_grad():
        ids, w = F.fp4_moe_route(logits, K)
        w = torch.exp2(-torch.arange(K, device="cuda").float()).expand(T, K).contiguous()
        off, order, pos = F.fp4_moe_sort(ids, E)
        n = order.numel()
        q1, q2 = F.linear.quantize_experts(w1), F.linear.quantize_experts(w2)
        h = F.fp4_gemm_grouped(*F.fp4_quantize_grouped(F.fp4_moe_gather(x, pos), off), off, *q1[2:], n)
        here = F.fp4_gemm_grouped(*F.fp4_quantize_grouped(F.fp4_glu(h, 0, w, order, off), off), off, *q2[2:], n)
        there = F.fp4_gemm_grouped(*F.fp4_quantize_grouped(F.fp4_glu(h, 0), off), off, *q2[2:], n)
        a, b = F.fp4_moe_combine(here, pos), F.fp4_moe_combine(there, pos, w)
    assert torch.equal(a, b)


@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_decode_step(tokens):
    need_gpu()
    say("moe decode", tokens)
    (x, logits, w1, w2), _ = leaves(3, tokens)
    with torch.no_grad():
        q1, q2 = F.linear.quantize_experts(w1), F.linear.quantize_experts(w2)
        codes, scales, _, _ = F.fp4_rmsnorm_quantize(x, torch.ones(C, device="cuda").bfloat16())
        got = F.moe.moe_decode(codes, scales, logits, K, *q1[2:], *q2[2:])
        ids, w = F.fp4_moe_route(logits, K)
        # every token by itself, an expert at a time, through the products without groups
        for t in range(tokens):
            acc = torch.zeros(C, device="cuda")
            for e, we in zip(ids[t].tolist(), w[t]):
                h = F.fp4_gemm_decode(codes[t:t + 1].clone(), scales[t:t + 1].clone(), q1[2][e], q1[3][e])
                z = F.fp4_gemm_decode(*F.fp4_glu_quantize(h), q2[2][e], q2[3][e])
                acc = acc + we * z[0].float()
            near = 2.0 ** -7 * acc.abs() + 2.0 ** -5 * acc.abs().max()   # other orders of the products' sums, then bf16 and 8 bits
            assert ((got[t].float() - acc).abs() <= near).all()


def test_tensors_that_are_not_contiguous():
    need_gpu()
    (x, logits, w1, w2), g = leaves(4)
    ref = F.moe.MXFP4MoE(E, K, C, I, device="cuda")
    with torch.no_grad():
        ref.gate_up.copy_(w1)
        ref.down.copy_(w2)
    out = ref(x, logits)
    d = torch.randn(T, C, device="cuda", generator=g).bfloat16()
    out.backward(d)
    x2 = torch.stack((x.detach(), x.detach()), 1)[:, 1].requires_grad_(True)
    l2 = logits.detach().t().contiguous().t().requires_grad_(True)
    out2 = ref(x2, l2)
    out2.backward(d.t().contiguous().t())
    assert torch.equal(out, out2) and torch.equal(x.grad, x2.grad) and torch.equal(logits.grad, l2.grad)


def test_captured_and_replayed():
    """Forward and backward as one graph, replayed with other inputs in the same
    buffers, eager work between: the same bits as the eager calls."""
    need_gpu()
    (x, logits, w1, w2), g = leaves(5)
    x, logits, w1, w2 = (t.detach() for t in (x, logits, w1, w2))
    d = torch.randn(T, C, device="cuda", generator=g).bfloat16()
    q1, q2 = F.linear.quantize_experts(w1), F.linear.quantize_experts(w2)

    def step():
        ids, w = F.fp4_moe_route(logits, K)
        off, order, pos = F.fp4_moe_sort(ids, E)
        n = order.numel()
        a = F.fp4_quantize_grouped_dual(F.fp4_moe_gather(x, pos), off)
        y, hq, hs = F.fp4_glu(F.fp4_gemm_grouped(*a[2:], off, *q1[2:], n), 0, w, order, off, checkpoint=True)
        b = F.fp4_quantize_grouped_dual(y, off)
        z = F.fp4_gemm_grouped(*b[2:], off, *q2[2:], n)
        out = F.fp4_moe_combine(z, pos)
        weighted = F.fp4_moe_combine(z, pos, w)
        dz, dw0 = F.fp4_moe_combine_backward(d, z, pos, w)
        dy = F.fp4_gemm_grouped(*F.fp4_quantize_grouped(dz, off), off, *q2[:2], n)
        dh, dw = F.fp4_glu_backward(dy, hq, hs, 0, w, order, off)
        dl = F.fp4_moe_route_backward(dw, logits, ids)
        dx = F.fp4_moe_combine(F.fp4_gemm_grouped(*F.fp4_quantize_grouped(dh, off), off, *q1[:2], n), pos)
        c8, s8, _, _ = F.fp4_rmsnorm_quantize(x, torch.ones(C, device="cuda").bfloat16())
        served = F.moe.moe_decode(c8, s8, logits, K, *q1[2:], *q2[2:])
        return ids, w, off, order, pos, out, weighted, dw0, dw, dl, dx, served

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = step()
    for i in range(4):
        logits.copy_(torch.randn(T, E, device="cuda", generator=g))
        x.mul_(1.25)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(caught, step()):
            assert torch.equal(a, b), i
        torch.cuda.synchronize()


def test_layer_captured_forward_and_backward():
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(6)
    layer = F.moe.MXFP4MoE(E, K, C, I, device="cuda")
    with torch.no_grad():
        layer.gate_up.normal_(0, 0.1, generator=g)
        layer.down.normal_(0, 0.1, generator=g)
    x = torch.randn(T, C, device="cuda", generator=g).bfloat16().requires_grad_(True)
    logits = torch.randn(T, E, device="cuda", generator=g).requires_grad_(True)
    d = torch.randn(T, C, device="cuda", generator=g).bfloat16()
    wanted = (x, logits, layer.gate_up, layer.down)

    def step():
        out = layer(x, logits)
        return (out.detach(),) + torch.autograd.grad(out, wanted, d)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = step()
    for i in range(3):
        with torch.no_grad():
            logits.mul_(-1.5)
            x.add_(0.25)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(caught, step()):
            assert torch.equal(a, b), i
        torch.cuda.synchronize()


def pool_of(t):
    """The stream whose pool t's memory came from."""
    p = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= p < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no segment holds the tensor")


@pytest.mark.parametrize("kind", ["stream", "integer"])
def test_every_call_on_a_given_stream(kind):
    need_gpu()
    say("moe calls on a given stream", kind)
    g = torch.Generator(device="cuda").manual_seed(7)
    logits = torch.randn(4000, E, device="cuda", generator=g)      # two launches of the sort
    x, d = (torch.randn(4000, C, device="cuda", generator=g).bfloat16() for _ in range(2))
    h = torch.randn(4000 * K, 2 * I, device="cuda", generator=g).bfloat16()
    r = torch.randn(4000 * K, C, device="cuda", generator=g).bfloat16()

    def work(stream):
        ids, w = F.fp4_moe_route(logits, K, stream=stream)
        off, order, pos = F.fp4_moe_sort(ids, E, stream=stream)
        rows = F.fp4_moe_gather(x, pos, stream=stream)
        out = F.fp4_moe_combine(r, pos, w, stream=stream)
        dy, dw = F.fp4_moe_combine_backward(d, r, pos, w, stream=stream)
        y, hq, hs = F.fp4_glu(h, 0, w, order, off, checkpoint=True, stream=stream)
        q, s = F.fp4_glu_quantize(h, 1, stream=stream)
        dh, dwh = F.fp4_glu_backward(y, hq, hs, 0, w, order, off, stream=stream)
        dl = F.fp4_moe_route_backward(dwh, logits, ids, stream=stream)
        return ids, w, off, order, pos, rows, out, dy, dw, y, hq, hs, q, s, dh, dwh, dl

    want = work(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = work(s if kind == "stream" else s.cuda_stream)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()
    assert all(pool_of(t) == s.cuda_stream for t in got)
    assert all(pool_of(t) != s.cuda_stream for t in want)


def test_outputs_of_one_allocation_are_apart():
    """Writing all of one output leaves the others as they were, whatever the sizes."""
    need_gpu()
    for T, k, E in ((1, 1, 1), (3, 3, 127), (129, 2, 128), (700, 5, 1000)):
        logits = torch.randn(T, E, device="cuda")
        x8 = torch.randint(0, 100, (T, 96), device="cuda", dtype=torch.uint8)
        s8 = torch.randint(0, 100, (T, 3), device="cuda", dtype=torch.uint8)
        h = torch.randn(T, 192, device="cuda").bfloat16()
        for call in (lambda: F.fp4_moe_route(logits, k), lambda: F.fp4_moe_sort(F.fp4_moe_route(logits, k)[0], E),
                     lambda: F.fp4_moe_gather(x8, torch.arange(T, device="cuda").int()[:, None], s8),
                     lambda: F.fp4_glu_quantize(h), lambda: F.fp4_glu_quantize(h, fmt=F.FMT_MXFP4, out=None)):
            n = len(call())
            for i in range(n):
                got = call()
                kept = [t.clone() for t in got]
                got[i].fill_(77)
                assert all(torch.equal(a, b) for j, (a, b) in enumerate(zip(got, kept)) if j != i)
                assert (got[i] == 77).all() and all(t.is_contiguous() and t._version == (j == i) for j, t in enumerate(got))


def test_two_sorts_at_once():
    """Calls on two streams, each with a workspace of its own."""
    need_gpu()
    a, b = (torch.randint(-1, 200, (30000, 4), device="cuda", dtype=torch.int32) for _ in range(2))
    want = [F.fp4_moe_sort(t, 200) for t in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [F.fp4_moe_sort(t, 200, stream=s) for t, s in zip((a, b), streams)]
        torch.cuda.synchronize()
        for x, y in zip(want, got):
            assert all(torch.equal(p, q) for p, q in zip(x, y))


def test_refusals():
    need_gpu()
    x, ids = torch.zeros(4, 64, device="cuda").bfloat16(), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    logits = torch.zeros(4, 8, device="cuda")
    for call, what in ((lambda: F.fp4_moe_route(logits.t(), 2), "contiguous"),
                       (lambda: F.fp4_moe_route_backward(logits[:, :2], logits, ids), "contiguous"),
                       (lambda: F.fp4_moe_route_backward(torch.zeros(4, 3, device="cuda"), logits, ids), "dweights must have shape"),
                       (lambda: F.fp4_moe_route_backward(torch.zeros(4, 2, device="cuda"), logits, ids[:3]), "ids must have shape"),
                       (lambda: F.fp4_moe_sort(ids.t(), 8), "contiguous"),
                       (lambda: F.fp4_moe_gather(x, ids[:3]), "for 4 tokens"),
                       (lambda: F.fp4_moe_gather(x, ids.cpu()), "GPU"),
                       (lambda: F.fp4_moe_gather(x.view(torch.uint8), ids, torch.zeros(4, 2, dtype=torch.uint8, device="cuda")), "scales must have shape"),
                       (lambda: F.fp4_moe_gather(x, ids, out=torch.zeros(9, 32, device="cuda").bfloat16()), "out must have shape"),
                       (lambda: F.fp4_moe_combine(x, ids, torch.zeros(4, 3, device="cuda")), "weights must have shape"),
                       (lambda: F.fp4_moe_combine(x, ids.view(-1)), "position must be"),
                       (lambda: F.fp4_moe_combine_backward(x[:2], x, ids, torch.zeros(4, 2, device="cuda")), "dout must have shape"),
                       (lambda: F.fp4_glu(x[:, :63].contiguous()), "side by side"),
                       (lambda: F.fp4_glu(x, 0, torch.zeros(5, device="cuda")), "each of 4 rows"),
                       (lambda: F.fp4_glu(x, 0, None, torch.zeros(3, dtype=torch.int32, device="cuda")), "each of 4 rows"),
                       (lambda: F.fp4_glu(x, offsets=ids), "offsets"),
                       (lambda: F.fp4_glu(x, checkpoint=True, out=(x, x)), "3 tensors"),
                       (lambda: F.fp4_glu_backward(x, x.view(torch.uint8), x.view(torch.uint8)), "scales must have shape")):
        with pytest.raises(ValueError, match=what):
            call()
    for call, what in ((lambda: F.fp4_moe_route(logits.double(), 2), "float32 or"),
                       (lambda: F.fp4_moe_sort(ids.long(), 8), "torch.int32"),
                       (lambda: F.fp4_moe_gather(x.float(), ids), "torch.bfloat16"),
                       (lambda: F.fp4_moe_combine(x, ids, torch.zeros(4, 2, device="cuda").bfloat16()), "torch.float32"),
                       (lambda: F.fp4_glu(x.half()), "torch.bfloat16")):
        with pytest.raises(TypeError, match=what):
            call()
    for call, status in ((lambda: F.fp4_moe_route(logits, 9), 2), (lambda: F.fp4_moe_route(logits, 0), 2),
                         (lambda: F.fp4_moe_route(logits, 2, 7), 4), (lambda: F.fp4_moe_route(logits[:0], 2), 2),
                         (lambda: F.fp4_moe_sort(ids, 0), 2), (lambda: F.fp4_moe_sort(ids, 1025), 2),
                         (lambda: F.fp4_moe_sort(ids[:0], 4), 2),
                         (lambda: F.fp4_moe_sort(torch.zeros(100000, 1, dtype=torch.int32, device="cuda"), 4,
                                                 workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")), 6),
                         (lambda: F.fp4_moe_gather(x[:0], ids[:0]), 2), (lambda: F.fp4_moe_combine(x, ids[:, :0]), 2),
                         (lambda: F.fp4_moe_gather(x[:, :40].contiguous(), ids), 2),
                         (lambda: F.fp4_glu(x, 2), 4), (lambda: F.fp4_glu(x[:, :40].contiguous()), 2),
                         (lambda: F.fp4_glu_quantize(x, fmt=3), 4), (lambda: F.fp4_glu(x[:0]), 2)):
        with pytest.raises(F.Fp4Error) as e:
            call()
        assert e.value.status == status
