"""Calls of the norm, grouped and few-row operators that a binding has to refuse
or to arrange on the host, without a GPU."""
import os

import pytest
import torch

import fp4_precision_gemms_amd as F


@pytest.fixture(autouse=True)
def built():
    if not os.path.exists(F.LIB_PATH):
        pytest.skip("libfp4.so not built")


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


@pytest.mark.parametrize("lead_codes,lead_scales", [((3,), (3,)), ((1,), (1,)), ((2, 3), (2, 3)), ((3,), (2,))])
def test_decode_refuses_stacks_of_activations(lead_codes, lead_scales):
    """One operand a call: a stack would lose all but its first."""
    M, N, K = 40, 64, 96
    w = u8(*F.code_shape(N, K)), u8(*F.scale_shape(N, K))
    with pytest.raises(ValueError, match="a codes must have two .* or three"):
        F.fp4_gemm_decode(u8(*lead_codes, *F.code_shape(M, K)), u8(*lead_scales, *F.scale_shape(M, K)), *w)


def test_decode_refuses_activations_of_one_dimension():
    w = u8(*F.code_shape(64, 96)), u8(*F.scale_shape(64, 96))
    with pytest.raises(ValueError, match="a codes must have two .* or three"):
        F.fp4_gemm_decode(u8(96), u8(3), *w)


class FakeStream:
    def __init__(self, pointer):
        self.cuda_stream = pointer


class FakeTensor:
    """A tensor of the GPU as far as the host's calls look at it."""
    is_cuda = True
    shape = (64, 64)
    device = torch.device("cuda", 0)

    def __init__(self):
        self.recorded = []

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)


CALLS = {
    "rmsnorm_quantize": lambda t, s: F.fp4_rmsnorm_quantize(t, t, stream=s),
    "rmsnorm_backward": lambda t, s: F.fp4_rmsnorm_backward(t, t, t, t, stream=s),
    "gemm_decode": lambda t, s: F.fp4_gemm_decode(t, t, t, t, stream=s),
    "quantize_grouped": lambda t, s: F.fp4_quantize_grouped(t, t, stream=s),
    "quantize_grouped dual": lambda t, s: F.fp4_quantize_grouped_dual(t, t, stream=s),
    "gemm_grouped": lambda t, s: F.fp4_gemm_grouped(t, t, t, t, t, 64, stream=s),
    "gemm_grouped_wgrad": lambda t, s: F.fp4_gemm_grouped_wgrad(t, t, t, t, t, 64, stream=s),
}


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("kind", ["object", "integer"])
def test_a_call_on_a_given_stream_allocates_there(monkeypatch, name, kind):
    """The binding runs with the given stream as the current one, so that outputs
    and workspace come from that stream's pool, and gets no workspace of the
    current stream's; the outputs are recorded on the caller's stream."""
    import contextlib

    current, seen, made = [FakeStream(0x10)], [], []

    @contextlib.contextmanager
    def use(stream):
        current.append(stream)
        yield
        current.pop()

    class Binding:
        def __getattr__(self, function):
            def call(*args):
                seen.append((function, current[-1].cuda_stream, args))
                made.append(FakeTensor())
                return (made[-1],) if function != "gemm_decode" else made[-1]
            return call

    monkeypatch.setattr(F, "_native", lambda: Binding())
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda p, device=None: FakeStream(p))
    monkeypatch.setattr(torch, "empty", lambda *a, **k: pytest.fail("allocated on the current stream"))
    CALLS[name](FakeTensor(), FakeStream(0x20) if kind == "object" else 0x20)
    assert [(f, s) for f, s, _ in seen] == [(name.split()[0], 0x20)]
    assert seen[0][2][-1] == 0x20 and made[0].recorded == [0x10]


def test_outputs_of_the_older_calls_come_from_the_given_stream(monkeypatch):
    """The quantizers, products and nvfp4_quantize's workspace likewise."""
    import contextlib

    current, made = [FakeStream(0x10)], []

    class Made(torch.Tensor):
        def record_stream(self, stream):
            made.append((current[-1].cuda_stream, stream.cuda_stream))

    @contextlib.contextmanager
    def use(stream):
        current.append(stream)
        yield
        current.pop()

    def empty(shape, dtype=None, device=None):
        assert current[-1].cuda_stream == 0x20, "allocated on the current stream"
        return torch.zeros(shape, dtype=dtype).as_subclass(Made)

    class Library:
        def __getattr__(self, name):
            return lambda *a: 64 if name == "nvfp4_workspace_bytes" else 0

    class Bf16(torch.Tensor):
        device = torch.device("cuda", 0)

    monkeypatch.setattr(F, "lib", lambda: Library())
    monkeypatch.setattr(F, "_need", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch, "empty", empty)
    x = torch.zeros(64, 64, dtype=torch.bfloat16).as_subclass(Bf16)
    q = [torch.zeros(s, dtype=torch.uint8).as_subclass(Bf16) for s in (F.code_shape(64, 64), F.scale_shape(64, 64))]
    s = FakeStream(0x20)
    monkeypatch.setattr(F, "_as_stream", lambda stream, device: stream)
    for call, count in ((lambda: F.fp4_hadamard_quantize(x, stream=s), 2),
                        (lambda: F.fp4_hadamard_quantize_dual(x, stream=s), 4),
                        (lambda: F.fp4_wgrad_quantize(x, x, stream=s), 4),
                        (lambda: F.fp4_gemm_fprop(*q, *q, stream=s), 1), (lambda: F.fp4_gemm_mx(*q, *q, stream=s), 1),
                        (lambda: F.nvfp4_quantize(x, stream=s), 4)):
        made.clear()
        call()
        assert made == [(0x10, 0x10)] * count


def test_products_of_more_columns_than_a_launch_holds_are_refused_for_their_shape():
    a, shape = 0x10000, 2
    L = F.lib()
    assert L.fp4_gemm_decode(a, a, 1, a, a, 1, 2 ** 30, 32, a, 1, None) == shape
    assert L.fp4_gemm_grouped(a, a, 1, a, 1, 1, a, a, 2 ** 30, 32, a, 1, None) == shape


def test_shapes_of_an_mxfp8_operand():
    assert F.mx8_shapes(7, 96) == ((7, 96), (7, 3))
    codes, scales = (u8(*s) for s in F.mx8_shapes(7, 96))
    with pytest.raises(ValueError, match="GPU"):       # its shapes are taken
        F.fp4_gemm_decode(codes, scales, u8(*F.code_shape(64, 96)), u8(*F.scale_shape(64, 96)))
