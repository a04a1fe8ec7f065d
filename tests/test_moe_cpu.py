"""The entry points around the experts' products without a GPU: arguments are
refused with the documented status codes before any HIP call, and by the binding
before the library is reached."""
import contextlib
import os

import pytest
import torch

import fp4_precision_gemms_amd as F

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_ENUM, ERR_LAUNCH, ERR_WORKSPACE = range(7)
A = 0x10000          # a fake 16-byte aligned device address (never dereferenced)
MIS = 0x10008        # misaligned to 16 bytes
ODD = 0x10002        # misaligned to 4


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(F.LIB_PATH):
        pytest.skip("libfp4.so not built")
    return F.lib()


def test_route_errors(L):
    def call(l=A, dt=0, T=4, E=64, k=6, score=0, norm=1, ids=A, w=A):
        return L.fp4_moe_route(l, dt, T, E, k, score, norm, ids, w, None)

    def back(dw=A, l=A, dt=0, ids=A, T=4, E=64, k=6, score=0, norm=1, d=A):
        return L.fp4_moe_route_backward(dw, l, dt, ids, T, E, k, score, norm, d, None)

    for f in (call, back):
        assert f(dt=2) == ERR_ENUM and f(score=2) == ERR_ENUM and f(score=-1) == ERR_ENUM and f(norm=2) == ERR_ENUM
        for bad in (dict(T=0), dict(T=-1), dict(T=2 ** 31), dict(E=0), dict(E=1025), dict(k=0), dict(k=65), dict(E=5),
                    dict(T=2 ** 30)):
            assert f(**bad) == ERR_SHAPE, bad
    for name in ("l", "ids", "w"):
        assert call(**{name: None}) == ERR_NULL and call(**{name: ODD}) == ERR_ALIGN, name
    for name in ("dw", "l", "ids", "d"):
        assert back(**{name: None}) == ERR_NULL and back(**{name: ODD}) == ERR_ALIGN, name
    assert call(l=A + 1, dt=1) == ERR_ALIGN and back(d=A + 1, dt=1) == ERR_ALIGN


def test_sort_errors(L):
    def call(ids=A, n=100000, E=64, off=A, order=A, pos=A, ws=A, b=1 << 20):
        return L.fp4_moe_sort(ids, n, E, off, order, pos, ws, b, None)

    for bad in (dict(n=0), dict(n=-4), dict(n=2 ** 31), dict(E=0), dict(E=1025), dict(E=-2 ** 40)):
        assert call(**bad) == ERR_SHAPE, bad
    for name in ("ids", "off", "order", "pos"):
        assert call(**{name: None}) == ERR_NULL and call(**{name: ODD}) == ERR_ALIGN, name
    need = F.fp4_moe_sort_workspace_bytes(100000, 64)
    assert need > 0 and call(b=need - 1) == ERR_WORKSPACE and call(ws=None) == ERR_WORKSPACE and call(ws=MIS) == ERR_ALIGN
    assert F.fp4_moe_sort_workspace_bytes(64, 1024) == 0 and F.fp4_moe_sort_workspace_bytes(0, 64) == 0
    assert F.fp4_moe_sort_workspace_bytes(2 ** 31 - 1, 1024) <= 256 * 1025 * 4


def test_gather_and_combine_errors(L):
    def gather(x=A, s=None, p=A, T=4, k=2, rows=8, cols=64, out=A, os=None):
        return L.fp4_moe_gather(x, s, p, T, k, rows, cols, out, os, None)

    def combine(y=A, p=A, w=A, T=4, k=2, rows=8, cols=64, out=A):
        return L.fp4_moe_combine(y, p, w, T, k, rows, cols, out, None)

    def back(d=A, y=A, p=A, w=A, T=4, k=2, rows=8, cols=64, dy=A, dw=A):
        return L.fp4_moe_combine_backward(d, y, p, w, T, k, rows, cols, dy, dw, None)

    for f in (gather, combine, back):
        for bad in (dict(T=0), dict(T=-1), dict(k=0), dict(k=2 ** 31), dict(T=2 ** 30), dict(rows=0), dict(rows=2 ** 31),
                    dict(cols=0), dict(cols=48), dict(cols=-32), dict(cols=2 ** 24)):
            assert f(**bad) == ERR_SHAPE, bad
        assert f(p=ODD) == ERR_ALIGN and f(p=None) == ERR_NULL
    assert gather(s=A) == ERR_NULL and gather(os=A) == ERR_NULL
    for f, names in ((gather, ("x", "out")), (combine, ("y", "out")), (back, ("d", "y", "dy"))):
        for n in names:
            assert f(**{n: None}) == ERR_NULL and f(**{n: MIS}) == ERR_ALIGN, n
    assert combine(w=ODD) == ERR_ALIGN
    for n in ("w", "dw"):
        assert back(**{n: None}) == ERR_NULL and back(**{n: ODD}) == ERR_ALIGN


def test_glu_errors(L):
    def call(x=A, w=None, o=None, off=None, E=0, act=0, rows=4, cols=64, y=A, fmt=1, q=A, s=A, xq=A, xs=A):
        return L.fp4_glu(x, w, o, off, E, act, rows, cols, y, fmt, q, s, xq, xs, None)

    def back(dy=A, xq=A, xs=A, w=A, o=A, off=A, E=4, act=0, rows=4, cols=64, dx=A, dw=A):
        return L.fp4_glu_backward(dy, xq, xs, w, o, off, E, act, rows, cols, dx, dw, None)

    for f in (call, back):
        assert f(act=2) == ERR_ENUM and f(act=-1) == ERR_ENUM
        for bad in (dict(rows=0), dict(rows=2 ** 31), dict(cols=0), dict(cols=48), dict(cols=2 ** 24), dict(off=A, E=0),
                    dict(off=A, E=1025), dict(rows=2 ** 31 - 1, cols=4096)):
            assert f(**bad) == ERR_SHAPE, bad
        for n in ("w", "o"):
            assert f(**{n: ODD}) == ERR_ALIGN, n
        assert f(off=ODD, E=4) == ERR_ALIGN
    assert call(fmt=2) == ERR_ENUM
    assert call(x=None) == ERR_NULL and call(q=None) == ERR_NULL and call(xs=None) == ERR_NULL
    assert call(y=None, q=None, s=None, xq=None, xs=None) == ERR_NULL
    for n in ("x", "y", "q", "s", "xq", "xs"):
        assert call(**{n: MIS}) == ERR_ALIGN, n
    for n in ("dy", "xq", "xs", "dx", "dw"):
        assert back(**{n: None}) == ERR_NULL, n
    for n in ("dy", "xq", "xs", "dx"):
        assert back(**{n: MIS}) == ERR_ALIGN, n
    assert back(dw=ODD) == ERR_ALIGN


def test_quantize_experts_errors(L):
    def call(w=A, E=4, N=64, K=96, wtq=A, wts=A, wq=A, ws=A):
        return L.fp4_quantize_experts(w, E, N, K, wtq, wts, wq, ws, None)

    for bad in (dict(E=0), dict(E=1025), dict(N=0), dict(N=48), dict(K=16), dict(K=-32), dict(N=2 ** 22),
                dict(E=1024, K=2 ** 40)):
        assert call(**bad) == ERR_SHAPE, bad
    for n in ("w", "wtq", "wts", "wq", "ws"):
        assert call(**{n: None}) == ERR_NULL and call(**{n: MIS}) == ERR_ALIGN, n
    with pytest.raises(ValueError, match="experts, N, K"):
        F.fp4_quantize_experts(torch.zeros(64, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="GPU"):
        F.fp4_quantize_experts(torch.zeros(2, 64, 64, dtype=torch.bfloat16))


def test_binding_refuses(L):
    f32, bf, i32, u8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8
    z = lambda *s, dtype=bf: torch.zeros(*s, dtype=dtype)  # noqa: E731
    with pytest.raises(ValueError, match="GPU"):
        F.fp4_moe_route(z(4, 8, dtype=f32), 2)
    with pytest.raises(TypeError, match="float32 or torch.bfloat16"):
        F.fp4_moe_route(z(4, 8, dtype=torch.float16), 2)
    with pytest.raises(ValueError, match="two dimensions"):
        F.fp4_moe_route(z(8, dtype=f32), 2)
    with pytest.raises(ValueError, match="GPU"):
        F.fp4_moe_route_backward(z(4, 2, dtype=f32), z(4, 8, dtype=f32), z(4, 2, dtype=i32))
    with pytest.raises(TypeError, match="ids must be torch.int32"):
        F.fp4_moe_sort(z(4, 2, dtype=torch.int64), 8)
    with pytest.raises(ValueError, match="GPU"):
        F.fp4_moe_sort(z(4, 2, dtype=i32), 8)
    with pytest.raises(TypeError, match="x must be torch.bfloat16"):
        F.fp4_moe_gather(z(4, 32, dtype=f32), z(4, 2, dtype=i32))
    with pytest.raises(TypeError, match="x must be torch.uint8"):
        F.fp4_moe_gather(z(4, 32), z(4, 2, dtype=i32), z(4, 1, dtype=u8))
    with pytest.raises(ValueError, match="GPU"):
        F.fp4_moe_combine(z(8, 32), z(4, 2, dtype=i32))
    with pytest.raises(ValueError, match="GPU"):
        F.fp4_glu(z(4, 64))
    with pytest.raises(ValueError, match="GPU"):
        F.fp4_glu_quantize(z(4, 64))
    with pytest.raises(ValueError, match="GPU"):
        F.fp4_glu_backward(z(4, 32), z(4, 64, dtype=u8), z(4, 2, dtype=u8))


class FakeStream:
    def __init__(self, pointer):
        self.cuda_stream = pointer


class FakeTensor:
    """A tensor of the GPU as far as the host's calls look at it."""
    is_cuda = True
    device = torch.device("cuda", 0)

    def __init__(self):
        self.recorded = []

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)


CALLS = {
    "moe_route": lambda t, s: F.fp4_moe_route(t, 2, stream=s),
    "moe_route_backward": lambda t, s: F.fp4_moe_route_backward(t, t, t, stream=s),
    "moe_sort": lambda t, s: F.fp4_moe_sort(t, 4, stream=s),
    "moe_gather": lambda t, s: F.fp4_moe_gather(t, t, stream=s),
    "moe_combine": lambda t, s: F.fp4_moe_combine(t, t, stream=s),
    "moe_combine_backward": lambda t, s: F.fp4_moe_combine_backward(t, t, t, t, stream=s),
    "glu": lambda t, s: F.fp4_glu(t, stream=s),
    "glu_quantize": lambda t, s: F.fp4_glu_quantize(t, stream=s),
    "glu_backward": lambda t, s: F.fp4_glu_backward(t, t, t, stream=s),
}


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("kind", ["object", "integer"])
def test_a_call_on_a_given_stream_allocates_there(monkeypatch, name, kind):
    """The binding runs with the given stream as the current one and gets it as its
    last argument; the outputs are recorded on the caller's stream."""
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
                return (made[-1],)
            return call

    monkeypatch.setattr(F, "_native", lambda: Binding())
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda p, device=None: FakeStream(p))
    monkeypatch.setattr(torch, "empty", lambda *a, **k: pytest.fail("allocated on the current stream"))
    CALLS[name](FakeTensor(), FakeStream(0x20) if kind == "object" else 0x20)
    assert [(f, s) for f, s, _ in seen] == [(name, 0x20)]
    assert seen[0][2][-1] == 0x20 and made[0].recorded == [0x10]
