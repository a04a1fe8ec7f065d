"""The operators of an MXFP4 mixture-of-experts block, measured: the norm that
feeds a quantized linear layer (residual added, output in 8 bits with block
scales) and its backward pass, the product of few rows with 4-bit weights
(serving), and products grouped by expert with ragged sizes (serving; training
forward and backward).

Formats.  MXFP4: blocks of 32 elements along the contraction, one E8M0 scale
2^e with e = floor(log2 max|v|) - 2, E2M1 elements (0, .5, 1, 1.5, 2, 3, 4, 6)
rounded to nearest, ties to the even code, saturating at 6.  MXFP8: the same
with E4M3 elements and e = floor(log2 max|v|) - 8, saturating at 448.
Layouts of an MXFP4 operand of R rows: codes [ceil(R/32), C/32, 512] (32-row
tiles, 16 bytes per row and block, even element in the low nibble), scales
[ceil(C/256), R, 8].  An MXFP8 operand is row-major: codes [R, C], scales
[R, C/32].
"""
import math

import torch

own = False

EPS = 1e-5
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------- cases
def listed():
    return [
        # one token's hidden state between two layers of a served model: latency
        {"name": "norm 1x4096", "op": "norm", "rows": 1, "cols": 4096, "residual": True},
        # a chunk of a prefill, odd in both sizes, at the first layer (no residual)
        {"name": "norm 333x5152", "op": "norm", "rows": 333, "cols": 5152, "residual": False},
        # a training batch at the hidden size of the repository's layers
        {"name": "norm 8192x4096", "op": "norm", "rows": 8192, "cols": 4096, "residual": True},
        # the norm's backward pass: a small odd batch, and a training batch of a larger model
        {"name": "norm back 1000x2080", "op": "norm back", "rows": 1000, "cols": 2080, "residual": False},
        {"name": "norm back 8192x8192", "op": "norm back", "rows": 8192, "cols": 8192, "residual": True},
        # one token through the gate/up projection, activations in 8 bits
        {"name": "decode8 1x14336x4096", "op": "decode", "rows": 1, "n": 14336, "k": 4096, "bits": 8},
        # a batch of tokens through the down projection, activations in 4 bits
        {"name": "decode4 24x4096x14336", "op": "decode", "rows": 24, "n": 4096, "k": 14336, "bits": 4},
        # a serving step: residual, norm and the query projection, an odd batch
        {"name": "token 5x4096x4096", "op": "token", "rows": 5, "n": 4096, "k": 4096, "bits": 8},
        # a decode batch spread over many small experts (some get no token)
        {"name": "experts8 96 of 64", "op": "experts8", "rows": 96, "experts": 64, "n": 1408, "k": 2048},
        # training forward: a ragged batch over eight experts of the gate/up size
        {"name": "experts 16384 of 8", "op": "experts", "rows": 16384, "experts": 8, "n": 14336, "k": 4096},
        # training backward: many small experts, odd sizes, some experts empty
        {"name": "experts back 1999 of 40", "op": "experts back", "rows": 1999, "experts": 40, "n": 736, "k": 1120},
        # training backward of the large layer
        {"name": "experts back 16384 of 8", "op": "experts back", "rows": 16384, "experts": 8, "n": 14336, "k": 4096},
    ]


def _spread(rng, low, high, step=1):
    """A size of [low, high], even over its logarithm, a multiple of `step`."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(v / step + 0.5) * step))


def draw(rng):
    op = rng.choice(["norm", "norm back", "decode", "token", "experts8", "experts", "experts back"])
    if op in ("norm", "norm back"):
        return {"op": op, "rows": _spread(rng, 1 if op == "norm" else 64, 8192), "cols": _spread(rng, 512, 8192, 32),
                "residual": rng.random() < 0.5}
    if op in ("decode", "token"):
        return {"op": op, "rows": _spread(rng, 1, 64), "n": _spread(rng, 512, 14336, 16), "k": _spread(rng, 512, 14336, 32),
                "bits": rng.choice([8, 4])}
    if op == "experts8":
        return {"op": op, "rows": _spread(rng, 1, 256), "experts": _spread(rng, 4, 96), "n": _spread(rng, 512, 4096, 16),
                "k": _spread(rng, 512, 4096, 32)}
    rows, n, k = _spread(rng, 512, 16384), _spread(rng, 512, 8192, 32), _spread(rng, 512, 4096, 32)
    most = min(64, rows // 48, 8 * 14336 * 4096 // (n * k))     # no more weights than the largest listed case has
    return {"op": op, "rows": rows, "experts": _spread(rng, 2, max(2, most)), "n": n, "k": k}


def work(case):
    if case["op"] in ("norm", "norm back"):
        n, back = case["rows"] * case["cols"], case["op"] == "norm back"
        each = (6 if back else 3) + (2 if back else 4) * case["residual"] + (0 if back else 1 / 32)
        return {"bytes": n * each + case["rows"] * 4 + case["cols"] * (6 if back else 2), "flops": n * (12 if back else 8)}
    m, n, k = case["rows"], case["n"], case["k"]
    four = 0.5 + 1 / 32
    if case["op"] == "decode":
        return {"bytes": n * k * four + m * k * (case["bits"] / 8 + 1 / 32) + 2 * m * n, "flops": 2 * m * n * k}
    if case["op"] == "token":
        return {"bytes": n * k * four + m * k * 6 + 2 * k + 2 * m * n, "flops": 2 * m * n * k + 8 * m * k}
    e = case["experts"]
    if case["op"] == "experts8":
        reached = e * (1 - (1 - 1 / e) ** m)     # experts that get a row, on average
        return {"bytes": reached * n * k * four + m * k * (1 + 1 / 32) + 2 * m * n, "flops": 2 * m * n * k}
    if case["op"] == "experts":
        return {"bytes": e * n * k * four + 2 * m * k + 2 * m * n, "flops": 2 * m * n * k}
    return {"bytes": e * n * k * four + 2 * m * n + 2 * m * k + 2 * m * k + 2 * e * n * k, "flops": 4 * m * n * k}


# ----------------------------------------------------------------- formats
def _pow2(e):
    """2^e in 32 bits, e whole numbers in [-127, 127]."""
    return torch.where(e < -126, 2.0 ** -127, ((e.clamp(min=-126) + 127).to(torch.int32) << 23).view(torch.float32))


def _exponent(v, top):
    """The shared exponent of each 32 values of the last axis."""
    m = v.abs().amax(-1, keepdim=True)
    return torch.where(m > 0, (torch.frexp(m)[1] - 1 - top).clamp(-127, 127), -127)


def _mxfp4(v):
    """(element values, exponents) of v [..., C]: both as [..., C/32, 32 or 1]."""
    v = v.unflatten(-1, (-1, 32))
    e = _exponent(v, 2)
    s = v * _pow2(-e)
    a = s.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(s / step) * step).clamp(-6, 6), e


def _mxfp8(v):
    v = v.unflatten(-1, (-1, 32))
    e = _exponent(v, 8)
    s = v * _pow2(-e)
    step = _pow2((torch.frexp(s)[1] - 1).clamp(min=-6) - 3)
    return (torch.round(s / step) * step).clamp(-448, 448), e


def _rounded(v):
    """v [..., C] through MXFP4 and back."""
    q, e = _mxfp4(v)
    return (q * _pow2(e)).flatten(-2)


def _pack(v):
    """(codes, scales) of v [..., R, C] in the layouts of an MXFP4 operand."""
    q, e = _mxfp4(v)
    grid = torch.tensor(GRID, device=v.device)
    code = torch.bucketize(q.abs(), grid).to(torch.uint8) | (torch.signbit(q).to(torch.uint8) << 3)
    code = code[..., 0::2] | (code[..., 1::2] << 4)                      # [..., R, nb, 16]
    r, nb = code.shape[-3], code.shape[-2]
    code = torch.nn.functional.pad(code, (0, 0, 0, 0, 0, -r % 32)).unflatten(-3, (-1, 32))
    code = code.transpose(-3, -2).flatten(-2).contiguous()               # [..., G, nb, 512]
    scale = torch.nn.functional.pad((e[..., 0] + 127).to(torch.uint8), (0, -nb % 8)).unflatten(-1, (-1, 8))
    return code, scale.transpose(-3, -2).contiguous()                    # [..., ceil(nb/8), R, 8]


def _unpack(codes, scales):
    """The values [..., R, C] of an MXFP4 operand, in 32 bits."""
    r, nb = scales.shape[-2], codes.shape[-2]
    c = codes.unflatten(-1, (32, 16)).transpose(-3, -2).flatten(-4, -3)[..., :r, :, :]
    c = torch.stack((c & 15, c >> 4), -1).flatten(-2)
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=codes.device)
    s = scales.transpose(-3, -2).flatten(-2)[..., :nb].to(torch.int32) - 127
    return (grid[c.to(torch.int32)] * _pow2(s)[..., None]).flatten(-2)


# ----------------------------------------------------------------- inputs
def _gauss(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _weight(g, case):
    """The MXFP4 operand of a Gaussian weight [n, k], as a program keeps it; for
    a backward pass that of its transpose."""
    w = _gauss(g, case["n"], case["k"]).mul_(0.02).bfloat16().float()
    return _pack(w.T if case["op"] == "experts back" else w)


def _counts(case, seed):
    """Rows of each expert: a router that likes some experts better."""
    g = torch.Generator().manual_seed(seed * 7919 + 13)
    like = torch.softmax(torch.randn(case["experts"], generator=g) * 0.4, 0)
    return torch.multinomial(like, case["rows"], replacement=True, generator=g).bincount(minlength=case["experts"])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    bf = torch.bfloat16
    if case["op"] in ("norm", "norm back", "token"):
        rows, cols = case["rows"], case["k"] if case["op"] == "token" else case["cols"]
        s["x"] = _gauss(g, rows, cols).mul_(1.5).to(bf)
        s["r"] = _gauss(g, rows, cols).to(bf) if case.get("residual", True) else None
        s["w"] = (1 + 0.1 * _gauss(g, cols)).to(bf)
        if case["op"] == "norm back":
            # what the forward pass keeps: the residual stream and 1 / its root mean square
            s["rstd"] = torch.rsqrt(s["x"].double().square().mean(1) + EPS).float()
            s["dy"] = _gauss(g, rows, cols).mul_(1e-3).to(bf)
            s["dh"] = _gauss(g, rows, cols).mul_(1e-3).to(bf) if case["residual"] else None
    if case["op"] in ("decode", "token"):
        s["wq"], s["ws"] = _weight(g, case)
    if case["op"] in ("decode", "experts8"):
        a = _gauss(g, case["rows"], case["k"])
        if case.get("bits", 8) == 8:
            q, e = _mxfp8(a)
            s["aq"] = q.flatten(-2).to(torch.float8_e4m3fn).view(torch.uint8)
            s["as"] = (e[..., 0] + 127).to(torch.uint8)
        else:
            s["aq"], s["as"] = _pack(a)
    if case["op"].startswith("experts"):
        counts = _counts(case, seed)
        s["most"] = int(counts.max())
        s["offsets"] = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32).cuda()
        if case["op"] != "experts8":
            s["x"] = _gauss(g, case["rows"], case["k"]).to(bf)
        s["wq"], s["ws"] = (torch.stack(p) for p in zip(*(_weight(g, case) for _ in range(case["experts"]))))
        if case["op"] == "experts back":
            s["dy"] = _gauss(g, case["rows"], case["n"]).mul_(1e-3).to(bf)
    return s


# ----------------------------------------------------------------- one pass
def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


def _run_own(s):
    import fp4_precision_gemms_amd as F

    op = s["op"]
    if op == "norm":
        codes, scales, h, rstd = F.fp4_rmsnorm_quantize(s["x"], s["w"], s["r"], EPS, F.FMT_MXFP8)
        return h, codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu), rstd
    if op == "norm back":
        return F.fp4_rmsnorm_backward(s["dy"], s["x"], s["w"], s["rstd"], s["dh"])
    if op == "decode":
        return F.fp4_gemm_decode(s["aq"], s["as"], s["wq"], s["ws"])
    if op == "token":
        codes, scales, h, _ = F.fp4_rmsnorm_quantize(s["x"], s["w"], s["r"], EPS, F.FMT_MXFP8 if s["bits"] == 8 else F.FMT_MXFP4)
        return h, F.fp4_gemm_decode(codes, scales, s["wq"], s["ws"])
    if op == "experts8":
        return F.fp4_gemm_grouped(s["aq"], s["as"], s["offsets"], s["wq"], s["ws"], s["rows"])
    if op == "experts":
        aq, as_ = F.fp4_quantize_grouped(s["x"], s["offsets"])
        return F.fp4_gemm_grouped(aq, as_, s["offsets"], s["wq"], s["ws"], s["rows"])
    dytq, dyts, dyq, dys = F.fp4_quantize_grouped_dual(s["dy"], s["offsets"], 32, F.HAD_DET)
    xtq, xts = F.fp4_quantize_grouped(s["x"], s["offsets"], F.AXIS_ROWS, 32, F.HAD_DET)
    dx = F.fp4_gemm_grouped(dyq, dys, s["offsets"], s["wq"], s["ws"], s["rows"])
    return dx, F.fp4_gemm_grouped_wgrad(dytq, dyts, xtq, xts, s["offsets"], s["rows"])


def _norm(s):
    """(h, y, rstd): the sum in 64 bits, since y is rounded to few bits next."""
    h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(torch.bfloat16)
    rstd = (1 / torch.sqrt(h.double().square().sum(1) / h.shape[1] + EPS)).float()
    return h, h.float() * rstd[:, None] * s["w"].float(), rstd


def _rotation(device):
    """The 32 x 32 Hadamard matrix in its natural order, over sqrt(32)."""
    i = torch.arange(32, device=device)
    both = i[:, None] & i[None, :]
    odd = (both ^ (both >> 1) ^ (both >> 2) ^ (both >> 3) ^ (both >> 4)) & 1
    return (1 - 2 * odd).float() / math.sqrt(32)


def _by_expert(s, v, to=1):
    """v [rows, C] as [experts, most, C], zero behind each expert's rows."""
    most = -(-s["most"] // to) * to
    first, end = s["offsets"][:-1, None], s["offsets"][1:, None]
    at = first + torch.arange(most, device=v.device, dtype=torch.int32)
    return torch.where((at < end)[..., None], v[at.clamp(max=v.shape[0] - 1)].float(), 0.0)


def _by_row(s, v):
    """[experts, most, C] back as [rows, C]."""
    at = torch.arange(s["rows"], device=v.device, dtype=torch.int32)
    e = (at[:, None] >= s["offsets"][None, 1:]).sum(1)
    return v[e, at - s["offsets"][e]]


def _run_plain(s):
    op, bf = s["op"], torch.bfloat16
    if op == "norm":
        h, y, rstd = _norm(s)
        q, e = _mxfp8(y)
        return (h, q.flatten(-2).to(torch.float8_e4m3fn), (e[..., 0] + 127).to(torch.uint8).view(torch.float8_e8m0fnu), rstd)
    if op == "norm back":
        dy, h, r = s["dy"].float(), s["x"].float(), s["rstd"][:, None]
        g = dy * s["w"].float()
        dx = r * g - h * (r * r * r * ((g * h).sum(1, keepdim=True) / h.shape[1]))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return dx.to(bf), (dy * (h * r)).sum(0)
    if op == "token":
        h, y, _ = _norm(s)
        if s["bits"] == 8:
            q, e = _mxfp8(y)
            a = (q * _pow2(e)).flatten(-2)
        else:
            a = _rounded(y)
        return h, (a @ _unpack(s["wq"], s["ws"]).T).to(bf)
    if op in ("decode", "experts8"):
        if s.get("bits", 8) == 8:
            a = (s["aq"].view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32)) * _pow2(s["as"].to(torch.int32) - 127)[..., None]).flatten(-2)
        else:
            a = _unpack(s["aq"], s["as"])
        if op == "decode":
            return (a @ _unpack(s["wq"], s["ws"]).T).to(bf)
        return _by_row(s, torch.bmm(_by_expert(s, a), _unpack(s["wq"], s["ws"]).transpose(1, 2))).to(bf)
    if op == "experts":
        a = _rounded(_by_expert(s, s["x"]))
        return _by_row(s, torch.bmm(a, _unpack(s["wq"], s["ws"]).transpose(1, 2))).to(bf)
    dy, x = _by_expert(s, s["dy"], 32), _by_expert(s, s["x"], 32)
    dx = _by_row(s, torch.bmm(_rounded(dy), _unpack(s["wq"], s["ws"]).transpose(1, 2))).to(bf)
    turn = _rotation(x.device)
    dyt = _rounded((dy.transpose(1, 2).unflatten(-1, (-1, 32)) @ turn).flatten(-2))
    xt = _rounded((x.transpose(1, 2).unflatten(-1, (-1, 32)) @ turn).flatten(-2))
    return dx, torch.bmm(dyt, xt.transpose(1, 2)).to(bf)


# ----------------------------------------------------------------- 64 bits
def _shared64(v, top):
    """Each 32 values' scale 2^(floor(log2 max) - top), in 64 bits."""
    m = v.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(m > 0, m, 1.0)))
    e = torch.where(torch.exp2(e) > m, e - 1, torch.where(torch.exp2(e + 1) <= m, e + 1, e))
    return torch.exp2(torch.where(m > 0, (e - top).clamp(-127, 127), -127.0))


def _four64(v):
    """v [..., C] through MXFP4 by a look at the grid's midpoints."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    s = _shared64(b, 2)
    a = (b / s).abs()
    n = torch.zeros_like(a, dtype=torch.int64)
    for code in range(7):     # ties go to the even code
        mid = (GRID[code] + GRID[code + 1]) / 2
        n += (a >= mid) if code % 2 else (a > mid)
    return (torch.tensor(GRID, dtype=torch.float64, device=v.device)[n] * torch.sign(b) * s).reshape(v.shape)


def _eight64(v):
    b = v.reshape(*v.shape[:-1], -1, 32)
    s = _shared64(b, 8)
    return (b / s).clamp(-448, 448).to(torch.float8_e4m3fn).double().reshape(v.shape), s[..., 0]


def _values64(codes, scales, rows):
    """An MXFP4 operand's values [rows, C], element by element of its layout."""
    groups, nb, _ = codes.shape
    r = torch.arange(rows, device=codes.device)[:, None, None]
    b = torch.arange(nb, device=codes.device)[None, :, None]
    i = torch.arange(32, device=codes.device)[None, None, :]
    byte = codes.reshape(-1)[((r // 32) * nb + b) * 512 + (r % 32) * 16 + i // 2].long()
    code = torch.where(i % 2 == 1, byte >> 4, byte & 15)
    table = torch.tensor(GRID + tuple(-x for x in GRID), dtype=torch.float64, device=codes.device)
    scale = scales.reshape(-1)[((b // 8) * rows + r) * 8 + b % 8].double() - 127
    return (table[code] * torch.exp2(scale)).reshape(rows, nb * 32)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "token"):
        h = s["x"] if s["r"] is None else (s["x"].double() + s["r"].double()).to(torch.bfloat16)
        mean = h.double().pow(2).mean(1, keepdim=True)
        y = h.double() / torch.sqrt(mean + EPS) * s["w"].double()
        if op == "norm":
            q, scale = _eight64(y)
            return h.double(), q, scale, (1 / torch.sqrt(mean + EPS))[:, 0]
        q, scale = _eight64(y)
        a = q * scale.repeat_interleave(32, 1) if case["bits"] == 8 else _four64(y)
        return h.double(), a @ _values64(s["wq"], s["ws"], case["n"]).T
    if op == "norm back":
        dy, h, w, r = s["dy"].double(), s["x"].double(), s["w"].double(), s["rstd"].double()[:, None]
        n = h * r
        g = dy * w
        dx = r * (g - n * (g * n).mean(1, keepdim=True))
        return dx if s["dh"] is None else dx + s["dh"].double(), (dy * n).sum(0)
    if op in ("decode", "experts8"):
        if case.get("bits", 8) == 8:
            a = s["aq"].view(torch.float8_e4m3fn).double() * torch.exp2(s["as"].double() - 127).repeat_interleave(32, 1)
        else:
            a = _values64(s["aq"], s["as"], case["rows"])
        if op == "decode":
            return a @ _values64(s["wq"], s["ws"], case["n"]).T
    ends = s["offsets"].tolist()
    if op == "experts":
        a = _four64(s["x"].double())
    if op in ("experts8", "experts"):
        return torch.cat([a[i:j] @ _values64(s["wq"][e], s["ws"][e], case["n"]).T for e, (i, j) in enumerate(zip(ends, ends[1:]))])
    dyq = _four64(s["dy"].double())
    h = torch.ones(1, 1, dtype=torch.float64, device="cuda")
    for _ in range(5):
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)

    def along_rows(v):
        """v [t, C] rotated and rounded along its rows, zero rows added to 32: [C, t']."""
        t = torch.nn.functional.pad(v.double(), (0, 0, 0, -v.shape[0] % 32)).T.contiguous()
        return _four64((t.reshape(t.shape[0], -1, 32) @ (h / math.sqrt(32))).reshape(t.shape[0], -1))

    dx, dw = [], []
    for e, (i, j) in enumerate(zip(ends, ends[1:])):
        dx.append(dyq[i:j] @ _values64(s["wq"][e], s["ws"][e], case["k"]).T)
        if j > i:
            dw.append((along_rows(s["dy"][i:j]) @ along_rows(s["x"][i:j]).T).float())
        else:
            dw.append(torch.zeros(case["n"], case["k"], device="cuda"))
    return torch.cat(dx), torch.stack(dw)
