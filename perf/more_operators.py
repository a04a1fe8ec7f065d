"""The operators around the experts' products of a mixture of experts, measured:
the router (the k best experts of each token, their weights, and its backward
pass), tokens sorted by expert (bf16 rows for training, 8-bit rows for serving)
and combined again with weights, both ways, and the gated activation between an
expert's two products, with its input kept in 8 bits for the backward pass.

T tokens choose k of E experts each; a slot is one such choice (slot t k + j).
Sorting gives offsets [E + 1] (expert e owns the rows offsets[e] ..
offsets[e + 1]), order [T k] (the slot of each row, slots in their order within
an expert; slots of no expert, id -1, behind the last expert's rows) and
position [T, k] (the row of each slot, -1 for one of no expert).

MXFP8: blocks of 32 elements along a row, one E8M0 scale 2^e with e =
floor(log2 max|v|) - 8, E4M3 elements to nearest even, saturating at 448; codes
[R, C] and scales [R, C/32], row-major.
"""
import math

import torch

own = False


# ----------------------------------------------------------------- cases
def listed():
    return [
        # one token of a served model chooses its experts: latency
        {"name": "route 1x64", "op": "route", "tokens": 1, "experts": 64, "k": 6, "score": "softmax", "normalize": True,
         "bf16": False, "masked": False, "back": False},
        # an odd training batch: bf16 logits (with ties), sigmoid scores, some experts out of reach
        # of a token, some tokens only filling
        {"name": "route 1999x40 both ways", "op": "route", "tokens": 1999, "experts": 40, "k": 4, "score": "sigmoid",
         "normalize": True, "bf16": True, "masked": True, "back": True},
        # a training batch over many experts, weights not normalized: a gradient for every logit
        {"name": "route 16384x256 both ways", "op": "route", "tokens": 16384, "experts": 256, "k": 8, "score": "softmax",
         "normalize": False, "bf16": False, "masked": False, "back": True},
        # a decode batch of 8-bit rows to the experts' few-row products
        {"name": "dispatch8 16 tokens", "op": "dispatch8", "tokens": 16, "experts": 64, "k": 6, "cols": 2048, "dropped": 0.0},
        # a training batch to 8 experts: 16384 rows of the hidden size
        {"name": "dispatch 8192 tokens", "op": "dispatch", "tokens": 8192, "experts": 8, "k": 2, "cols": 4096, "dropped": 0.0},
        # the decode batch's way back
        {"name": "combine 16 tokens", "op": "combine", "tokens": 16, "experts": 64, "k": 6, "cols": 2048, "dropped": 0.0},
        # the training batch's way back, and its gradients
        {"name": "combine 8192 tokens", "op": "combine", "tokens": 8192, "experts": 8, "k": 2, "cols": 4096, "dropped": 0.0},
        {"name": "combine back 8192 tokens", "op": "combine back", "tokens": 8192, "experts": 8, "k": 2, "cols": 4096,
         "dropped": 0.0},
        # the activation of a decode batch, out in 8 bits for the next few-row product
        {"name": "glu8 96x1408", "op": "glu8", "rows": 96, "inner": 1408, "act": "silu", "experts": 64},
        # an odd batch of small experts: the backward pass of the other activation
        {"name": "glu back 1999x736", "op": "glu back", "rows": 1999, "inner": 736, "act": "gelu", "experts": 40},
        # the training batch through the gate/up size, input kept in 8 bits, and its backward pass
        {"name": "glu 16384x14336", "op": "glu", "rows": 16384, "inner": 14336, "act": "silu", "experts": 8},
        {"name": "glu back 16384x14336", "op": "glu back", "rows": 16384, "inner": 14336, "act": "silu", "experts": 8},
    ]


def _spread(rng, low, high, step=1):
    """A size of [low, high], even over its logarithm, a multiple of `step`."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(v / step + 0.5) * step))


def draw(rng):
    op = rng.choice(["route", "route", "dispatch8", "dispatch", "combine", "combine back", "glu8", "glu", "glu back"])
    if op == "route":
        experts = _spread(rng, 4, 256)
        return {"op": op, "tokens": _spread(rng, 1, 16384), "experts": experts, "k": _spread(rng, 1, min(8, experts)),
                "score": rng.choice(["softmax", "sigmoid"]), "normalize": rng.random() < 0.5, "bf16": rng.random() < 0.5,
                "masked": rng.random() < 0.5, "back": rng.random() < 0.7}
    if op.startswith("glu"):
        rows, inner = _spread(rng, 1, 256 if op == "glu8" else 16384), _spread(rng, 256, 14336, 32)
        return {"op": op, "rows": rows, "inner": inner, "act": rng.choice(["silu", "gelu"]), "experts": _spread(rng, 4, 64)}
    k, cols = rng.randint(1, 8), _spread(rng, 512, 8192, 32)
    most = 64 if op == "dispatch8" else min(8192, 8192 * 2 * 4096 // (k * cols))     # rows times columns as listed at most
    return {"op": op, "tokens": _spread(rng, 1, most), "experts": _spread(rng, 8, 256), "k": k, "cols": cols,
            "dropped": rng.choice([0.0, 0.0, 0.1])}


def work(case):
    if case["op"] == "route":
        t, e, k, size = case["tokens"], case["experts"], case["k"], 2 if case["bf16"] else 4
        one = t * (e * size + 8 * k)
        return {"bytes": one + case["back"] * (t * e * size + one), "flops": t * e * (4 + 4 * case["back"])}
    if case["op"].startswith("glu"):
        n, r = case["rows"] * case["inner"], case["rows"]
        kept = 2 * n * (1 + 1 / 32)
        if case["op"] == "glu8":
            return {"bytes": 4 * n + n * (1 + 1 / 32) + 8 * r, "flops": 12 * n}
        if case["op"] == "glu":
            return {"bytes": 4 * n + 2 * n + kept + 8 * r, "flops": 16 * n}
        return {"bytes": 2 * n + kept + 4 * n + 12 * r, "flops": 24 * n}
    t, slots, c = case["tokens"], case["tokens"] * case["k"], case["cols"]
    live = slots * (1 - case["dropped"])
    if case["op"] == "dispatch8":
        return {"bytes": (t + live) * c * (1 + 1 / 32) + 12 * slots, "flops": 0}
    if case["op"] == "dispatch":
        return {"bytes": (t + live) * c * 2 + 12 * slots, "flops": 0}
    if case["op"] == "combine":
        return {"bytes": (t + live) * c * 2 + 8 * slots, "flops": 2 * live * c}
    return {"bytes": (t + 2 * live) * c * 2 + 12 * slots, "flops": 3 * live * c}


# ----------------------------------------------------------------- formats
def _pow2(e):
    """2^e in 32 bits, e whole numbers in [-127, 127]."""
    return torch.where(e < -126, 2.0 ** -127, ((e.clamp(min=-126) + 127).to(torch.int32) << 23).view(torch.float32))


def _mxfp8(v):
    """MXFP8 codes and scales of v [R, C], as bytes."""
    v = v.unflatten(-1, (-1, 32))
    m = v.abs().amax(-1, keepdim=True)
    e = torch.where(m > 0, (torch.frexp(m)[1] - 9).clamp(-127, 127), -127)
    q = (v * _pow2(-e)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.flatten(-2).view(torch.uint8), (e[..., 0] + 127).to(torch.uint8)


def _values(codes, scales):
    """The values [R, C] that MXFP8 bytes stand for, in 32 bits."""
    v = codes.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32))
    return (v * _pow2(scales.to(torch.int32) - 127)[..., None]).flatten(-2)


# ----------------------------------------------------------------- inputs
def _gauss(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ids(g, case):
    """k different experts of each token, some experts chosen more often; a share
    of the slots goes to no expert."""
    like = _gauss(g, case["tokens"], case["experts"]) + 0.4 * _gauss(g, case["experts"])
    ids = torch.argsort(like, 1, descending=True)[:, :case["k"]].to(torch.int32)
    if case["dropped"]:
        ids = torch.where(torch.rand(ids.shape, generator=g, device="cuda") < case["dropped"], -1, ids)
    return ids.contiguous()


def _sorted(ids, experts):
    """(offsets, order, position) of ids [T, k]."""
    flat = torch.where(ids < 0, experts, ids).flatten()
    order = torch.argsort(flat, stable=True).to(torch.int32)
    offsets = (flat[None, :] < torch.arange(experts + 1, device=ids.device)[:, None]).sum(1).to(torch.int32)
    position = torch.empty_like(flat)
    position[order.long()] = torch.arange(flat.numel(), dtype=torch.int32, device=ids.device)
    return offsets, order, torch.where(flat == experts, -1, position).view(ids.shape)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    bf = torch.bfloat16
    if case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        v = 1.5 * _gauss(g, t, e) + 0.5 * _gauss(g, e)
        if case["masked"]:
            v = v.masked_fill(torch.rand(t, e, generator=g, device="cuda") < 0.25, -math.inf)
            v = v.masked_fill(torch.rand(t, 1, generator=g, device="cuda") < 0.02, -math.inf)
        s["logits"] = v.to(bf) if case["bf16"] else v
        s["dweights"] = 1e-2 * _gauss(g, t, case["k"])
        return s
    if case["op"].startswith("glu"):
        rows, inner = case["rows"], case["inner"]
        # what the first product gives, and each row's weight by way of the sorted order
        x = _gauss(g, rows, 2 * inner).to(bf)
        s["weights"] = torch.rand(rows, generator=g, device="cuda") * 0.9 + 0.05
        ids = torch.randint(case["experts"], (rows, 1), generator=g, device="cuda", dtype=torch.int32)
        s["offsets"], s["order"], _ = _sorted(ids, case["experts"])
        if case["op"] == "glu back":
            s["xq"], s["xs"] = _mxfp8(x.float())
            s["dy"] = (1e-3 * _gauss(g, rows, inner)).to(bf)
        else:
            s["x"] = x
        return s
    t, slots, cols = case["tokens"], case["tokens"] * case["k"], case["cols"]
    s["ids"] = _ids(g, case)
    # rows of no expert are left as they were: the program's own buffer, cleared once
    s["kept"] = torch.zeros(slots, cols, dtype=bf, device="cuda") if case["dropped"] else None
    if case["op"] == "dispatch":
        s["x"] = _gauss(g, t, cols).to(bf)
    elif case["op"] == "dispatch8":
        s["xq"], s["xs"] = _mxfp8(_gauss(g, t, cols))
        if case["dropped"]:
            s["kept"] = tuple(torch.zeros(slots, n, dtype=torch.uint8, device="cuda") for n in (cols, cols // 32))
    else:
        s["offsets"], s["order"], s["position"] = _sorted(s["ids"], case["experts"])
        s["y"] = _gauss(g, slots, cols).to(bf)
        s["weights"] = torch.softmax(_gauss(g, t, case["k"]), 1)
        s["dout"] = (1e-3 * _gauss(g, t, cols)).to(bf)
    return s


# ----------------------------------------------------------------- one pass
def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


def _run_own(s):
    import fp4_precision_gemms_amd as F

    op = s["op"]
    if op == "route":
        score = F.SCORE_SOFTMAX if s["score"] == "softmax" else F.SCORE_SIGMOID
        ids, weights = F.fp4_moe_route(s["logits"], s["k"], score, s["normalize"])
        if not s["back"]:
            return ids, weights
        return ids, weights, F.fp4_moe_route_backward(s["dweights"], s["logits"], ids, score, s["normalize"])
    if op.startswith("glu"):
        act = F.ACT_SILU if s["act"] == "silu" else F.ACT_GELU
        if op == "glu8":
            codes, scales = F.fp4_glu_quantize(s["x"], act, s["weights"], s["order"], s["offsets"])
            return codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)
        if op == "glu":
            y, xq, xs = F.fp4_glu(s["x"], act, s["weights"], s["order"], s["offsets"], checkpoint=True)
            return y, xq.view(torch.float8_e4m3fn), xs.view(torch.float8_e8m0fnu)
        return F.fp4_glu_backward(s["dy"], s["xq"], s["xs"], act, s["weights"], s["order"], s["offsets"])
    if op == "dispatch":
        offsets, order, position = F.fp4_moe_sort(s["ids"], s["experts"])
        return offsets, order, position, F.fp4_moe_gather(s["x"], position, out=s["kept"])
    if op == "dispatch8":
        offsets, order, position = F.fp4_moe_sort(s["ids"], s["experts"])
        codes, scales = F.fp4_moe_gather(s["xq"], position, s["xs"], out=s["kept"])
        return offsets, order, position, codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)
    if op == "combine":
        return F.fp4_moe_combine(s["y"], s["position"], s["weights"])
    out = None if s["kept"] is None else (s["kept"], torch.empty_like(s["weights"]))
    return F.fp4_moe_combine_backward(s["dout"], s["y"], s["position"], s["weights"], out=out)


def _logsigmoid(v):
    return torch.clamp(v, max=0) - torch.log1p(torch.exp(-v.abs()))


def _route(s, logits):
    """(ids, weights, scores by expert): the sort is stable, so that ties go to
    the lowest index; an expert that is out of reach is no choice."""
    k = s["k"]
    best, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    live = best > -math.inf
    if s["score"] == "softmax":
        top = torch.where(live[:, :1], best[:, :1], 0.0)
        every = torch.exp(logits - top)
        chosen = torch.exp(best - top)
        total = (chosen if s["normalize"] else every).sum(1, keepdim=True)
        weights = chosen / torch.where(total > 0, total, 1.0)
        score = every / torch.where(total > 0, total, 1.0)
    else:
        score = torch.sigmoid(logits)
        weights = torch.sigmoid(best)
        if s["normalize"]:
            log = _logsigmoid(best)
            chosen = torch.exp(log - torch.where(live[:, :1], log[:, :1], 0.0))
            total = chosen.sum(1, keepdim=True)
            weights = chosen / torch.where(total > 0, total, 1.0)
    return torch.where(live, ids, -1).to(torch.int32), torch.where(live, weights, 0.0), score


def _route_back(s, ids, weights, score):
    live = ids >= 0
    at = torch.where(live, ids, 0).long()
    g = torch.where(live, s["dweights"].to(weights.dtype), 0.0)
    each = weights * (g - (g * weights).sum(1, keepdim=True))
    if s["score"] == "softmax" and not s["normalize"]:
        full = torch.zeros_like(score).scatter_add_(1, at, g)
        return score * (full - (g * weights).sum(1, keepdim=True))
    if s["score"] == "sigmoid":
        here = torch.gather(score, 1, at)
        each = (each if s["normalize"] else g * weights) * (1 - here)
    return torch.zeros_like(score).scatter_add_(1, at, torch.where(live, each, 0.0))


def _slope(s, v):
    """(sigma(s(v)), v s'(v)) of the activation v sigma(s(v))."""
    if s["act"] == "silu":
        return torch.sigmoid(v), v
    c = 2 * math.sqrt(2 / math.pi)
    return torch.sigmoid(c * (v + 0.044715 * v * v * v)), c * (v + 3 * 0.044715 * v * v * v)


def _run_plain(s):
    op, bf = s["op"], torch.bfloat16
    if op == "route":
        ids, weights, score = _route(s, s["logits"].float())
        if not s["back"]:
            return ids, weights
        return ids, weights, _route_back(s, ids, weights, score).to(s["logits"].dtype)
    if op.startswith("glu"):
        w = s["weights"][s["order"].long()][:, None]
        if op == "glu back":
            gate, up = _values(s["xq"], s["xs"]).chunk(2, 1)
            sigma, slope = _slope(s, gate)
            act, dy = gate * sigma, s["dy"].float()
            dgate = dy * w * up * (sigma + slope * sigma * (1 - sigma))
            dweights = torch.empty_like(s["weights"])
            dweights[s["order"].long()] = (dy * (act * up)).sum(1)
            return torch.cat((dgate, dy * w * act), 1).to(bf), dweights
        x = s["x"].float()
        gate, up = x.chunk(2, 1)
        y = gate * _slope(s, gate)[0] * up * w
        if op == "glu8":
            codes, scales = _mxfp8(y)
            return codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)
        xq, xs = _mxfp8(x)
        return y.to(bf), xq.view(torch.float8_e4m3fn), xs.view(torch.float8_e8m0fnu)
    if op.startswith("dispatch"):
        offsets, order, position = _sorted(s["ids"], s["experts"])
        at = order.long()
        live = (s["ids"].flatten()[at] >= 0)[:, None]
        token = at // s["k"]

        def rows(x, kept):
            return x[token] if kept is None else torch.where(live, x[token], kept)

        if op == "dispatch":
            return offsets, order, position, rows(s["x"], s["kept"])
        kept = s["kept"] or (None, None)
        return (offsets, order, position, rows(s["xq"], kept[0]).view(torch.float8_e4m3fn),
                rows(s["xs"], kept[1]).view(torch.float8_e8m0fnu))
    live, at = s["position"] >= 0, s["position"].clamp(min=0).long()
    w = torch.where(live, s["weights"], 0.0)
    if op == "combine":
        return (s["y"].float()[at] * w[..., None]).sum(1).to(bf)
    dout, at_row = s["dout"].float(), s["order"].long()
    dy = (dout[at_row // s["k"]] * s["weights"].flatten()[at_row][:, None]).to(bf)
    if s["kept"] is not None:
        dy = torch.where((s["ids"].flatten()[at_row] >= 0)[:, None], dy, s["kept"])
    dweights = (s["y"].float()[at] * dout[:, None]).sum(-1)
    return dy, torch.where(live, dweights, 0.0)


# ----------------------------------------------------------------- 64 bits
def _route64(s):
    """The choice one after another, the first of the largest that are left; each
    gradient from the derivatives of the weights' definition."""
    l = s["logits"].double()
    t, e = l.shape
    left, ids, probability = l.clone(), [], None
    for _ in range(min(s["k"], e)):
        m = left.amax(1, keepdim=True)
        hit = left == m
        hit &= hit.cumsum(1) == 1
        ids.append(torch.where(m[:, 0] > -math.inf, hit.int().argmax(1), -1))
        left = left.masked_fill(hit, -math.inf)
    ids = torch.stack(ids, 1)
    live = ids >= 0
    one = torch.zeros(t, s["k"], e, dtype=torch.float64, device=l.device)
    one.scatter_(2, ids.clamp(min=0)[..., None], live[..., None].double())
    finite = torch.where(l > -math.inf, l, -1e9)
    if s["score"] == "softmax":
        a = torch.exp(finite - finite.amax(1, keepdim=True)) * (l > -math.inf)
        rate = torch.ones_like(a)                                   # d log a / d l
    else:
        a = 1 / (1 + torch.exp(-finite))
        rate = 1 - a
    chosen = (one * a[:, None]).sum(2)
    if s["normalize"]:
        total, part = chosen.sum(1, keepdim=True), one.sum(1)
    else:
        total, part = (a.sum(1, keepdim=True), torch.ones_like(a)) if s["score"] == "softmax" else (None, None)
    if total is None:
        weights = chosen
        d = (one * (s["dweights"].double() * chosen)[..., None]).sum(1) * rate
    else:
        total = torch.where(total > 0, total, 1.0)
        weights = chosen / total
        g = s["dweights"].double() * live
        inner = (g * weights).sum(1, keepdim=True)
        d = ((one * g[..., None]).sum(1) - part * inner) * a * rate / total
    return ids, weights, d


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        if case["tokens"] * case["experts"] * case["k"] > 1 << 26:
            return None
        ids, weights, d = _route64(s)
        return (None, weights, d) if case["back"] else (None, weights)
    if op.startswith("glu"):
        w = torch.index_select(s["weights"].double(), 0, s["order"].long()).unsqueeze(1)
        c = math.sqrt(2 / math.pi)
        if op == "glu back":
            v = s["xq"].view(torch.float8_e4m3fn).double() * torch.exp2(s["xs"].double() - 127).repeat_interleave(32, 1)
        else:
            v = s["x"].double()
        gate, up = v[:, :case["inner"]], v[:, case["inner"]:]
        if case["act"] == "silu":
            act = gate / (1 + torch.exp(-gate))
            slope = (1 + torch.exp(-gate) * (1 + gate)) / (1 + torch.exp(-gate)).square()
        else:
            th = torch.tanh(c * (gate + 0.044715 * gate.pow(3)))
            act = gate / 2 * (1 + th)
            slope = (1 + th) / 2 + gate / 2 * (1 - th.square()) * c * (1 + 0.134145 * gate.square())
        if op == "glu back":
            dy = s["dy"].double()
            dw = torch.zeros(case["rows"], dtype=torch.float64, device="cuda")
            dw.index_add_(0, s["order"].long(), (dy * act * up).sum(1))
            return torch.cat((dy * w * up * slope, dy * w * act), 1), dw

        def eight(a):
            b = a.reshape(a.shape[0], -1, 32)
            m = b.abs().amax(-1, keepdim=True)
            e = torch.floor(torch.log2(torch.where(m > 0, m, 1.0)))
            e = torch.where(torch.exp2(e) > m, e - 1, torch.where(torch.exp2(e + 1) <= m, e + 1, e))
            scale = torch.exp2(torch.where(m > 0, (e - 8).clamp(-127, 127), -127.0))
            return (b / scale).clamp(-448, 448).reshape(a.shape), scale[..., 0]

        y = act * up * w
        return eight(y) if op == "glu8" else (y, *eight(v))
    if op.startswith("dispatch"):
        # moved, not computed: each expert's slots one after another
        flat = s["ids"].flatten()
        slots = torch.cat([torch.nonzero(flat == e)[:, 0] for e in range(case["experts"])])

        def rows(x, kept):
            out = torch.zeros(flat.numel(), x.shape[1], dtype=torch.float64, device="cuda") if kept is None else kept.double()
            out[:slots.numel()] = x.double()[slots // case["k"]]
            return out

        if op == "dispatch":
            return None, None, None, rows(s["x"], s["kept"])
        eight = (s["xq"].view(torch.float8_e4m3fn), s["xs"].view(torch.float8_e8m0fnu))
        kept = (None, None) if s["kept"] is None else (s["kept"][0].view(eight[0].dtype), s["kept"][1].view(eight[1].dtype))
        return None, None, None, rows(eight[0], kept[0]), rows(eight[1], kept[1])
    y, w, p = s["y"].double(), s["weights"].double(), s["position"].long()
    dout = s["dout"].double()
    if op == "combine":
        out = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            out += torch.where(p[:, j:j + 1] >= 0, w[:, j:j + 1] * y[p[:, j].clamp(min=0)], 0.0)
        return out
    dy, dw = torch.zeros_like(y), torch.zeros_like(w)
    for j in range(case["k"]):
        t = torch.nonzero(p[:, j] >= 0)[:, 0]
        dy[p[t, j]] = w[t, j:j + 1] * dout[t]
        dw[t, j] = (y[p[t, j]] * dout[t]).sum(1)
    return dy, dw
