// torch_binding_moe.cpp -- the entry points around the experts' products as CPython
// functions on torch tensors (see torch_binding.cpp): router, sorted slots, rows
// gathered and combined, gated activation.
#include "torch_binding.hpp"

namespace fp4py {

namespace {

at::ScalarType logits_type(const at::Tensor& t, const char* name) {
    if (t.scalar_type() != at::kFloat && t.scalar_type() != at::kBFloat16)
        fail(PyExc_TypeError, "%s must be torch.float32 or torch.bfloat16, got %s", name, c10::toString(t.scalar_type()));
    return t.scalar_type();
}

// Logits [T, E].
const at::Tensor& logits_of(PyObject* o) {
    return matrix(o, logits_type(tensor(o, "logits"), "logits"), "logits");
}

fp4_out_dtype dtype_of(const at::Tensor& t) { return t.scalar_type() == at::kBFloat16 ? FP4_OUT_BF16 : FP4_OUT_F32; }

// position int32 [T, k] on like's device, T as given
const at::Tensor& position_of(PyObject* o, int64_t tokens, const at::Tensor& like) {
    const at::Tensor& t = tensor(o, "position");
    if (t.dim() != 2 || (tokens >= 0 && t.size(0) != tokens))
        fail(PyExc_ValueError, "position must be int32 [tokens, k], got shape %s for %lld tokens", text(t.sizes()).c_str(),
             (long long)tokens);
    return need(t, at::kInt, t.sizes(), like, "position");
}

int truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v;
}

// A tensor of `count` elements in any shape, null for None.
const at::Tensor* counted(PyObject* o, at::ScalarType type, int64_t count, const at::Tensor& like, const char* name) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.numel() != count)
        fail(PyExc_ValueError, "%s must hold one value for each of %lld rows, got shape %s", name, (long long)count,
             text(t.sizes()).c_str());
    return &need(t, type, t.sizes(), like, name);
}

// weights, order and offsets of the gated activation's rows
struct RowArgs {
    const at::Tensor *weights, *order, *offsets;
    int64_t experts;
    const float* w() const { return weights ? ptr<float>(*weights) : nullptr; }
    const int32_t* o() const { return order ? ptr<int32_t>(*order) : nullptr; }
    const int32_t* off() const { return offsets ? ptr<int32_t>(*offsets) : nullptr; }
};
RowArgs row_args(PyObject* weights, PyObject* order, PyObject* offsets, int64_t rows, const at::Tensor& like) {
    RowArgs r{counted(weights, at::kFloat, rows, like, "weights"), counted(order, at::kInt, rows, like, "order"), nullptr, 0};
    if (offsets != Py_None) {
        r.offsets = &tensor(offsets, "offsets");
        r.experts = experts_of(*r.offsets, like);
    }
    return r;
}

// x [rows, 2 cols] of the gated activation
const at::Tensor& gate_and_up(PyObject* o) {
    const at::Tensor& x = matrix(o, at::kBFloat16, "x");
    if (x.size(1) % 2) fail(PyExc_ValueError, "x must hold gate and up side by side, got shape %s", text(x.sizes()).c_str());
    return x;
}

}  // namespace

// (logits, k, score, normalize, out, stream)
FP4_FUNCTION(moe_route) {
    HANDLE_TH_ERRORS
    arguments(n, 6);
    const at::Tensor& l = logits_of(a[0]);
    const int64_t T = l.size(0), E = l.size(1), k = integer(a[1]);
    if (k <= 0 || k > 64) check(FP4_ERR_SHAPE);        // before outputs of that size are allocated
    const c10::DeviceGuard guard(l.device());
    at::Tensor ids, weights;
    if (a[4] == Py_None) {
        const auto o = empty_together(l, {{{T, k}, at::kInt}, {{T, k}, at::kFloat}});
        ids = o[0];
        weights = o[1];
    } else {
        const auto o = items(a[4], 2);
        ids = need(o[0], at::kInt, {T, k}, l, "ids");
        weights = need(o[1], at::kFloat, {T, k}, l, "weights");
    }
    check(fp4_moe_route(ptr(l), dtype_of(l), T, E, k, option<fp4_score>(a[2]), truth(a[3]), ptr<int32_t>(ids),
                        ptr<float>(weights), stream(a[5], l)));
    return tuple(ids, weights);
    END_HANDLE_TH_ERRORS
}

// (dweights, logits, ids, score, normalize, out, stream)
FP4_FUNCTION(moe_route_backward) {
    HANDLE_TH_ERRORS
    arguments(n, 7);
    const at::Tensor& l = logits_of(a[1]);
    const at::Tensor& ids = matrix(a[2], at::kInt, "ids");
    const int64_t T = l.size(0), E = l.size(1), k = ids.size(1);
    need(ids, at::kInt, {T, k}, l, "ids");
    const at::Tensor& dw = need(a[0], at::kFloat, {T, k}, l, "dweights");
    const c10::DeviceGuard guard(l.device());
    const at::Tensor d = a[5] == Py_None ? empty({T, E}, l.scalar_type(), l) : need(a[5], l.scalar_type(), {T, E}, l, "out");
    check(fp4_moe_route_backward(ptr<float>(dw), ptr(l), dtype_of(l), ptr<int32_t>(ids), T, E, k,
                                 option<fp4_score>(a[3]), truth(a[4]), ptr(d), stream(a[6], l)));
    return wrap(d);
    END_HANDLE_TH_ERRORS
}

// (ids, experts, out, workspace, stream)
FP4_FUNCTION(moe_sort) {
    HANDLE_TH_ERRORS
    arguments(n, 5);
    const at::Tensor& ids = matrix(a[0], at::kInt, "ids");
    const int64_t slots = ids.numel(), E = integer(a[1]);
    if (E <= 0 || E > 1024) check(FP4_ERR_SHAPE);      // before an output of that size is allocated
    const c10::DeviceGuard guard(ids.device());
    at::Tensor offsets, order, position, ws;
    if (a[2] == Py_None) {
        const auto o = empty_together(ids, {{{E + 1}, at::kInt}, {{slots}, at::kInt}, {ids.sizes().vec(), at::kInt}});
        offsets = o[0];
        order = o[1];
        position = o[2];
    } else {
        const auto o = items(a[2], 3);
        offsets = need(o[0], at::kInt, {E + 1}, ids, "offsets");
        order = need(o[1], at::kInt, {slots}, ids, "order");
        position = need(o[2], at::kInt, ids.sizes(), ids, "position");
    }
    const int64_t bytes = (int64_t)fp4_moe_sort_workspace_bytes(slots, E);
    if (a[3] != Py_None) {
        ws = tensor(a[3], "workspace");
        need(ws, at::kByte, ws.sizes(), ids, "workspace");
    } else if (bytes) {
        ws = empty({bytes}, at::kByte, ids);
    }
    check(fp4_moe_sort(ptr<int32_t>(ids), slots, E, ptr<int32_t>(offsets), ptr<int32_t>(order), ptr<int32_t>(position),
                       ws.defined() ? ptr(ws) : nullptr, ws.defined() ? (size_t)ws.numel() : 0, stream(a[4], ids)));
    return tuple(offsets, order, position);
    END_HANDLE_TH_ERRORS
}

// (x, position, scales, out, stream)
FP4_FUNCTION(moe_gather) {
    HANDLE_TH_ERRORS
    arguments(n, 5);
    const bool eight = a[2] != Py_None;
    const at::ScalarType type = eight ? at::kByte : at::kBFloat16;
    const at::Tensor& x = matrix(a[0], type, "x");
    const int64_t T = x.size(0), cols = x.size(1);
    const at::Tensor& p = position_of(a[1], T, x);
    const int64_t k = p.size(1);
    const at::Tensor* s = eight ? &need(a[2], at::kByte, {T, cols / 32}, x, "scales") : nullptr;
    const c10::DeviceGuard guard(x.device());
    at::Tensor out, os;
    int64_t rows = T * k;
    // a given `out` may hold any number of rows
    auto given = [&](const at::Tensor& t, int64_t width, const char* name) {
        if (t.dim() != 2) fail(PyExc_ValueError, "%s must have two dimensions, got shape %s", name, text(t.sizes()).c_str());
        return need(t, type, {t.size(0), width}, x, name);
    };
    if (a[3] == Py_None) {
        if (eight) {
            const auto o = empty_together(x, {{{rows, cols}, type}, {{rows, cols / 32}, type}});
            out = o[0];
            os = o[1];
        } else {
            out = empty({rows, cols}, type, x);
        }
    } else if (eight) {
        const auto o = items(a[3], 2);
        out = given(o[0], cols, "out");
        rows = out.size(0);
        os = need(o[1], at::kByte, {rows, cols / 32}, x, "out scales");
    } else {
        out = given(tensor(a[3], "out"), cols, "out");
        rows = out.size(0);
    }
    check(fp4_moe_gather(ptr(x), s ? ptr<uint8_t>(*s) : nullptr, ptr<int32_t>(p), T, k, rows, cols, ptr(out),
                         eight ? ptr<uint8_t>(os) : nullptr, stream(a[4], x)));
    return eight ? tuple(out, os) : wrap(out);
    END_HANDLE_TH_ERRORS
}

// (y, position, weights, out, stream)
FP4_FUNCTION(moe_combine) {
    HANDLE_TH_ERRORS
    arguments(n, 5);
    const at::Tensor& y = matrix(a[0], at::kBFloat16, "y");
    const at::Tensor& p = position_of(a[1], -1, y);
    const int64_t T = p.size(0), k = p.size(1), rows = y.size(0), cols = y.size(1);
    const float* w = a[2] == Py_None ? nullptr : ptr<float>(need(a[2], at::kFloat, {T, k}, y, "weights"));
    const c10::DeviceGuard guard(y.device());
    const at::Tensor out = a[3] == Py_None ? empty({T, cols}, at::kBFloat16, y) : need(a[3], at::kBFloat16, {T, cols}, y, "out");
    check(fp4_moe_combine(ptr(y), ptr<int32_t>(p), w, T, k, rows, cols, ptr(out), stream(a[4], y)));
    return wrap(out);
    END_HANDLE_TH_ERRORS
}

// (dout, y, position, weights, out, stream)
FP4_FUNCTION(moe_combine_backward) {
    HANDLE_TH_ERRORS
    arguments(n, 6);
    const at::Tensor& y = matrix(a[1], at::kBFloat16, "y");
    const at::Tensor& p = position_of(a[2], -1, y);
    const int64_t T = p.size(0), k = p.size(1), rows = y.size(0), cols = y.size(1);
    const at::Tensor& d = need(a[0], at::kBFloat16, {T, cols}, y, "dout");
    const at::Tensor& w = need(a[3], at::kFloat, {T, k}, y, "weights");
    const c10::DeviceGuard guard(y.device());
    at::Tensor dy, dw;
    if (a[4] == Py_None) {
        dy = empty({rows, cols}, at::kBFloat16, y);
        dw = empty({T, k}, at::kFloat, y);
    } else {
        const auto o = items(a[4], 2);
        dy = need(o[0], at::kBFloat16, {rows, cols}, y, "dy");
        dw = need(o[1], at::kFloat, {T, k}, y, "dweights");
    }
    check(fp4_moe_combine_backward(ptr(d), ptr(y), ptr<int32_t>(p), ptr<float>(w), T, k, rows, cols, ptr(dy),
                                   ptr<float>(dw), stream(a[5], y)));
    return tuple(dy, dw);
    END_HANDLE_TH_ERRORS
}

// (x, act, weights, order, offsets, checkpoint, out, stream)
FP4_FUNCTION(glu) {
    HANDLE_TH_ERRORS
    arguments(n, 8);
    const at::Tensor& x = gate_and_up(a[0]);
    const int64_t rows = x.size(0), cols = x.size(1) / 2;
    const RowArgs r = row_args(a[2], a[3], a[4], rows, x);
    const bool kept = truth(a[5]);
    const c10::DeviceGuard guard(x.device());
    at::Tensor y, xq, xs;
    const Shape ys{rows, cols}, qs{rows, 2 * cols}, ss{rows, 2 * cols / 32};
    if (a[6] == Py_None) {
        y = empty(ys, at::kBFloat16, x);
        if (kept) xq = empty(qs, at::kByte, x), xs = empty(ss, at::kByte, x);
    } else if (kept) {
        const auto o = items(a[6], 3);
        y = need(o[0], at::kBFloat16, ys, x, "y");
        xq = need(o[1], at::kByte, qs, x, "checkpoint codes");
        xs = need(o[2], at::kByte, ss, x, "checkpoint scales");
    } else {
        y = need(a[6], at::kBFloat16, ys, x, "out");
    }
    check(fp4_glu(ptr(x), r.w(), r.o(), r.off(), r.experts, option<fp4_act>(a[1]), rows, cols, ptr(y), FP4_FMT_MXFP8,
                  nullptr, nullptr, kept ? ptr<uint8_t>(xq) : nullptr, kept ? ptr<uint8_t>(xs) : nullptr, stream(a[7], x)));
    return kept ? tuple(y, xq, xs) : wrap(y);
    END_HANDLE_TH_ERRORS
}

// (x, act, weights, order, offsets, fmt, out, stream)
FP4_FUNCTION(glu_quantize) {
    HANDLE_TH_ERRORS
    arguments(n, 8);
    const at::Tensor& x = gate_and_up(a[0]);
    const int64_t rows = x.size(0), cols = x.size(1) / 2;
    const int fmt = option<int>(a[5]);
    const RowArgs r = row_args(a[2], a[3], a[4], rows, x);
    const Shape cs = fmt == FP4_FMT_MXFP8 ? Shape{rows, cols} : code_shape(rows, cols);
    const Shape ss = fmt == FP4_FMT_MXFP8 ? Shape{rows, cols / 32} : scale_shape(rows, cols);
    const c10::DeviceGuard guard(x.device());
    at::Tensor codes, scales;
    if (a[6] == Py_None) {
        const auto o = empty_together(x, {{cs, at::kByte}, {ss, at::kByte}});
        codes = o[0];
        scales = o[1];
    } else {
        const auto o = items(a[6], 2);
        codes = need(o[0], at::kByte, cs, x, "codes");
        scales = need(o[1], at::kByte, ss, x, "scales");
    }
    check(fp4_glu(ptr(x), r.w(), r.o(), r.off(), r.experts, option<fp4_act>(a[1]), rows, cols, nullptr, (fp4_format)fmt,
                  ptr<uint8_t>(codes), ptr<uint8_t>(scales), nullptr, nullptr, stream(a[7], x)));
    return tuple(codes, scales);
    END_HANDLE_TH_ERRORS
}

// (dy, xq, xs, act, weights, order, offsets, out, stream)
FP4_FUNCTION(glu_backward) {
    HANDLE_TH_ERRORS
    arguments(n, 9);
    const at::Tensor& dy = matrix(a[0], at::kBFloat16, "dy");
    const int64_t rows = dy.size(0), cols = dy.size(1);
    const at::Tensor& xq = need(a[1], at::kByte, {rows, 2 * cols}, dy, "checkpoint codes");
    const at::Tensor& xs = need(a[2], at::kByte, {rows, 2 * cols / 32}, dy, "checkpoint scales");
    const RowArgs r = row_args(a[4], a[5], a[6], rows, dy);
    const c10::DeviceGuard guard(dy.device());
    at::Tensor dx, dw;
    if (a[7] == Py_None) {
        dx = empty({rows, 2 * cols}, at::kBFloat16, dy);
        if (r.weights) dw = empty(r.weights->sizes(), at::kFloat, dy);
    } else if (r.weights) {
        const auto o = items(a[7], 2);
        dx = need(o[0], at::kBFloat16, {rows, 2 * cols}, dy, "dx");
        dw = need(o[1], at::kFloat, r.weights->sizes(), dy, "dweights");
    } else {
        dx = need(a[7], at::kBFloat16, {rows, 2 * cols}, dy, "out");
    }
    check(fp4_glu_backward(ptr(dy), ptr<uint8_t>(xq), ptr<uint8_t>(xs), r.w(), r.o(), r.off(), r.experts,
                           option<fp4_act>(a[3]), rows, cols, ptr(dx), r.weights ? ptr<float>(dw) : nullptr,
                           stream(a[8], dy)));
    return r.weights ? tuple(dx, dw) : wrap(dx);
    END_HANDLE_TH_ERRORS
}

}  // namespace fp4py
