// torch_binding.cpp -- the norm, grouped and few-row entry points of libfp4.so
// as CPython functions on torch tensors: checks of the arguments, allocation
// of the outputs, the call.  A served token's calls are a few microseconds of
// GPU time each, so what the host spends per call counts: the same marshalling
// in Python with ctypes measured 14 us a norm (1.7 us an output tensor, 2 us
// for the stream, 4 us the launch itself), here 6.4.
//
// Every function takes its arguments by position (the Python functions of the
// package name and document them) and the stream as an integer, or None for the
// current one.  Wrong types
// raise TypeError, wrong shapes or devices ValueError, a nonzero status the
// package's Fp4Error.
#include "torch_binding.hpp"

using namespace fp4py;

namespace {

// (x, weight, residual, eps, fmt, out, y, stream)
PyObject* rmsnorm_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 8);
    const at::Tensor& x = matrix(a[0], at::kBFloat16, "x");
    const int64_t rows = x.size(0), cols = x.size(1);
    const int fmt = option<int>(a[4]);
    const at::Tensor& w = need(a[1], at::kBFloat16, {cols}, x, "weight");
    const bool added = a[2] != Py_None;
    if (added) need(a[2], at::kBFloat16, x.sizes(), x, "residual");
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw python_error();
    const Shape cs = fmt == FP4_FMT_MXFP8 ? Shape{rows, cols} : code_shape(rows, cols);
    const Shape ss = fmt == FP4_FMT_MXFP8 ? Shape{rows, cols / 32} : scale_shape(rows, cols);
    const c10::DeviceGuard guard(x.device());
    at::Tensor codes, scales, h, rstd;
    if (a[5] == Py_None) {
        codes = empty(cs, at::kByte, x);
        scales = empty(ss, at::kByte, x);
        h = added ? empty(x.sizes(), at::kBFloat16, x) : x;
        rstd = empty({rows}, at::kFloat, x);
    } else {
        const auto o = items(a[5], 4);
        codes = need(o[0], at::kByte, cs, x, "codes");
        scales = need(o[1], at::kByte, ss, x, "scales");
        h = need(o[2], at::kBFloat16, x.sizes(), x, "h");
        rstd = need(o[3], at::kFloat, {rows}, x, "rstd");
    }
    void* y = a[6] == Py_None ? nullptr : ptr(need(a[6], at::kBFloat16, x.sizes(), x, "y"));
    const bool same = !added && ptr(h) == ptr(x);
    check(fp4_rmsnorm_quantize(ptr(x), added ? ptr(THPVariable_Unpack(a[2])) : nullptr, ptr(w), eps, rows, cols,
                               (fp4_format)fmt, same ? nullptr : ptr(h), ptr<float>(rstd), y, ptr<uint8_t>(codes),
                               ptr<uint8_t>(scales), stream(a[7], x)));
    return tuple(codes, scales, h, rstd);
    END_HANDLE_TH_ERRORS
}

// (dy, h, weight, rstd, dh, out, workspace, stream)
PyObject* rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 8);
    const at::Tensor& dy = matrix(a[0], at::kBFloat16, "dy");
    const int64_t rows = dy.size(0), cols = dy.size(1);
    const at::Tensor& h = need(a[1], at::kBFloat16, dy.sizes(), dy, "h");
    const at::Tensor& w = need(a[2], at::kBFloat16, {cols}, dy, "weight");
    const at::Tensor& rstd = need(a[3], at::kFloat, {rows}, dy, "rstd");
    void* dh = a[4] == Py_None ? nullptr : ptr(need(a[4], at::kBFloat16, dy.sizes(), dy, "dh"));
    const c10::DeviceGuard guard(dy.device());
    at::Tensor dx, dw, ws;
    if (a[5] == Py_None) {
        dx = empty(dy.sizes(), at::kBFloat16, dy);
        dw = empty({cols}, at::kFloat, dy);
    } else {
        const auto o = items(a[5], 2);
        dx = need(o[0], at::kBFloat16, dy.sizes(), dy, "dx");
        dw = need(o[1], at::kFloat, {cols}, dy, "dw");
    }
    if (a[6] == Py_None) {
        ws = empty({(int64_t)fp4_rmsnorm_workspace_bytes(rows, cols)}, at::kByte, dy);
    } else {
        ws = tensor(a[6], "workspace");
        need(ws, at::kByte, ws.sizes(), dy, "workspace");
    }
    check(fp4_rmsnorm_backward(ptr(dy), ptr(h), ptr(w), ptr<float>(rstd), dh, rows, cols, ptr(dx), ptr<float>(dw),
                               ptr(ws), (size_t)ws.numel(), stream(a[7], dy)));
    return tuple(dx, dw);
    END_HANDLE_TH_ERRORS
}

// R and C of an MXFP4 operand (or a stack of them) from its last three sizes
std::pair<int64_t, int64_t> mx_dims(at::IntArrayRef codes, at::IntArrayRef scales) {
    const size_t d = codes.size();
    if (d == scales.size() && d >= 3) {
        const int64_t R = scales[d - 2], C = codes[d - 2] * 32;
        if (codes.slice(d - 3) == at::IntArrayRef(code_shape(R, C)) &&
            scales.slice(d - 3) == at::IntArrayRef(scale_shape(R, C)))
            return {R, C};
    }
    fail(PyExc_ValueError, "codes %s and scales %s do not describe one operand", text(codes).c_str(),
                            text(scales).c_str());
}

// (aq, as, wq, ws, out, out_dtype, stream)
PyObject* gemm_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 7);
    const at::Tensor &aq = tensor(a[0], "a codes"), &as = tensor(a[1], "a scales");
    const at::Tensor &wq = tensor(a[2], "w codes"), &ws = tensor(a[3], "w scales");
    if (aq.dim() != 2 && aq.dim() != 3)
        fail(PyExc_ValueError, "a codes must have two dimensions (MXFP8) or three (MXFP4), got shape %s",
             text(aq.sizes()).c_str());
    const fp4_format fmt = aq.dim() == 2 ? FP4_FMT_MXFP8 : FP4_FMT_MXFP4;
    int64_t M, K;
    if (fmt == FP4_FMT_MXFP8) {
        M = aq.size(0);
        K = aq.size(1);
        if (as.sizes() != at::IntArrayRef({M, K / 32}))
            fail(PyExc_ValueError, "MXFP8 codes %s and scales %s do not describe one operand",
                                    text(aq.sizes()).c_str(), text(as.sizes()).c_str());
    } else {
        std::tie(M, K) = mx_dims(aq.sizes(), as.sizes());
    }
    if (wq.dim() != 3) fail(PyExc_ValueError, "w codes must have three dimensions, got shape %s", text(wq.sizes()).c_str());
    const auto [N, Kw] = mx_dims(wq.sizes(), ws.sizes());
    if (K != Kw)
        fail(PyExc_ValueError, "decode operands have different contraction sizes (%lld, %lld)", (long long)K, (long long)Kw);
    need(aq, at::kByte, aq.sizes(), aq, "a codes");
    need(as, at::kByte, as.sizes(), aq, "a scales");
    need(wq, at::kByte, wq.sizes(), aq, "w codes");
    need(ws, at::kByte, ws.sizes(), aq, "w scales");
    const c10::DeviceGuard guard(aq.device());
    const int64_t od = integer(a[5]);
    const at::Tensor c = output(a[4], {M, N}, od, aq);
    check(fp4_gemm_decode(ptr<uint8_t>(aq), ptr<uint8_t>(as), fmt, ptr<uint8_t>(wq), ptr<uint8_t>(ws), M, N, K,
                          ptr(c), (fp4_out_dtype)od, stream(a[6], aq)));
    return wrap(c);
    END_HANDLE_TH_ERRORS
}

Shape grouped_codes(int64_t rows, int64_t cols, int64_t E, bool along_rows) {
    return along_rows ? Shape{cols / 32, 8 * FP4_GROUPED_STAGES(rows, E), 512}
                      : Shape{FP4_GROUPED_UNITS(rows, E), cols / 32, 512};
}
Shape grouped_scales(int64_t rows, int64_t cols, int64_t E, bool along_rows) {
    return along_rows ? Shape{FP4_GROUPED_STAGES(rows, E), cols, 8}
                      : scale_shape(32 * FP4_GROUPED_UNITS(rows, E), cols);
}

// (x, offsets, axes: 1 cols, 2 rows, 3 both (rows first), had_n, had, sign_seed,
//  rnd, sr_seed_rows, sr_seed_cols, out, stream)
PyObject* quantize_grouped(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 11);
    const at::Tensor& x = matrix(a[0], at::kBFloat16, "x");
    const at::Tensor& off = tensor(a[1], "offsets");
    const int64_t rows = x.size(0), cols = x.size(1), E = experts_of(off, x), axes = integer(a[2]);
    const c10::DeviceGuard guard(x.device());
    std::vector<at::Tensor> given;
    if (a[9] != Py_None) given = items(a[9], axes == 3 ? 4 : 2);
    at::Tensor out[4];
    int m = 0;
    for (const bool along_rows : {true, false}) {
        if (!(axes & (along_rows ? 2 : 1))) continue;
        for (const Shape& s : {grouped_codes(rows, cols, E, along_rows), grouped_scales(rows, cols, E, along_rows)}) {
            out[m] = given.empty() ? empty(s, at::kByte, x) : need(given[m], at::kByte, s, x, "output");
            ++m;
        }
    }
    uint8_t* p[4] = {};                                // rows codes, rows scales, cols codes, cols scales
    for (int i = 0; i < m; ++i) p[axes == 1 ? i + 2 : i] = ptr<uint8_t>(out[i]);
    check(fp4_quantize_grouped(ptr(x), ptr<int32_t>(off), E, rows, cols, option<int>(a[3]),
                               option<fp4_hadamard>(a[4]), seed(a[5]), option<fp4_rounding>(a[6]), seed(a[7]),
                               seed(a[8]), p[0], p[1], p[2], p[3], stream(a[10], x)));
    return axes == 3 ? tuple(out[0], out[1], out[2], out[3]) : tuple(out[0], out[1]);
    END_HANDLE_TH_ERRORS
}

// (aq, as, offsets, wq, ws, rows, out, out_dtype, stream)
PyObject* gemm_grouped(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 9);
    const at::Tensor &aq = tensor(a[0], "a codes"), &as = tensor(a[1], "a scales"), &off = tensor(a[2], "offsets");
    const at::Tensor &wq = tensor(a[3], "w codes"), &ws = tensor(a[4], "w scales");
    const int64_t E = experts_of(off, aq), rows = integer(a[5]);
    if (wq.dim() != 4 || ws.dim() != 4 || wq.size(0) != E || ws.size(0) != E)
        fail(PyExc_ValueError, "weights must be codes [experts, ceil(N/32), K/32, 512] and scales [experts, ceil(K/256), N, 8] of %lld "
            "experts, got %s and %s", (long long)E, text(wq.sizes()).c_str(), text(ws.sizes()).c_str());
    const auto [N, K] = mx_dims(wq.sizes(), ws.sizes());
    const fp4_format fmt = aq.dim() == 2 ? FP4_FMT_MXFP8 : FP4_FMT_MXFP4;
    need(aq, at::kByte, fmt == FP4_FMT_MXFP8 ? Shape{rows, K} : grouped_codes(rows, K, E, false), aq, "a codes");
    need(as, at::kByte, fmt == FP4_FMT_MXFP8 ? Shape{rows, K / 32} : grouped_scales(rows, K, E, false), aq, "a scales");
    need(wq, at::kByte, wq.sizes(), aq, "w codes");
    need(ws, at::kByte, ws.sizes(), aq, "w scales");
    const c10::DeviceGuard guard(aq.device());
    const int64_t od = integer(a[7]);
    const at::Tensor c = output(a[6], {rows, N}, od, aq);
    check(fp4_gemm_grouped(ptr<uint8_t>(aq), ptr<uint8_t>(as), fmt, ptr<int32_t>(off), E, rows, ptr<uint8_t>(wq),
                           ptr<uint8_t>(ws), N, K, ptr(c), (fp4_out_dtype)od, stream(a[8], aq)));
    return wrap(c);
    END_HANDLE_TH_ERRORS
}

// (dytq, dyts, xtq, xts, offsets, rows, out, out_dtype, stream)
PyObject* gemm_grouped_wgrad(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 9);
    const at::Tensor &dq = tensor(a[0], "dY codes"), &ds = tensor(a[1], "dY scales");
    const at::Tensor &xq = tensor(a[2], "X codes"), &xs = tensor(a[3], "X scales"), &off = tensor(a[4], "offsets");
    const int64_t E = experts_of(off, dq), rows = integer(a[5]);
    if (ds.dim() != 3 || xs.dim() != 3) fail(PyExc_ValueError, "scales must have three dimensions");
    const int64_t N = ds.size(1), K = xs.size(1);
    need(dq, at::kByte, grouped_codes(rows, N, E, true), dq, "dY codes");
    need(ds, at::kByte, grouped_scales(rows, N, E, true), dq, "dY scales");
    need(xq, at::kByte, grouped_codes(rows, K, E, true), dq, "X codes");
    need(xs, at::kByte, grouped_scales(rows, K, E, true), dq, "X scales");
    const c10::DeviceGuard guard(dq.device());
    const int64_t od = integer(a[7]);
    const at::Tensor c = output(a[6], {E, N, K}, od, dq);
    check(fp4_gemm_grouped_wgrad(ptr<uint8_t>(dq), ptr<uint8_t>(ds), ptr<uint8_t>(xq), ptr<uint8_t>(xs),
                                 ptr<int32_t>(off), E, rows, N, K, ptr(c), (fp4_out_dtype)od, stream(a[8], dq)));
    return wrap(c);
    END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
    Py_XDECREF(fp4_error);
    Py_INCREF(cls);
    fp4_error = cls;
    Py_RETURN_NONE;
}

#define FP4_METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FP4_METHOD(rmsnorm_quantize), FP4_METHOD(rmsnorm_backward), FP4_METHOD(gemm_decode),
                         FP4_METHOD(quantize_grouped), FP4_METHOD(gemm_grouped), FP4_METHOD(gemm_grouped_wgrad),
                         FP4_METHOD(moe_route), FP4_METHOD(moe_route_backward), FP4_METHOD(moe_sort),
                         FP4_METHOD(moe_gather), FP4_METHOD(moe_combine), FP4_METHOD(moe_combine_backward),
                         FP4_METHOD(glu), FP4_METHOD(glu_quantize), FP4_METHOD(glu_backward),
                         {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_torch_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_binding() { return PyModule_Create(&module_def); }
