// torch_binding.hpp -- what the binding's functions share: checks of arguments,
// allocation of outputs, errors, and the functions themselves for the module's table.
#pragma once

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>

#include <cstdarg>
#include <string>
#include <tuple>
#include <utility>
#include <vector>

#include "fp4.h"

namespace fp4py {

inline PyObject* fp4_error = nullptr;      // the package's Fp4Error

using Shape = std::vector<int64_t>;

// Raises `cls` with a printf-like message.
[[noreturn]] inline void fail(PyObject* cls, const char* format, ...) {
    va_list args;
    va_start(args, format);
    PyErr_FormatV(cls, format, args);
    va_end(args);
    throw python_error();
}

inline std::string text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

inline const char* type_text(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kByte: return "torch.uint8";
        case at::kInt: return "torch.int32";
        default: return "torch.float32";
    }
}

inline const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a tensor, got %s", name, Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

// A contiguous tensor of that type and shape on `like`'s device (a GPU).
inline const at::Tensor& need(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape, const at::Tensor& like,
                       const char* name) {
    if (t.sizes() != shape)
        fail(PyExc_ValueError, "%s must have shape %s, got %s", name, text(shape).c_str(), text(t.sizes()).c_str());
    if (t.scalar_type() != type)
        fail(PyExc_TypeError, "%s must be %s, got %s", name, type_text(type), c10::toString(t.scalar_type()));
    if (!t.is_cuda() || t.device() != like.device())
        fail(PyExc_ValueError, "%s must be a GPU tensor on %s, got one on %s", name, like.device().str().c_str(),
                                t.device().str().c_str());
    if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", name);
    return t;
}

inline const at::Tensor& need(PyObject* o, at::ScalarType type, at::IntArrayRef shape, const at::Tensor& like,
                       const char* name) {
    return need(tensor(o, name), type, shape, like, name);
}

inline const at::Tensor& matrix(PyObject* o, at::ScalarType type, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != 2) fail(PyExc_ValueError, "%s must have two dimensions, got shape %s", name, text(t.sizes()).c_str());
    return need(t, type, t.sizes(), t, name);
}

// A new tensor on `like`'s device, which is the current one: torch's caching
// allocator without the dispatch of at::empty (a norm's call with its four
// outputs 6.4 against 7.1 us).
inline at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
    return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

// New tensors in one allocation, each at a multiple of 512 bytes: outputs that live
// and die together, or are small.  An allocation costs 0.5 us of a call's 4 to 5, a
// tensor in one 0.1.
inline std::vector<at::Tensor> empty_together(const at::Tensor& like,
                                              std::initializer_list<std::pair<Shape, at::ScalarType>> parts) {
    auto bytes = [](const std::pair<Shape, at::ScalarType>& p) {
        int64_t n = (int64_t)c10::elementSize(p.second);
        for (const int64_t s : p.first) n *= s;
        return n;
    };
    int64_t total = 0;
    for (const auto& p : parts) total += (bytes(p) + 511) / 512 * 512;
    const c10::Storage storage = empty({total}, at::kByte, like).storage();
    std::vector<at::Tensor> out;
    int64_t at = 0;
    for (const auto& p : parts) {
        at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(storage), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                                c10::scalarTypeToTypeMeta(p.second));
        t.unsafeGetTensorImpl()->set_storage_offset(at / (int64_t)c10::elementSize(p.second));
        t.unsafeGetTensorImpl()->set_sizes_contiguous(p.first);
        out.push_back(std::move(t));
        at += (bytes(p) + 511) / 512 * 512;
    }
    return out;
}

template <typename T = void>
T* ptr(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }

inline void check(fp4_status s) {
    if (s == FP4_OK) return;
    PyObject* e = PyObject_CallFunction(fp4_error, "is", (int)s, fp4_status_string(s));
    if (e) {
        PyErr_SetObject(fp4_error, e);
        Py_DECREF(e);
    }
    throw python_error();
}

inline int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
// an enumeration's value, or a size of a few bits; what is no int is none of them
template <typename E>
E option(PyObject* o) {
    const int64_t v = integer(o);
    if (v != (int)v) check(FP4_ERR_ENUM);
    return static_cast<E>(v);
}
// seeds: the low 64 bits of any Python integer
inline uint64_t seed(PyObject* o) {
    const unsigned long long v = PyLong_AsUnsignedLongLongMask(o);
    if (PyErr_Occurred()) throw python_error();
    return v;
}
// a stream's handle as an integer; None: the current stream of like's device
inline void* stream(PyObject* o, const at::Tensor& like) {
    if (o == Py_None) return c10::hip::getCurrentHIPStream(like.device().index()).stream();
    return reinterpret_cast<void*>(static_cast<uintptr_t>(seed(o)));
}

inline void arguments(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) fail(PyExc_TypeError, "%d arguments expected, got %d", (int)want, (int)got);
}

inline PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

template <typename... T>
PyObject* tuple(const T&... t) {
    PyObject* r = PyTuple_New(sizeof...(T));
    if (!r) throw python_error();
    Py_ssize_t i = 0;
    ((PyTuple_SET_ITEM(r, i++, wrap(t))), ...);
    return r;
}

// The items of an `out` argument: any sequence or iterator of tensors.
inline std::vector<at::Tensor> items(PyObject* o, Py_ssize_t n) {
    const THPObjectPtr f(PySequence_Fast(o, "out must be a sequence of tensors"));
    if (!f) throw python_error();
    if (PySequence_Fast_GET_SIZE(f.get()) != n)
        fail(PyExc_ValueError, "out must hold %d tensors, got %d", (int)n, (int)PySequence_Fast_GET_SIZE(f.get()));
    std::vector<at::Tensor> v;
    for (Py_ssize_t i = 0; i < n; ++i) v.push_back(tensor(PySequence_Fast_GET_ITEM(f.get(), i), "output"));
    return v;
}

inline int64_t groups32(int64_t n) { return (n + 31) / 32; }
inline Shape code_shape(int64_t R, int64_t C) { return {groups32(R), C / 32, 512}; }
inline Shape scale_shape(int64_t R, int64_t C) { return {(C / 32 + 7) / 8, R, 8}; }

inline at::ScalarType out_type(int64_t out) {
    if (out != FP4_OUT_F32 && out != FP4_OUT_BF16) check(FP4_ERR_ENUM);
    return out == FP4_OUT_BF16 ? at::kBFloat16 : at::kFloat;
}

inline at::Tensor output(PyObject* o, at::IntArrayRef shape, int64_t out, const at::Tensor& like) {
    return o == Py_None ? empty(shape, out_type(out), like) : need(o, out_type(out), shape, like, "out");
}

// the number of experts of row offsets (int32 [experts + 1])
inline int64_t experts_of(const at::Tensor& offsets, const at::Tensor& like) {
    if (offsets.dim() != 1 || offsets.size(0) < 2)
        fail(PyExc_ValueError, "offsets must be int32 [experts + 1], got shape %s", text(offsets.sizes()).c_str());
    need(offsets, at::kInt, offsets.sizes(), like, "offsets");
    return offsets.size(0) - 1;
}

#define FP4_FUNCTION(name) PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n)
FP4_FUNCTION(moe_route);
FP4_FUNCTION(moe_route_backward);
FP4_FUNCTION(moe_sort);
FP4_FUNCTION(moe_gather);
FP4_FUNCTION(moe_combine);
FP4_FUNCTION(moe_combine_backward);
FP4_FUNCTION(glu);
FP4_FUNCTION(glu_quantize);
FP4_FUNCTION(glu_backward);

}  // namespace fp4py
