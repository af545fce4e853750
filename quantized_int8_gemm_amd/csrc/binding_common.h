// What the extension modules share: checks of arguments (TypeError, ValueError),
// tensors seen as matrices, and the call on the tensors' device and stream.
#pragma once
#include <string>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include "../../include/qgemm.h"

namespace {

using at::Tensor;

// The function that raises for a status, as the package hands it over.
PyObject* raise_status;

// ---------------------------------------------------------------------------
// Arguments
// ---------------------------------------------------------------------------

std::string str(at::IntArrayRef v) {
    std::string s = "(";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + (v.size() == 1 ? ",)" : ")");
}

[[noreturn]] void type_error(const std::string& s) {
    PyErr_SetString(PyExc_TypeError, s.c_str());
    throw python_error();
}
[[noreturn]] void value_error(const std::string& s) {
    PyErr_SetString(PyExc_ValueError, s.c_str());
    throw python_error();
}

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

// None: an undefined tensor.
const Tensor& tensor_or_none(PyObject* o, const char* name) {
    static const Tensor none;
    return o == Py_None ? none : tensor(o, name);
}

[[noreturn]] void wrong_dtype(const Tensor& t, const char* name, const char* expected) {
    type_error(std::string(name) + " has dtype " + c10::toString(t.scalar_type()) + "; expected " + expected);
}

// The library's number for a floating type, or -1.
int float_kind(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return QG_FP32;
        case at::kBFloat16: return QG_BF16;
        case at::kHalf: return QG_FP16;
        default: return -1;
    }
}

qg_dtype need_float(const Tensor& t, const char* name) {
    const int k = float_kind(t.scalar_type());
    if (k < 0) wrong_dtype(t, name, "float32, bfloat16 or float16");
    return (qg_dtype)k;
}

void need_dtype(const Tensor& t, at::ScalarType d, const char* name) {
    if (t.scalar_type() != d) wrong_dtype(t, name, c10::toString(d));
}

at::ScalarType dtype_arg(PyObject* o, const char* what) {
    if (!THPDtype_Check(o)) type_error(what);
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

// A tensor seen as a matrix of its last dimension: rows, columns and row stride
// in elements.  More than two dimensions have to lie like one matrix; without rows
// nothing lies anywhere.
struct Matrix { int64_t rows, n, ld; };

Matrix matrix(const Tensor& t, const char* name) {
    const at::IntArrayRef size = t.sizes(), stride = t.strides();
    const int64_t d = (int64_t)size.size();
    if (d == 0) value_error(std::string(name) + " must have at least one dimension");
    const int64_t n = size[d - 1];
    for (int64_t i = 0; i < d - 1; ++i)
        if (size[i] == 0) return {0, n, n};
    if (n > 1 && stride[d - 1] != 1) value_error(std::string(name) + " must have unit column stride");
    int64_t rows = 1, ld = -1;
    for (int64_t i = d - 2; i >= 0; --i) {
        if (size[i] == 1) continue;
        if (ld < 0) ld = stride[i];
        else if (stride[i] != ld * rows) value_error("the rows of " + std::string(name) + " must lie at one stride");
        rows *= size[i];
    }
    if (rows > 1 && ld < n) value_error("the rows of " + std::string(name) + " overlap");
    return {rows, n, rows > 1 ? ld : n};
}

// Every tensor (undefined ones left out) on t's GPU.
void on_gpu(const Tensor& t) {
    if (!t.is_cuda()) value_error("tensors must be on a GPU device");
}
template <typename... More>
void on_gpu(const Tensor& t, const Tensor& o, const More&... more) {
    if (o.defined()) {
        if (!o.is_cuda()) value_error("tensors must be on a GPU device");
        if (t.is_cuda() && o.get_device() != t.get_device()) value_error("tensors must be on the same device");
    }
    on_gpu(t, more...);
}

void need_like(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType d) {
    need_dtype(t, d, name);
    if (t.sizes() != shape) value_error(std::string(name) + " has shape " + str(t.sizes()) + "; expected " + str(shape));
}

Tensor weight_of(const Tensor& w, int64_t n, at::ScalarType d) {
    if (w.scalar_type() != d && w.scalar_type() != at::kFloat) wrong_dtype(w, "weight", "x's dtype or float32");
    if (w.dim() != 1 || w.size(0) != n) value_error("weight has shape " + str(w.sizes()) + "; expected (" + std::to_string(n) + ",)");
    return w.contiguous();
}

Tensor make(at::IntArrayRef shape, at::ScalarType d, const Tensor& like) {
    return at::empty(shape, at::TensorOptions().dtype(d).device(like.device()));
}

void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// Runs a C call on t's device and torch's current stream there.
template <typename F>
void launch(const Tensor& t, const char* name, F&& call) {
    qg_status st;
    {
        c10::DeviceGuard guard(t.device());
        void* stream = (void*)c10::hip::getCurrentHIPStream(t.get_device()).stream();
        pybind11::gil_scoped_release nogil;
        st = call(stream);
    }
    if (st == QG_OK) return;
    PyObject* r = PyObject_CallFunction(raise_status, "is", (int)st, name);
    Py_XDECREF(r);
    throw python_error();
}

void count(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) type_error("expected " + std::to_string(want) + " arguments");
}

PyObject* tuple(std::initializer_list<Tensor> ts) {
    Py_ssize_t n = 0;
    for (const Tensor& t : ts) n += t.defined();
    PyObject* r = PyTuple_New(n);
    if (r == nullptr) throw python_error();
    n = 0;
    for (const Tensor& t : ts)
        if (t.defined()) PyTuple_SET_ITEM(r, n++, THPVariable_Wrap(t));
    return r;
}

at::IntArrayRef lead(const Tensor& x) { return x.sizes().slice(0, x.dim() - 1); }

// The addresses of `n` entry points behind the function that raises for a status.
void bind_entries(PyObject* const* v, Py_ssize_t got, void** p, int n) {
    count(got, n + 1);
    for (int i = 0; i < n; ++i) {
        p[i] = PyLong_AsVoidPtr(v[i + 1]);
        if (p[i] == nullptr) {
            if (PyErr_Occurred()) throw python_error();
            value_error("an entry point is missing");
        }
    }
    Py_INCREF(v[0]);
    Py_XSETREF(raise_status, v[0]);
}

}  // namespace
