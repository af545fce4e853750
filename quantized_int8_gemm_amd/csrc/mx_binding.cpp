// Python binding of the calls of qgemm_mx.h: a CPython extension module over
// torch's C++ tensors.  It checks dtypes (TypeError) and shapes (ValueError),
// allocates the outputs and calls the C entry point on the tensors' device and
// torch's current stream there; it computes nothing.  The smallest of these calls
// take 3 us on the GPU, and the same marshalling through ctypes took 6 to 9 us of a
// call, so it is done here: norm to int8 of one row 14.2 -> 5.1 us a call, gradient
// of 1000 x 1000 15.1 -> 9.7, MXFP8 quantiser 16 x 8192 9.0 -> 4.8 (the launch itself
// takes about 2.8).
#include "binding_common.h"

#include "../../include/qgemm_mx.h"

namespace {

// The library's entry points, as the package hands them over.
struct Entry {
    decltype(&rms_norm) norm;
    decltype(&rms_norm_grad_workspace_bytes) grad_workspace;
    decltype(&rms_norm_grad) grad;
    decltype(&mx_quantize) quantize;
    decltype(&mx_dequantize) dequantize;
    decltype(&mx_matmul) matmul;
} entry;

// ---------------------------------------------------------------------------
// The norm
// ---------------------------------------------------------------------------

struct Norm {
    Tensor x, weight, residual, h;
    qg_dtype kind;
    Matrix m, r, hm;
    float eps;
};

Norm norm_inputs(PyObject* x, PyObject* weight, PyObject* eps, PyObject* residual, PyObject* residual_out) {
    Norm a{};
    a.x = tensor(x, "x");
    a.kind = need_float(a.x, "x");
    a.m = matrix(a.x, "x");
    if (a.m.n == 0) value_error("x must have at least one column");
    a.weight = weight_of(tensor(weight, "weight"), a.m.n, a.x.scalar_type());
    const double e = PyFloat_AsDouble(eps);
    if (e == -1.0 && PyErr_Occurred()) throw python_error();
    a.eps = (float)e;
    a.residual = tensor_or_none(residual, "residual");
    if (a.residual.defined()) {
        need_dtype(a.residual, a.x.scalar_type(), "residual");
        if (a.residual.sizes() != a.x.sizes())
            value_error("residual has shape " + str(a.residual.sizes()) + "; x has " + str(a.x.sizes()));
        a.r = matrix(a.residual, "residual");
        a.h = tensor_or_none(residual_out, "residual_out");
        if (a.h.defined()) need_like(a.h, "residual_out", a.x.sizes(), a.x.scalar_type());
    } else if (residual_out != Py_None) {
        value_error("residual_out needs a residual");
    }
    return a;
}

// The last check of the inputs, and h.
void norm_begin(Norm& a, const Tensor& out) {
    on_gpu(a.x, a.weight, a.residual, a.h, out);
    if (a.residual.defined()) {
        if (!a.h.defined()) a.h = make(a.x.sizes(), a.x.scalar_type(), a.x);
        a.hm = matrix(a.h, "residual_out");
    }
}

void norm_call(const Norm& a, const Tensor& out, qg_dtype format, int64_t ldo, const Tensor& block_scale, int64_t lds,
               const Tensor& row_scale) {
    launch(a.x, "rms_norm", [&](void* s) {
        return entry.norm(a.m.rows, a.m.n, ptr(a.x), a.kind, a.m.ld, ptr(a.residual), a.r.ld, ptr(a.weight),
                          (qg_dtype)float_kind(a.weight.scalar_type()), a.eps, ptr(a.h), a.hm.ld, ptr(out), format, ldo,
                          (uint8_t*)ptr(block_scale), lds, (float*)ptr(row_scale), s);
    });
}

// x, weight, eps, residual, out_dtype, out, residual_out
PyObject* py_rms_norm(PyObject*, PyObject* const* v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 7);
    Norm a = norm_inputs(v[0], v[1], v[2], v[3], v[6]);
    at::ScalarType d = a.x.scalar_type();
    if (v[4] != Py_None) {
        const at::ScalarType want = dtype_arg(v[4], "out_dtype must be a torch.dtype");
        if (want != d && want != at::kFloat) type_error("out_dtype must be x's dtype or torch.float32");
        d = want;
    }
    Tensor y = tensor_or_none(v[5], "out");
    if (y.defined()) need_like(y, "out", a.x.sizes(), d);
    norm_begin(a, y);
    if (!y.defined()) y = make(a.x.sizes(), d, a.x);
    const Tensor rstd = make(lead(a.x), at::kFloat, a.x);
    norm_call(a, y, (qg_dtype)float_kind(d), matrix(y, "out").ld, Tensor(), 0, rstd);
    return tuple({y, rstd, a.h});
    END_HANDLE_TH_ERRORS
}

// Format names; 0 for any other.
int mx_format(PyObject* o) {
    if (!PyUnicode_Check(o)) return 0;
    return PyUnicode_CompareWithASCIIString(o, "mxfp8") == 0   ? QG_MXFP8
           : PyUnicode_CompareWithASCIIString(o, "mxfp4") == 0 ? QG_MXFP4
                                                               : 0;
}

// Codes and scale bytes of rows of n; scale rows start at multiples of 16 bytes.
struct Coded { Tensor codes, scale; int64_t ldc, lds; };

Coded coded(at::IntArrayRef lead, int64_t n, int format, const Tensor& like) {
    Coded c;
    const int64_t blocks = (n + 31) / 32;
    c.ldc = blocks * (format == QG_MXFP8 ? 32 : 16);
    c.lds = (blocks + 15) / 16 * 16;
    c10::SmallVector<int64_t, 5> shape(lead.begin(), lead.end());
    shape.push_back(c.ldc);
    c.codes = make(shape, format == QG_MXFP8 ? at::kFloat8_e4m3fn : at::kByte, like);
    shape.back() = c.lds;
    c.scale = make(shape, at::kByte, like);
    if (c.lds != blocks) c.scale = c.scale.narrow(-1, 0, blocks);
    return c;
}

[[noreturn]] void unknown_format(PyObject* o, const char* expected) {
    PyObject* r = PyObject_Repr(o);
    const char* text = r == nullptr ? nullptr : PyUnicode_AsUTF8(r);
    const std::string s = text == nullptr ? "?" : text;
    PyErr_Clear();
    Py_XDECREF(r);
    value_error("unknown format " + s + "; expected one of " + expected);
}

// x, weight, eps, residual, format, residual_out
PyObject* py_rms_norm_quantize(PyObject*, PyObject* const* v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 6);
    const bool int8 = PyUnicode_Check(v[4]) && PyUnicode_CompareWithASCIIString(v[4], "int8") == 0;
    const int format = int8 ? QG_INT8 : mx_format(v[4]);
    if (format == 0) unknown_format(v[4], "['int8', 'mxfp4', 'mxfp8']");
    Norm a = norm_inputs(v[0], v[1], v[2], v[3], v[5]);
    norm_begin(a, Tensor());
    const Tensor row_scale = make(lead(a.x), at::kFloat, a.x);
    if (int8) {
        const Tensor q = make(a.x.sizes(), at::kChar, a.x);
        norm_call(a, q, QG_INT8, a.m.n, Tensor(), 0, row_scale);
        return tuple({q, row_scale, a.h});
    }
    const Coded c = coded(lead(a.x), a.m.n, format, a.x);
    norm_call(a, c.codes, (qg_dtype)format, c.ldc, c.scale, c.lds, row_scale);
    return tuple({c.codes, c.scale, row_scale, a.h});
    END_HANDLE_TH_ERRORS
}

// dy, h, weight, rstd, dh
PyObject* py_rms_norm_grad(PyObject*, PyObject* const* v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 5);
    const Tensor &h = tensor(v[1], "h"), &dy = tensor(v[0], "dy"), &dh = tensor_or_none(v[4], "dh");
    const at::ScalarType d = h.scalar_type();
    const qg_dtype kind = need_float(h, "h");
    need_dtype(dy, d, "dy");
    const Matrix hm = matrix(h, "h");
    if (hm.n == 0) value_error("h must have at least one column");
    if (dy.sizes() != h.sizes()) value_error("dy has shape " + str(dy.sizes()) + "; h has " + str(h.sizes()));
    const Matrix ym = matrix(dy, "dy");
    const Tensor weight = weight_of(tensor(v[2], "weight"), hm.n, d);
    const Tensor& r = tensor(v[3], "rstd");
    need_like(r, "rstd", lead(h), at::kFloat);
    Matrix sm{};
    if (dh.defined()) {
        need_like(dh, "dh", h.sizes(), d);
        sm = matrix(dh, "dh");
    }
    on_gpu(h, dy, weight, r, dh);
    const Tensor rstd = r.contiguous();
    const Tensor dx = make(h.sizes(), d, h), dweight = make({hm.n}, weight.scalar_type(), h);
    const size_t need = entry.grad_workspace(hm.rows, hm.n);
    const Tensor ws = need == 0 ? Tensor() : make({(int64_t)need}, at::kByte, h);
    launch(h, "rms_norm_grad", [&](void* s) {
        return entry.grad(hm.rows, hm.n, ptr(dy), kind, ym.ld, ptr(h), hm.ld, ptr(weight),
                          (qg_dtype)float_kind(weight.scalar_type()), (const float*)ptr(rstd), ptr(dh), sm.ld, ptr(dx), hm.n,
                          ptr(dweight), ptr(ws), need, s);
    });
    return tuple({dx, dweight});
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------------------
// MX
// ---------------------------------------------------------------------------

// x, format
PyObject* py_mx_quantize(PyObject*, PyObject* const* v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 2);
    const Tensor& x = tensor(v[0], "x");
    const qg_dtype kind = need_float(x, "x");
    const Matrix m = matrix(x, "x");
    if (m.n == 0) value_error("x must have at least one column");
    const int format = mx_format(v[1]);
    if (format == 0) unknown_format(v[1], "['mxfp4', 'mxfp8']");
    on_gpu(x);
    const Coded c = coded(lead(x), m.n, format, x);
    launch(x, "mx_quantize", [&](void* s) {
        return entry.quantize(m.rows, m.n, ptr(x), kind, m.ld, ptr(c.codes), (qg_dtype)format, c.ldc, (uint8_t*)ptr(c.scale),
                              c.lds, s);
    });
    return tuple({c.codes, c.scale});
    END_HANDLE_TH_ERRORS
}

// One MX operand: format, rows, K, strides in bytes.
struct Operand { qg_dtype format; int64_t rows, k, ldc, lds; };

Operand operand(const Tensor& codes, const Tensor& scale, const char* name) {
    Operand o{};
    if (codes.scalar_type() == at::kFloat8_e4m3fn) o.format = QG_MXFP8;
    else if (codes.scalar_type() == at::kByte) o.format = QG_MXFP4;
    else wrong_dtype(codes, name, "float8_e4m3fn or uint8");
    const std::string scale_name = std::string(name) + " scale";
    need_dtype(scale, at::kByte, scale_name.c_str());
    const Matrix c = matrix(codes, name), s = matrix(scale, scale_name.c_str());
    const int64_t per = o.format == QG_MXFP8 ? 32 : 16;
    if (c.n == 0 || c.n % per != 0)
        value_error(std::string(name) + " has " + std::to_string(c.n) + " code columns; expected whole blocks of " +
                    std::to_string(per));
    if (s.n * per != c.n || lead(codes) != lead(scale))
        value_error("the scale of " + std::string(name) + " has shape " + str(scale.sizes()) + "; expected " +
                    std::to_string(c.n / per) + " columns for codes of shape " + str(codes.sizes()));
    o.rows = c.rows;
    o.k = s.n * 32;
    o.ldc = c.ld;
    o.lds = s.ld;
    return o;
}

// codes, scale, out_dtype, columns, out
PyObject* py_mx_dequantize(PyObject*, PyObject* const* v, Py_ssize_t argc) {
    HANDLE_TH_ERRORS
    count(argc, 5);
    const Tensor &codes = tensor(v[0], "codes"), &scale = tensor(v[1], "codes scale");
    const Operand o = operand(codes, scale, "codes");
    const char* what = "out_dtype must be torch.float32, torch.bfloat16 or torch.float16";
    const at::ScalarType d = dtype_arg(v[2], what);
    if (float_kind(d) < 0) type_error(what);
    int64_t n = o.k;
    if (v[3] != Py_None) {
        n = PyLong_AsLongLong(v[3]);
        if (n == -1 && PyErr_Occurred()) throw python_error();
    }
    if (n <= o.k - 32 || n > o.k)
        value_error("columns = " + std::to_string(n) + " does not fill " + std::to_string(o.k / 32) + " blocks");
    Tensor out = tensor_or_none(v[4], "out");
    on_gpu(codes, scale, out);
    c10::SmallVector<int64_t, 5> shape(codes.sizes().begin(), codes.sizes().end());
    shape.back() = n;
    if (out.defined()) need_like(out, "out", shape, d);
    else out = make(shape, d, codes);
    const Matrix om = matrix(out, "out");
    launch(codes, "mx_dequantize", [&](void* s) {
        return entry.dequantize(o.rows, n, ptr(codes), o.format, o.ldc, (const uint8_t*)ptr(scale), o.lds, ptr(out),
                                (qg_dtype)float_kind(d), om.ld, s);
    });
    return THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// Whether every scale row can be read to the end of its last 4-byte word.
bool rows_readable(const Tensor& scale, const Operand& o) {
    const int64_t blocks = o.k / 32;
    if (blocks % 4 == 0) return true;
    const int64_t last = scale.storage_offset() + (o.rows - 1) * o.lds;
    return (int64_t)scale.storage().nbytes() - last >= (blocks + 3) / 4 * 4;
}

// A, a_scale, W, w_scale, act_scale, out_dtype, out
PyObject* py_mx_matmul(PyObject*, PyObject* const* v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 7);
    const Tensor &A = tensor(v[0], "A"), &as = tensor(v[1], "A scale"), &W = tensor(v[2], "W"), &ws = tensor(v[3], "W scale");
    if (A.dim() != 2) value_error("A must be 2-D");
    if (W.dim() != 2) value_error("W must be 2-D");
    need_dtype(W, at::kByte, "W");
    const char* what = "out_dtype must be torch.float32, torch.bfloat16 or torch.float16";
    const at::ScalarType d = dtype_arg(v[5], what);
    if (float_kind(d) < 0) type_error(what);
    const Operand a = operand(A, as, "A"), w = operand(W, ws, "W");
    if (a.k != w.k)
        value_error("inner dimensions differ: A has " + std::to_string(a.k) + " columns, W has " + std::to_string(w.k));
    Tensor act = tensor_or_none(v[4], "act_scale");
    if (act.defined()) {
        need_dtype(act, at::kFloat, "act_scale");
        const at::IntArrayRef z = act.sizes();
        const bool one = act.numel() == 1 && act.dim() <= 2;
        if (!one && !((act.dim() == 1 || (act.dim() == 2 && z[1] == 1)) && z[0] == a.rows))
            value_error("act_scale of shape " + str(z) + " is not [M], [M,1] or scalar (M=" + std::to_string(a.rows) + ")");
        act = (one && a.rows != 1 ? act.reshape({1}).expand({a.rows}) : act).contiguous();
    }
    Tensor out = tensor_or_none(v[6], "out");
    on_gpu(A, as, W, ws, act, out);
    if (out.defined()) need_like(out, "out", {a.rows, w.rows}, d);
    else out = make({a.rows, w.rows}, d, A);
    if (out.numel() != 0) {
        const Matrix om = matrix(out, "out");
        const int padded = rows_readable(as, a) && rows_readable(ws, w);
        launch(A, "mx_matmul", [&](void* s) {
            return entry.matmul(a.rows, w.rows, a.k, ptr(A), a.format, a.ldc, (const uint8_t*)ptr(as), a.lds, ptr(W), w.ldc,
                                (const uint8_t*)ptr(ws), w.lds, padded, (const float*)ptr(act), ptr(out),
                                (qg_dtype)float_kind(d), om.ld, s);
        });
    }
    return THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// The function that raises for a status, then the entry points' addresses in the
// order of Entry.
PyObject* py_bind(PyObject*, PyObject* const* v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    void* p[6];
    bind_entries(v, n, p, 6);
    entry.norm = reinterpret_cast<decltype(entry.norm)>(p[0]);
    entry.grad_workspace = reinterpret_cast<decltype(entry.grad_workspace)>(p[1]);
    entry.grad = reinterpret_cast<decltype(entry.grad)>(p[2]);
    entry.quantize = reinterpret_cast<decltype(entry.quantize)>(p[3]);
    entry.dequantize = reinterpret_cast<decltype(entry.dequantize)>(p[4]);
    entry.matmul = reinterpret_cast<decltype(entry.matmul)>(p[5]);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

#define QG_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    QG_METHOD(bind), QG_METHOD(rms_norm), QG_METHOD(rms_norm_quantize), QG_METHOD(rms_norm_grad), QG_METHOD(mx_quantize),
    QG_METHOD(mx_dequantize), QG_METHOD(mx_matmul), {nullptr, nullptr, 0, nullptr}};
#undef QG_METHOD

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mx_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mx_binding(void) { return PyModule_Create(&module); }
