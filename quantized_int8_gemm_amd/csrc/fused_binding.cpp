// Python binding of the calls of qgemm_fused.h, made as the norm's and MX's is: a
// CPython extension module that checks dtypes (TypeError) and shapes (ValueError),
// allocates outputs and workspace and calls the C entry point on the tensors' device
// and torch's current stream there.
#include "binding_common.h"

#include "../../include/qgemm_fused.h"

namespace {

struct Entry {
    decltype(&qgemm_a8w8_linear_workspace_bytes) linear_workspace;
    decltype(&qgemm_a8w8_linear) linear;
    decltype(&qgemm_a8w8_gated_workspace_bytes) gated_workspace;
    decltype(&qgemm_a8w8_gated) gated;
    decltype(&qgemm_a8w8_linear_grad_workspace_bytes) linear_grad_workspace;
    decltype(&qgemm_a8w8_linear_grad) linear_grad;
    decltype(&qgemm_a8w8_gated_grad_workspace_bytes) gated_grad_workspace;
    decltype(&qgemm_a8w8_gated_grad) gated_grad;
    decltype(&int8_quantize) quantize;
    decltype(&int8_dequantize) dequantize;
} entry;

bool flag(PyObject* o) {
    const int r = PyObject_IsTrue(o);
    if (r < 0) throw python_error();
    return r != 0;
}

std::string repr(PyObject* o) {
    PyObject* r = PyObject_Repr(o);
    const char* text = r == nullptr ? nullptr : PyUnicode_AsUTF8(r);
    const std::string s = text == nullptr ? "?" : text;
    PyErr_Clear();
    Py_XDECREF(r);
    return s;
}

qg_activation activation(PyObject* o) {
    static const char* const names[] = {"none", "relu", "silu", "gelu", "gelu_tanh"};
    if (o == Py_None) return QG_ACT_NONE;
    if (PyUnicode_Check(o))
        for (int i = 0; i < 5; ++i)
            if (PyUnicode_CompareWithASCIIString(o, names[i]) == 0) return (qg_activation)i;
    value_error("unknown activation " + repr(o) + "; expected None or one of ['none', 'relu', 'silu', 'gelu', 'gelu_tanh']");
}

qg_dtype out_type(PyObject* o, at::ScalarType* d) {
    const char* what = "out_dtype must be torch.float32, torch.bfloat16 or torch.float16";
    *d = dtype_arg(o, what);
    const int k = float_kind(*d);
    if (k < 0) type_error(what);
    return (qg_dtype)k;
}

// A matrix of two dimensions; rows that do not exist lie anywhere.
Matrix matrix2(const Tensor& t, const char* name) {
    if (t.dim() != 2) value_error(std::string(name) + " must be 2-D");
    return matrix(t, name);
}

// A scale of `n` rows (shape [n], [n,1]) or columns ([n], [1,n]), or of one value, flat.
struct Scale { Tensor t; int64_t len; };

Scale scale_of(PyObject* o, const char* name, int64_t n, bool of_rows) {
    const Tensor& s = tensor(o, name);
    need_dtype(s, at::kFloat, name);
    const at::IntArrayRef z = s.sizes();
    const int64_t count = s.numel();
    const bool right = count == 1 || count == n;
    if (!(z.size() == 0 || (z.size() == 1 && right) || (z.size() == 2 && right && z[of_rows ? 1 : 0] == 1))) {
        const char* dim = of_rows ? "M" : "N";
        value_error(std::string(name) + " of shape " + str(z) + " is not [" + dim + "], " + (of_rows ? "[M,1]" : "[1,N]") +
                    " or scalar (" + dim + "=" + std::to_string(n) + ")");
    }
    if (s.is_contiguous()) return {s, count};
    return {s.contiguous(), count};
}

// A weight: [K,N], or [N,K] with b_trans.
struct Weight { Tensor t; int64_t n, k, ld; };

Weight weight_of(PyObject* o, const char* name, bool b_trans) {
    Weight w{};
    w.t = tensor(o, name);
    need_dtype(w.t, at::kChar, name);
    w.ld = matrix2(w.t, name).ld;
    w.n = w.t.size(b_trans ? 0 : 1);
    w.k = w.t.size(b_trans ? 1 : 0);
    return w;
}

Tensor workspace_of(size_t bytes, const Tensor& like) {
    return bytes == 0 ? Tensor() : make({(int64_t)bytes}, at::kByte, like);
}

// A checkpoint: codes of `shape` and their scales.
struct Checkpoint { Tensor codes, scale; int64_t ldc, lds; };

Checkpoint new_checkpoint(int64_t halves, int64_t m, int64_t n, const Tensor& like) {
    Checkpoint c{};
    c.ldc = n;
    c.lds = (n + 31) / 32;
    c.codes = halves == 1 ? make({m, n}, at::kChar, like) : make({halves, m, n}, at::kChar, like);
    c.scale = halves == 1 ? make({m, c.lds}, at::kFloat, like) : make({halves, m, c.lds}, at::kFloat, like);
    return c;
}

Checkpoint given_checkpoint(PyObject* o, int64_t halves, int64_t m, int64_t n) {
    Checkpoint c{};
    if (o == Py_None) return c;
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2) type_error("checkpoint must be the (codes, scale) of the forward call");
    c.codes = tensor(PyTuple_GET_ITEM(o, 0), "checkpoint codes");
    c.scale = tensor(PyTuple_GET_ITEM(o, 1), "checkpoint scale");
    c.ldc = n;
    c.lds = (n + 31) / 32;
    const std::vector<int64_t> one = {m, n}, two = {halves, m, n}, s1 = {m, c.lds}, s2 = {halves, m, c.lds};
    need_like(c.codes, "checkpoint codes", halves == 1 ? one : two, at::kChar);
    need_like(c.scale, "checkpoint scale", halves == 1 ? s1 : s2, at::kFloat);
    if (!c.codes.is_contiguous() || !c.scale.is_contiguous()) value_error("checkpoint must be contiguous");
    return c;
}

PyObject* with_checkpoint(const Tensor& out, const Checkpoint& c) {
    if (!c.codes.defined()) return THPVariable_Wrap(out);
    PyObject* pair = tuple({c.codes, c.scale});
    PyObject* r = PyTuple_New(2);
    if (r == nullptr) {
        Py_DECREF(pair);
        throw python_error();
    }
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(out));
    PyTuple_SET_ITEM(r, 1, pair);
    return r;
}

// A, W, act_scale, weight_scale, bias, activation, residual, out_dtype, b_trans, checkpoint, out
PyObject* py_linear(PyObject*, PyObject* const* v, Py_ssize_t argc) {
    HANDLE_TH_ERRORS
    count(argc, 11);
    const Tensor& A = tensor(v[0], "A");
    need_dtype(A, at::kChar, "A");
    const Matrix a = matrix2(A, "A");
    const int64_t m = A.size(0), k = a.n;
    const bool b_trans = flag(v[8]), save = flag(v[9]);
    const Weight w = weight_of(v[1], "W", b_trans);
    if (w.k != k) value_error("inner dimensions differ: A is " + str(A.sizes()) + ", W is " + str(w.t.sizes()));
    const Scale as = scale_of(v[2], "act_scale", m, true), ws = scale_of(v[3], "weight_scale", w.n, false);
    Tensor bias = tensor_or_none(v[4], "bias");
    if (bias.defined()) {
        need_like(bias, "bias", {w.n}, at::kFloat);
        bias = bias.contiguous();
    }
    const qg_activation act = activation(v[5]);
    at::ScalarType d;
    const qg_dtype kind = out_type(v[7], &d);
    const Tensor& res = tensor_or_none(v[6], "residual");
    Matrix rm{};
    if (res.defined()) {
        need_like(res, "residual", {m, w.n}, d);
        rm = matrix(res, "residual");
    }
    Tensor out = tensor_or_none(v[10], "out");
    if (out.defined()) need_like(out, "out", {m, w.n}, d);
    on_gpu(A, w.t, as.t, ws.t, bias, res, out);
    if (!out.defined()) out = make({m, w.n}, d, A);
    const Matrix om = matrix(out, "out");
    const Checkpoint c = save ? new_checkpoint(1, m, w.n, A) : Checkpoint{};
    const size_t need = entry.linear_workspace(m, w.n, k, (const int8_t*)ptr(A), a.ld, (const int8_t*)ptr(w.t), w.ld, b_trans, save);
    const Tensor work = workspace_of(need, A);
    launch(A, "qgemm_a8w8_linear", [&](void* s) {
        return entry.linear(m, w.n, k, (const int8_t*)ptr(A), a.ld, (const int8_t*)ptr(w.t), w.ld, b_trans, (const float*)ptr(as.t),
                            as.len, (const float*)ptr(ws.t), ws.len, (const float*)ptr(bias), act, ptr(res), rm.ld, ptr(out), kind,
                            om.ld, (int8_t*)ptr(c.codes), c.ldc, (float*)ptr(c.scale), c.lds, ptr(work), need, s);
    });
    return with_checkpoint(out, c);
    END_HANDLE_TH_ERRORS
}

// A, W_gate, W_up, act_scale, gate_scale, up_scale, activation, out_dtype, b_trans, checkpoint, out
PyObject* py_gated(PyObject*, PyObject* const* v, Py_ssize_t argc) {
    HANDLE_TH_ERRORS
    count(argc, 11);
    const Tensor& A = tensor(v[0], "A");
    need_dtype(A, at::kChar, "A");
    const Matrix a = matrix2(A, "A");
    const int64_t m = A.size(0), k = a.n;
    const bool b_trans = flag(v[8]), save = flag(v[9]);
    const Weight g = weight_of(v[1], "W_gate", b_trans), u = weight_of(v[2], "W_up", b_trans);
    if (u.t.sizes() != g.t.sizes()) value_error("W_gate is " + str(g.t.sizes()) + ", W_up is " + str(u.t.sizes()));
    if (g.k != k) value_error("inner dimensions differ: A is " + str(A.sizes()) + ", W_gate is " + str(g.t.sizes()));
    const Scale as = scale_of(v[3], "act_scale", m, true), gs = scale_of(v[4], "gate_scale", g.n, false),
                us = scale_of(v[5], "up_scale", g.n, false);
    const qg_activation act = activation(v[6]);
    at::ScalarType d;
    const qg_dtype kind = out_type(v[7], &d);
    Tensor out = tensor_or_none(v[10], "out");
    if (out.defined()) need_like(out, "out", {m, g.n}, d);
    on_gpu(A, g.t, u.t, as.t, gs.t, us.t, out);
    if (!out.defined()) out = make({m, g.n}, d, A);
    const Matrix om = matrix(out, "out");
    const Checkpoint c = save ? new_checkpoint(2, m, g.n, A) : Checkpoint{};
    const size_t need = entry.gated_workspace(m, g.n, k, (const int8_t*)ptr(A), a.ld, (const int8_t*)ptr(g.t), g.ld,
                                              (const int8_t*)ptr(u.t), u.ld, b_trans, save);
    const Tensor work = workspace_of(need, A);
    launch(A, "qgemm_a8w8_gated", [&](void* s) {
        return entry.gated(m, g.n, k, (const int8_t*)ptr(A), a.ld, (const int8_t*)ptr(g.t), g.ld, (const int8_t*)ptr(u.t), u.ld,
                           b_trans, (const float*)ptr(as.t), as.len, (const float*)ptr(gs.t), gs.len, (const float*)ptr(us.t), us.len,
                           act, ptr(out), kind, om.ld, (int8_t*)ptr(c.codes), c.ldc, (float*)ptr(c.scale), c.lds, ptr(work), need, s);
    });
    return with_checkpoint(out, c);
    END_HANDLE_TH_ERRORS
}

struct Upstream { Tensor t; qg_dtype kind; Matrix m; };

Upstream upstream(PyObject* o) {
    Upstream y{};
    y.t = tensor(o, "dy");
    if (y.t.scalar_type() != at::kBFloat16 && y.t.scalar_type() != at::kHalf) wrong_dtype(y.t, "dy", "bfloat16 or float16");
    y.kind = need_float(y.t, "dy");
    y.m = matrix2(y.t, "dy");
    return y;
}

// dy, W, weight_scale, checkpoint, activation, b_trans, bias_grad
PyObject* py_linear_grad(PyObject*, PyObject* const* v, Py_ssize_t argc) {
    HANDLE_TH_ERRORS
    count(argc, 7);
    const Upstream dy = upstream(v[0]);
    const bool b_trans = flag(v[5]), with_bias = flag(v[6]);
    const Weight w = weight_of(v[1], "W", b_trans);
    const int64_t m = dy.t.size(0), n = w.n, k = w.k;
    if (dy.t.size(1) != n) value_error("dy is " + str(dy.t.sizes()) + " but W is " + str(w.t.sizes()) + "; both need N columns");
    const Scale ws = scale_of(v[2], "weight_scale", n, false);
    const qg_activation act = activation(v[4]);
    const Checkpoint c = given_checkpoint(v[3], 1, m, n);
    if (!c.codes.defined() && act != QG_ACT_NONE) value_error("an activation's gradient needs the forward call's checkpoint");
    on_gpu(dy.t, w.t, ws.t, c.codes, c.scale);
    const Tensor dx = make({m, k}, dy.t.scalar_type(), dy.t);
    const Tensor db = with_bias ? make({n}, at::kFloat, dy.t) : Tensor();
    const size_t need = entry.linear_grad_workspace(m, n, k, (const int8_t*)ptr(w.t), w.ld, b_trans, with_bias);
    const Tensor work = workspace_of(need, dy.t);
    launch(dy.t, "qgemm_a8w8_linear_grad", [&](void* s) {
        return entry.linear_grad(m, n, k, ptr(dy.t), dy.kind, dy.m.ld, (const int8_t*)ptr(w.t), w.ld, b_trans, (const float*)ptr(ws.t),
                                 ws.len, (const int8_t*)ptr(c.codes), c.ldc, (const float*)ptr(c.scale), c.lds, act, ptr(dx), k,
                                 (float*)ptr(db), ptr(work), need, s);
    });
    return with_bias ? tuple({dx, db}) : THPVariable_Wrap(dx);
    END_HANDLE_TH_ERRORS
}

// dy, W_gate, W_up, gate_scale, up_scale, checkpoint, activation, b_trans
PyObject* py_gated_grad(PyObject*, PyObject* const* v, Py_ssize_t argc) {
    HANDLE_TH_ERRORS
    count(argc, 8);
    const Upstream dy = upstream(v[0]);
    const bool b_trans = flag(v[7]);
    const Weight g = weight_of(v[1], "W_gate", b_trans), u = weight_of(v[2], "W_up", b_trans);
    if (u.t.sizes() != g.t.sizes()) value_error("W_gate is " + str(g.t.sizes()) + ", W_up is " + str(u.t.sizes()));
    const int64_t m = dy.t.size(0), n = g.n, k = g.k;
    if (dy.t.size(1) != n) value_error("dy is " + str(dy.t.sizes()) + " but W_gate is " + str(g.t.sizes()) + "; both need N columns");
    const Scale gs = scale_of(v[3], "gate_scale", n, false), us = scale_of(v[4], "up_scale", n, false);
    const Checkpoint c = given_checkpoint(v[5], 2, m, n);
    if (!c.codes.defined()) type_error("checkpoint must be the (codes, scale) of the forward call");
    const qg_activation act = activation(v[6]);
    on_gpu(dy.t, g.t, u.t, gs.t, us.t, c.codes, c.scale);
    const Tensor dx = make({m, k}, dy.t.scalar_type(), dy.t);
    const size_t need = entry.gated_grad_workspace(m, n, k, (const int8_t*)ptr(g.t), g.ld, (const int8_t*)ptr(u.t), u.ld, b_trans);
    const Tensor work = workspace_of(need, dy.t);
    launch(dy.t, "qgemm_a8w8_gated_grad", [&](void* s) {
        return entry.gated_grad(m, n, k, ptr(dy.t), dy.kind, dy.m.ld, (const int8_t*)ptr(g.t), g.ld, (const int8_t*)ptr(u.t), u.ld,
                                b_trans, (const float*)ptr(gs.t), gs.len, (const float*)ptr(us.t), us.len, (const int8_t*)ptr(c.codes),
                                c.ldc, (const float*)ptr(c.scale), c.lds, act, ptr(dx), k, ptr(work), need, s);
    });
    return THPVariable_Wrap(dx);
    END_HANDLE_TH_ERRORS
}

int block_arg(PyObject* o) {
    if (o == Py_None) return 0;
    const long b = PyLong_Check(o) ? PyLong_AsLong(o) : -1;
    if (b != 32) {
        PyErr_Clear();
        value_error("block must be None or 32, not " + repr(o));
    }
    return 32;
}

// x, block
PyObject* py_int8_quantize(PyObject*, PyObject* const* v, Py_ssize_t argc) {
    HANDLE_TH_ERRORS
    count(argc, 2);
    const Tensor& x = tensor(v[0], "x");
    const qg_dtype kind = need_float(x, "x");
    const Matrix m = matrix(x, "x");
    if (m.n == 0) value_error("x must have at least one column");
    const int block = block_arg(v[1]);
    on_gpu(x);
    const Tensor codes = make(x.sizes(), at::kChar, x);
    c10::SmallVector<int64_t, 5> shape(x.sizes().begin(), x.sizes().end());
    shape.pop_back();
    const int64_t lds = block == 0 ? 1 : (m.n + 31) / 32;
    if (block != 0) shape.push_back(lds);
    const Tensor scale = make(shape, at::kFloat, x);
    launch(x, "int8_quantize", [&](void* s) {
        return entry.quantize(m.rows, m.n, ptr(x), kind, m.ld, block, (int8_t*)ptr(codes), m.n, (float*)ptr(scale), lds, s);
    });
    return tuple({codes, scale});
    END_HANDLE_TH_ERRORS
}

// codes, scale, out_dtype, out
PyObject* py_int8_dequantize(PyObject*, PyObject* const* v, Py_ssize_t argc) {
    HANDLE_TH_ERRORS
    count(argc, 4);
    const Tensor &codes = tensor(v[0], "codes"), &given = tensor(v[1], "scale");
    need_dtype(codes, at::kChar, "codes");
    need_dtype(given, at::kFloat, "scale");
    const Matrix m = matrix(codes, "codes");
    if (m.n == 0) value_error("codes must have at least one column");
    at::ScalarType d;
    const qg_dtype kind = out_type(v[2], &d);
    const int64_t blocks = (m.n + 31) / 32;
    const bool by_row = given.sizes() == lead(codes);
    if (!by_row && !(given.dim() == codes.dim() && lead(given) == lead(codes) && given.size(-1) == blocks))
        value_error("scale has shape " + str(given.sizes()) + "; expected one a row or " + std::to_string(blocks) +
                    " a row for codes of shape " + str(codes.sizes()));
    Tensor out = tensor_or_none(v[3], "out");
    if (out.defined()) need_like(out, "out", codes.sizes(), d);
    on_gpu(codes, given, out);
    const Tensor scale = given.contiguous();
    if (!out.defined()) out = make(codes.sizes(), d, codes);
    const Matrix om = matrix(out, "out");
    launch(codes, "int8_dequantize", [&](void* s) {
        return entry.dequantize(m.rows, m.n, (const int8_t*)ptr(codes), m.ld, (const float*)ptr(scale), by_row ? 1 : blocks,
                                by_row ? 0 : 32, ptr(out), kind, om.ld, s);
    });
    return THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// The function that raises for a status, then the entry points' addresses in the
// order of Entry.
PyObject* py_bind(PyObject*, PyObject* const* v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    void* p[10];
    bind_entries(v, n, p, 10);
    entry.linear_workspace = reinterpret_cast<decltype(entry.linear_workspace)>(p[0]);
    entry.linear = reinterpret_cast<decltype(entry.linear)>(p[1]);
    entry.gated_workspace = reinterpret_cast<decltype(entry.gated_workspace)>(p[2]);
    entry.gated = reinterpret_cast<decltype(entry.gated)>(p[3]);
    entry.linear_grad_workspace = reinterpret_cast<decltype(entry.linear_grad_workspace)>(p[4]);
    entry.linear_grad = reinterpret_cast<decltype(entry.linear_grad)>(p[5]);
    entry.gated_grad_workspace = reinterpret_cast<decltype(entry.gated_grad_workspace)>(p[6]);
    entry.gated_grad = reinterpret_cast<decltype(entry.gated_grad)>(p[7]);
    entry.quantize = reinterpret_cast<decltype(entry.quantize)>(p[8]);
    entry.dequantize = reinterpret_cast<decltype(entry.dequantize)>(p[9]);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

#define QG_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {QG_METHOD(bind), QG_METHOD(linear), QG_METHOD(gated), QG_METHOD(linear_grad), QG_METHOD(gated_grad),
                         QG_METHOD(int8_quantize), QG_METHOD(int8_dequantize), {nullptr, nullptr, 0, nullptr}};
#undef QG_METHOD

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fused_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fused_binding(void) { return PyModule_Create(&module); }
