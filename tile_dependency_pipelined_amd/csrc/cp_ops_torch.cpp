// cp_ops_torch.cpp -- Python module _cp_ops_torch: the operators of cp_ops.h on
// torch tensors.  Checks of arguments, outputs and scratch memory from PyTorch's
// allocator on the current stream, one call into libcpchain.so.  A call costs
// little more than its kernel launches: 4.7 us for a linear layer and 10.4 for
// its gradients, where the same steps in Python took 9.1 and 18.6.  ops.py
// documents the functions.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <string>

#include "cp_ops.h"

namespace {

using at::Tensor;

PyObject *g_error = nullptr;  // called with (status, function, detail) for a failed library call; it raises

struct Refused {
    PyObject *type;
    std::string what;
};

[[noreturn]] void refuse(PyObject *type, const char *fmt, ...) {
    char text[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    throw Refused{type, text};
}

struct Raised {};  // a Python exception is set already

void check(int64_t rc, const char *where) {
    if (rc >= 0) return;
    PyObject *r = PyObject_CallFunction(g_error, "Lss", (long long)rc, where, cp_ops_last_error());
    Py_XDECREF(r);
    throw Raised{};
}

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
    return THPVariable_Unpack(o);
}

// The tensor that sets the call's device and element type.
const Tensor &first(PyObject *o, const char *name) {
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
        refuse(PyExc_TypeError, "%s must be a device tensor", name);
    const Tensor &t = THPVariable_Unpack(o);
    if (t.scalar_type() != at::kFloat && t.scalar_type() != at::kBFloat16)
        refuse(PyExc_ValueError, "%s must be float32 or bfloat16, got %s", name, c10::toString(t.scalar_type()));
    if (t.dim() != 2) refuse(PyExc_ValueError, "%s must have 2 dimensions, got %d", name, (int)t.dim());
    return t;
}

// A tensor of x's device with this type and shape.
const Tensor &like(PyObject *o, const Tensor &x, at::IntArrayRef shape, const char *name, at::ScalarType type) {
    const Tensor &t = tensor(o, name);
    if (t.device() != x.device())
        refuse(PyExc_ValueError, "%s is on %s, expected %s", name, t.device().str().c_str(), x.device().str().c_str());
    if (t.scalar_type() != type || t.sizes() != shape)
        refuse(PyExc_ValueError, "%s must be a %s tensor of shape %s, got %s %s", name, c10::toString(type),
               shape_text(shape).c_str(), c10::toString(t.scalar_type()), shape_text(t.sizes()).c_str());
    return t;
}
const Tensor &like(PyObject *o, const Tensor &x, at::IntArrayRef shape, const char *name) {
    return like(o, x, shape, name, x.scalar_type());
}

// Row stride of a matrix with unit stride within its rows.
int64_t rows(const Tensor &t, const char *name) {
    const int64_t s0 = t.stride(0), s1 = t.stride(1), M = t.size(0), N = t.size(1);
    if (s1 != 1 && N > 1 && M > 0)
        refuse(PyExc_ValueError, "%s must have unit stride within a row (strides %s); call .contiguous()", name,
               shape_text(t.strides()).c_str());
    if (s0 < N && M > 1)
        refuse(PyExc_ValueError, "the rows of %s overlap (strides %s); call .contiguous()", name,
               shape_text(t.strides()).c_str());
    return s0;
}

// Row stride of a weight [K][N] (or each of [E][K][N]) and whether it is stored [N][K].
int64_t weight(const Tensor &w, bool *stored_transposed) {
    const int64_t d = w.dim(), s0 = w.stride(d - 2), s1 = w.stride(d - 1), K = w.size(d - 2), N = w.size(d - 1);
    *stored_transposed = false;
    if (s1 == 1 && (s0 >= N || K <= 1) && N > 1) return s0;
    if ((s0 == 1 || K <= 1) && (s1 >= K || N <= 1)) {
        *stored_transposed = true;
        return s1;
    }
    if ((s1 == 1 || N <= 1) && (s0 >= N || K <= 1)) return s0;
    refuse(PyExc_ValueError,
           "w must be rows of unit stride that do not overlap, or the transpose of such (strides %s); call .contiguous()",
           shape_text(w.strides()).c_str());
}

const void *vector(PyObject *o, const Tensor &x, at::IntArrayRef shape, const char *name, at::ScalarType type) {
    const Tensor &t = like(o, x, shape, name, type);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
    return t.data_ptr();
}
const void *optional_vector(PyObject *o, const Tensor &x, at::IntArrayRef shape, const char *name) {
    return o == Py_None ? nullptr : vector(o, x, shape, name, x.scalar_type());
}

int code(const Tensor &x) { return x.scalar_type() == at::kBFloat16 ? CP_BF16 : CP_F32; }

void *data(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

Tensor empty(const Tensor &x, at::IntArrayRef shape) { return at::empty(shape, x.options()); }

Tensor empty_weight(const Tensor &w, bool stored_transposed) {
    if (!stored_transposed) return at::empty(w.sizes(), w.options());
    auto s = w.sizes().vec();
    std::swap(s[s.size() - 2], s[s.size() - 1]);
    return at::empty(s, w.options()).transpose(-1, -2);
}

// The tensor to write: `out`, or a new one.
Tensor output(PyObject *o, const Tensor &x, at::IntArrayRef shape) {
    if (o == Py_None) return empty(x, shape);
    const Tensor &t = like(o, x, shape, "out");
    if (c10::GradMode::is_enabled() && t.requires_grad())
        refuse(PyExc_RuntimeError, "out requires a gradient, which is not recorded here; pass out.detach() or call under torch.no_grad()");
    return t;
}
// Autograd takes what it saved as unchanged while its version is (tensors made
// in inference mode have none, and are never saved).
void written(const Tensor &out) {
    if (!out.is_inference()) out.unsafeGetTensorImpl()->bump_version();
}

bool aligned(const Tensor &x, std::initializer_list<const Tensor *> mats, std::initializer_list<int64_t> elements) {
    uint64_t bits = 0;
    for (const Tensor *t : mats) bits |= (uint64_t)t->data_ptr();
    for (int64_t e : elements) bits |= (uint64_t)(e * (int64_t)x.element_size());
    return bits % 16 == 0;
}

struct Scratch {
    Tensor t;
    int64_t n;
    Scratch(const Tensor &x, int op, int64_t M, int64_t K, int64_t N, int64_t E, bool al) {
        n = cp_ops_workspace(op, code(x), M, K, N, (int32_t)E, al);
        check(n, "cp_ops_workspace");
        if (n) t = at::empty({n}, x.options().dtype(at::kByte));
    }
};

void *stream(const Tensor &x) { return (void *)c10::hip::getCurrentHIPStream(x.get_device()).stream(); }

int activation(PyObject *o) {
    const long a = PyLong_AsLong(o);
    if (a == -1 && PyErr_Occurred()) throw Raised{};
    if (a != (int)a) refuse(PyExc_ValueError, "activation %ld is not supported", a);
    return (int)a;
}
bool truth(PyObject *o) {
    const int r = PyObject_IsTrue(o);
    if (r < 0) throw Raised{};
    return r != 0;
}

PyObject *wrap(const Tensor &t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
template <class... Ts>
PyObject *wrap_tuple(const Ts &...t) {
    PyObject *items[] = {wrap(t)...};
    PyObject *r = PyTuple_New(sizeof...(t));
    bool ok = r != nullptr;
    for (PyObject *o : items) ok = ok && o;
    if (!ok) {
        for (PyObject *o : items) Py_XDECREF(o);
        Py_XDECREF(r);
        throw Raised{};
    }
    for (size_t i = 0; i < sizeof...(t); ++i) PyTuple_SET_ITEM(r, i, items[i]);
    return r;
}

const Tensor &experts(PyObject *w, PyObject *off, const Tensor &x, const Tensor **offsets) {
    const Tensor &t = tensor(w, "w");
    if (t.dim() != 3) refuse(PyExc_ValueError, "w must have 3 dimensions [E][K][N]");
    const int64_t E = t.size(0);
    if (!THPVariable_Check(off)) refuse(PyExc_ValueError, "offsets must be a tensor");
    const Tensor &o = THPVariable_Unpack(off);
    if (o.scalar_type() != at::kInt || o.dim() != 1 || o.size(0) != E + 1 || !o.is_contiguous() || o.device() != x.device())
        refuse(PyExc_ValueError, "offsets must be a contiguous int32 tensor of %lld elements on %s", (long long)(E + 1),
               x.device().str().c_str());
    *offsets = &o;
    return t;
}

// linear(x, w, bias, residual, act, need_pre, out)
PyObject *linear(PyObject *const *a) {
    const Tensor &x = first(a[0], "x");
    const int64_t M = x.size(0), K = x.size(1);
    const Tensor &w = tensor(a[1], "w");
    if (w.dim() != 2) refuse(PyExc_ValueError, "w must be a matrix");
    const int64_t N = w.size(1);
    like(a[1], x, {K, N}, "w");
    bool wt;
    const int64_t ldw = weight(w, &wt), ldx = rows(x, "x");
    const void *bias = optional_vector(a[2], x, {N}, "bias");
    const Tensor *r = a[3] == Py_None ? nullptr : &like(a[3], x, {M, N}, "residual");
    const int64_t ldr = r ? rows(*r, "residual") : 0;
    const int act = activation(a[4]);
    const bool need_pre = truth(a[5]);
    const c10::DeviceGuard guard(x.device());
    const Tensor y = output(a[6], x, {M, N});
    const int64_t ldy = rows(y, "out");
    const Tensor pre = need_pre ? empty(x, {M, N}) : Tensor();
    const Scratch ws(x, CP_OP_LINEAR, M, K, N, 0, aligned(x, {&x, &w}, {ldx, K, ldw, N}));
    check(cp_linear(code(x), M, K, N, x.data_ptr(), ldx, w.data_ptr(), ldw, wt, bias, r ? r->data_ptr() : nullptr, ldr, act,
                    y.data_ptr(), ldy, data(pre), N, data(ws.t), ws.n, stream(x)),
          "cp_linear");
    written(y);
    return need_pre ? wrap_tuple(y, pre) : wrap(y);
}

// linear_backward(dy, x, w, pre, act, need_x, need_w, need_bias)
PyObject *linear_backward(PyObject *const *a) {
    const Tensor &dy = first(a[0], "dy");
    const int64_t M = dy.size(0), N = dy.size(1);
    const Tensor &w = tensor(a[2], "w");
    if (w.dim() != 2) refuse(PyExc_ValueError, "w must be a matrix");
    const int64_t K = w.size(0);
    like(a[2], dy, {K, N}, "w");
    const Tensor &x = like(a[1], dy, {M, K}, "x");
    bool wt;
    const int64_t ldw = weight(w, &wt), ldd = rows(dy, "dy"), ldx = rows(x, "x");
    const int act = activation(a[4]);
    if (act != CP_ACT_NONE && a[3] == Py_None) refuse(PyExc_ValueError, "pre is needed with an activation");
    const Tensor *pre = act == CP_ACT_NONE ? nullptr : &like(a[3], dy, {M, N}, "pre");
    const int64_t ldp = pre ? rows(*pre, "pre") : 0;
    const bool need_x = truth(a[5]), need_w = truth(a[6]), need_b = truth(a[7]);
    const c10::DeviceGuard guard(dy.device());
    const Tensor dx = need_x ? empty(dy, {M, K}) : Tensor(), dw = need_w ? empty_weight(w, wt) : Tensor();
    const Tensor db = need_b ? empty(dy, {N}) : Tensor();
    const Scratch ws(dy, CP_OP_LINEAR_BACKWARD, M, K, N, 0, aligned(dy, {&dy, &x, &w}, {ldd, ldx, ldw, K, N}));
    check(cp_linear_backward(code(dy), M, K, N, dy.data_ptr(), ldd, x.data_ptr(), ldx, w.data_ptr(), ldw, wt,
                             pre ? pre->data_ptr() : nullptr, ldp, act, data(dx), K, data(dw), wt ? K : N, data(db),
                             data(ws.t), ws.n, stream(dy)),
          "cp_linear_backward");
    return wrap_tuple(dx, dw, db);
}

// grouped_linear(x, w, offsets, bias, act, need_pre, out)
PyObject *grouped_linear(PyObject *const *a) {
    const Tensor &x = first(a[0], "x");
    const Tensor *off;
    const Tensor &w = experts(a[1], a[2], x, &off);
    const int64_t T = x.size(0), K = x.size(1), E = w.size(0), N = w.size(2), sw = w.stride(0);
    like(a[1], x, {E, K, N}, "w");
    bool wt;
    const int64_t ldw = weight(w, &wt), ldx = rows(x, "x");
    const void *bias = optional_vector(a[3], x, {E, N}, "bias");
    const int act = activation(a[4]);
    const bool need_pre = truth(a[5]);
    const c10::DeviceGuard guard(x.device());
    const Tensor y = output(a[6], x, {T, N});
    const int64_t ldy = rows(y, "out");
    const Tensor pre = need_pre ? empty(x, {T, N}) : Tensor();
    const Scratch ws(x, CP_OP_GROUPED_LINEAR, T, K, N, E, aligned(x, {&x, &w}, {ldx, K, ldw, N, sw}));
    check(cp_grouped_linear(code(x), T, K, N, (int32_t)E, x.data_ptr(), ldx, w.data_ptr(), ldw, sw, wt,
                            (const int32_t *)off->data_ptr(), bias, act, y.data_ptr(), ldy, data(pre), N, data(ws.t), ws.n,
                            stream(x)),
          "cp_grouped_linear");
    written(y);
    return need_pre ? wrap_tuple(y, pre) : wrap(y);
}

// grouped_linear_backward(dy, x, w, offsets, pre, act, need_x, need_w, need_bias)
PyObject *grouped_linear_backward(PyObject *const *a) {
    const Tensor &dy = first(a[0], "dy");
    const Tensor *off;
    const Tensor &w = experts(a[2], a[3], dy, &off);
    const int64_t T = dy.size(0), N = dy.size(1), E = w.size(0), K = w.size(1), sw = w.stride(0);
    like(a[2], dy, {E, K, N}, "w");
    const Tensor &x = like(a[1], dy, {T, K}, "x");
    bool wt;
    const int64_t ldw = weight(w, &wt), ldd = rows(dy, "dy"), ldx = rows(x, "x");
    const int act = activation(a[5]);
    if (act != CP_ACT_NONE && a[4] == Py_None) refuse(PyExc_ValueError, "pre is needed with an activation");
    const Tensor *pre = act == CP_ACT_NONE ? nullptr : &like(a[4], dy, {T, N}, "pre");
    const int64_t ldp = pre ? rows(*pre, "pre") : 0;
    const bool need_x = truth(a[6]), need_w = truth(a[7]), need_b = truth(a[8]);
    const c10::DeviceGuard guard(dy.device());
    const Tensor dx = need_x ? empty(dy, {T, K}) : Tensor(), dw = need_w ? empty_weight(w, wt) : Tensor();
    const Tensor db = need_b ? empty(dy, {E, N}) : Tensor();
    const Scratch ws(dy, CP_OP_GROUPED_LINEAR_BACKWARD, T, K, N, E, aligned(dy, {&dy, &x, &w}, {ldd, ldx, ldw, K, N, sw}));
    check(cp_grouped_linear_backward(code(dy), T, K, N, (int32_t)E, dy.data_ptr(), ldd, x.data_ptr(), ldx, w.data_ptr(), ldw,
                                     sw, wt, (const int32_t *)off->data_ptr(), pre ? pre->data_ptr() : nullptr, ldp, act,
                                     data(dx), K, data(dw), wt ? K : N, K * N, data(db), data(ws.t), ws.n, stream(dy)),
          "cp_grouped_linear_backward");
    return wrap_tuple(dx, dw, db);
}

// layer_norm(x, weight, bias, eps, out)
PyObject *layer_norm(PyObject *const *a) {
    const Tensor &x = first(a[0], "x");
    const int64_t M = x.size(0), N = x.size(1), ldx = rows(x, "x");
    const void *w = optional_vector(a[1], x, {N}, "weight"), *b = optional_vector(a[2], x, {N}, "bias");
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raised{};
    const c10::DeviceGuard guard(x.device());
    const Tensor y = output(a[4], x, {M, N});
    const int64_t ldy = rows(y, "out");
    const auto f32 = x.options().dtype(at::kFloat);
    const Tensor mean = at::empty({M}, f32), rstd = at::empty({M}, f32);
    check(cp_layer_norm(code(x), M, N, x.data_ptr(), ldx, w, b, (float)eps, y.data_ptr(), ldy, (float *)mean.data_ptr(),
                        (float *)rstd.data_ptr(), stream(x)),
          "cp_layer_norm");
    written(y);
    return wrap_tuple(y, mean, rstd);
}

// layer_norm_backward(dy, x, mean, rstd, weight, need_x, need_weight, need_bias)
PyObject *layer_norm_backward(PyObject *const *a) {
    const Tensor &dy = first(a[0], "dy");
    const int64_t M = dy.size(0), N = dy.size(1);
    const Tensor &x = like(a[1], dy, {M, N}, "x");
    const int64_t ldd = rows(dy, "dy"), ldx = rows(x, "x");
    const void *mean = vector(a[2], dy, {M}, "mean", at::kFloat), *rstd = vector(a[3], dy, {M}, "rstd", at::kFloat);
    const void *w = optional_vector(a[4], dy, {N}, "weight");
    const bool need_x = truth(a[5]), need_w = truth(a[6]), need_b = truth(a[7]);
    const c10::DeviceGuard guard(dy.device());
    const Tensor dx = need_x ? empty(dy, {M, N}) : Tensor(), dw = need_w ? empty(dy, {N}) : Tensor();
    const Tensor db = need_b ? empty(dy, {N}) : Tensor();
    const Scratch ws(dy, CP_OP_LAYER_NORM_BACKWARD, M, 0, N, 0, true);
    check(cp_layer_norm_backward(code(dy), M, N, dy.data_ptr(), ldd, x.data_ptr(), ldx, (const float *)mean,
                                 (const float *)rstd, w, data(dx), N, data(dw), data(db), data(ws.t), ws.n, stream(dy)),
          "cp_layer_norm_backward");
    return wrap_tuple(dx, dw, db);
}

// Argument count, and C++ exceptions into Python's (torch's own, out of memory
// among them, keep their types).
template <PyObject *(*F)(PyObject *const *), int ARGS>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != ARGS) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", ARGS, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused &r) {
        PyErr_SetString(r.type, r.what.c_str());
        return nullptr;
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *set_error(PyObject *, PyObject *f) {
    Py_INCREF(f);
    Py_XDECREF(g_error);
    g_error = f;
    Py_RETURN_NONE;
}

#define CP_METHOD(name, args) {#name, (PyCFunction)(void (*)(void))entry<name, args>, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {CP_METHOD(linear, 7),
                           CP_METHOD(linear_backward, 8),
                           CP_METHOD(grouped_linear, 7),
                           CP_METHOD(grouped_linear_backward, 9),
                           CP_METHOD(layer_norm, 5),
                           CP_METHOD(layer_norm_backward, 8),
                           {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_cp_ops_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cp_ops_torch() { return PyModule_Create(&g_module); }
