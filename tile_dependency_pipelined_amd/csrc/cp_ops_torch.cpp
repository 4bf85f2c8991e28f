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
#include <optional>
#include <string>
#include <vector>

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

// ---- router, exchange of rows, 4-bit layers, clipping ----------------------

int64_t integer(PyObject *o, const char *name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (v != (int32_t)v) refuse(PyExc_ValueError, "%s = %lld is out of range", name, v);
    return v;
}
double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
}

// Outputs of one element type in one allocation on the current device, each from a
// multiple of 256 bytes on: at::empty costs as much as a quarter of a launch each time,
// its allocator alone less.  (Not outputs of two types: torch.save refuses memory that
// tensors view as both.)
struct Pool {
    c10::Storage storage;
    caffe2::TypeMeta type;
    int64_t used = 0;
    static int64_t up(int64_t n) { return (n + 63) / 64 * 64; }  // elements of 4 bytes
    static size_t bytes(std::initializer_list<int64_t> elements) {
        int64_t n = 0;
        for (int64_t e : elements) n += up(e);
        return (size_t)n * 4;
    }
    // at::empty's allocator, the same for every device and as long as the process lives
    static c10::Allocator *allocator(const Tensor &x) {
        static c10::Allocator *const a = at::empty({0}, x.options()).storage().allocator();
        return a;
    }
    Pool(const Tensor &x, at::ScalarType t, std::initializer_list<int64_t> elements)
        : storage(c10::Storage::use_byte_size_t(), bytes(elements), allocator(x), true), type(c10::scalarTypeToTypeMeta(t)) {}
    Tensor take(at::IntArrayRef shape) {
        auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(storage), c10::DispatchKeySet(c10::DispatchKey::CUDA), type);
        impl->set_storage_offset(used);
        impl->set_sizes_contiguous(shape);
        used += up(impl->numel());
        return Tensor(std::move(impl));
    }
};

// An int32 matrix [T][k] of a token's slots.
const Tensor &slots(PyObject *o, const Tensor &x, const char *name) {
    const Tensor &t = tensor(o, name);
    if (t.scalar_type() != at::kInt || t.dim() != 2 || !t.is_contiguous() || t.device() != x.device())
        refuse(PyExc_ValueError, "%s must be a contiguous int32 matrix on %s", name, x.device().str().c_str());
    if (t.size(1) > INT32_MAX) refuse(PyExc_ValueError, "%s has %lld slots to a token", name, (long long)t.size(1));
    return t;
}
// The last of offsets [E + 1].
const int32_t *last_offset(PyObject *o, const Tensor &x) {
    const Tensor &t = tensor(o, "offsets");
    if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) < 1 || !t.is_contiguous() || t.device() != x.device())
        refuse(PyExc_ValueError, "offsets must be a contiguous int32 vector on %s", x.device().str().c_str());
    return (const int32_t *)t.data_ptr() + (t.size(0) - 1);
}

// route(logits, k, normalize, valid) -> experts, gates, rows, counts, offsets, loss, slopes
PyObject *route(PyObject *const *a) {
    const Tensor &x = first(a[0], "logits");
    const int64_t T = x.size(0), E = x.size(1), k = integer(a[1], "k"), ld = rows(x, "logits");
    const bool normalize = truth(a[2]);
    const void *valid = a[3] == Py_None ? nullptr : vector(a[3], x, {T}, "valid", at::kBool);
    if (E < 1 || E > CP_OPS_MAX_ROUTED || k < 1 || k > E || k > CP_OPS_MAX_CHOSEN)
        refuse(PyExc_ValueError, "%lld of %lld experts to a token (1 to %d of at most %d)", (long long)k, (long long)E,
               CP_OPS_MAX_CHOSEN, CP_OPS_MAX_ROUTED);
    const c10::DeviceGuard guard(x.device());
    const int64_t ws = cp_ops_workspace(CP_OP_ROUTE, code(x), T, 0, E, 0, 1);
    check(ws, "cp_ops_workspace");
    Pool ints(x, at::kInt, {T * k, T * k, E, E + 1}), floats(x, at::kFloat, {T * k, E}), one(x, at::kFloat, {1});
    const Tensor experts = ints.take({T, k}), places = ints.take({T, k}), counts = ints.take({E}), offsets = ints.take({E + 1});
    const Tensor gates = floats.take({T, k}), slopes = floats.take({E});
    const Tensor loss = one.take({});  // by itself: the one that a program keeps for its log
    const Tensor scratch = ws ? at::empty({ws}, x.options().dtype(at::kByte)) : Tensor();
    check(cp_route(code(x), T, (int32_t)E, (int32_t)k, normalize, x.data_ptr(), ld, (const uint8_t *)valid,
                   (int32_t *)experts.data_ptr(), (float *)gates.data_ptr(), (int32_t *)places.data_ptr(),
                   (int32_t *)counts.data_ptr(), (int32_t *)offsets.data_ptr(), (float *)loss.data_ptr(),
                   (float *)slopes.data_ptr(), data(scratch), ws, stream(x)),
          "cp_route");
    return wrap_tuple(experts, gates, places, counts, offsets, loss, slopes);
}

// route_backward(dgates, dloss, logits, experts, slopes, normalize)
PyObject *route_backward(PyObject *const *a) {
    const Tensor &x = first(a[2], "logits");
    const int64_t T = x.size(0), E = x.size(1), ld = rows(x, "logits");
    if (E > CP_OPS_MAX_ROUTED) refuse(PyExc_ValueError, "%lld experts (at most %d)", (long long)E, CP_OPS_MAX_ROUTED);
    const Tensor &experts = slots(a[3], x, "experts");
    const int64_t k = experts.size(1);
    like(a[3], x, {T, k}, "experts", at::kInt);
    const void *dgates = a[0] == Py_None ? nullptr : vector(a[0], x, {T, k}, "dgates", at::kFloat);
    const void *dloss = a[1] == Py_None ? nullptr : vector(a[1], x, {}, "dloss", at::kFloat);
    const void *slopes = dloss ? vector(a[4], x, {E}, "slopes", at::kFloat) : nullptr;
    const bool normalize = truth(a[5]);
    const c10::DeviceGuard guard(x.device());
    const Tensor d = empty(x, {T, E});
    check(cp_route_backward(code(x), T, (int32_t)E, (int32_t)k, normalize, (const float *)dgates, (const float *)dloss,
                            x.data_ptr(), ld, (const int32_t *)experts.data_ptr(), (const float *)slopes, d.data_ptr(), E,
                            stream(x)),
          "cp_route_backward");
    return wrap(d);
}

// dispatch(x, rows, offsets, out)
PyObject *dispatch(PyObject *const *a) {
    const Tensor &x = first(a[0], "x");
    const int64_t T = x.size(0), D = x.size(1), ldx = rows(x, "x");
    const Tensor &places = slots(a[1], x, "rows");
    const int64_t k = places.size(1), R = T * k;
    like(a[1], x, {T, k}, "rows", at::kInt);
    const int32_t *end = last_offset(a[2], x);
    const c10::DeviceGuard guard(x.device());
    const Tensor out = output(a[3], x, {R, D});
    const int64_t ldo = rows(out, "out");
    check(cp_dispatch(code(x), T, (int32_t)k, R, D, x.data_ptr(), ldx, (const int32_t *)places.data_ptr(), end,
                      out.data_ptr(), ldo, stream(x)),
          "cp_dispatch");
    written(out);
    return wrap(out);
}

// combine(y, rows, gates, residual, out)
PyObject *combine(PyObject *const *a) {
    const Tensor &y = first(a[0], "y");
    const int64_t R = y.size(0), D = y.size(1), ldy = rows(y, "y");
    const Tensor &places = slots(a[1], y, "rows");
    const int64_t T = places.size(0), k = places.size(1);
    const void *gates = a[2] == Py_None ? nullptr : vector(a[2], y, {T, k}, "gates", at::kFloat);
    const Tensor *r = a[3] == Py_None ? nullptr : &like(a[3], y, {T, D}, "residual");
    const int64_t ldr = r ? rows(*r, "residual") : 0;
    const c10::DeviceGuard guard(y.device());
    const Tensor out = output(a[4], y, {T, D});
    const int64_t ldo = rows(out, "out");
    check(cp_combine(code(y), T, (int32_t)k, R, D, y.data_ptr(), ldy, (const int32_t *)places.data_ptr(), (const float *)gates,
                     r ? r->data_ptr() : nullptr, ldr, out.data_ptr(), ldo, stream(y)),
          "cp_combine");
    written(out);
    return wrap(out);
}

// combine_backward(dout, y, rows, offsets, gates, need_y, need_gates)
PyObject *combine_backward(PyObject *const *a) {
    const Tensor &d = first(a[0], "dout");
    const int64_t T = d.size(0), D = d.size(1), ldd = rows(d, "dout");
    const Tensor &y = tensor(a[1], "y");
    if (y.dim() != 2) refuse(PyExc_ValueError, "y must have 2 dimensions, got %d", (int)y.dim());
    const int64_t R = y.size(0);
    like(a[1], d, {R, D}, "y");
    const int64_t ldy = rows(y, "y");
    const Tensor &places = slots(a[2], d, "rows");
    const int64_t k = places.size(1);
    like(a[2], d, {T, k}, "rows", at::kInt);
    const int32_t *end = last_offset(a[3], d);
    const void *gates = a[4] == Py_None ? nullptr : vector(a[4], d, {T, k}, "gates", at::kFloat);
    const bool need_y = truth(a[5]), need_gates = truth(a[6]);
    const c10::DeviceGuard guard(d.device());
    const Tensor dy = need_y ? empty(d, {R, D}) : Tensor();
    const Tensor dg = need_gates ? at::empty({T, k}, d.options().dtype(at::kFloat)) : Tensor();
    check(cp_combine_backward(code(d), T, (int32_t)k, R, D, d.data_ptr(), ldd, y.data_ptr(), ldy,
                              (const int32_t *)places.data_ptr(), end, (const float *)gates, data(dy), D, (float *)data(dg),
                              stream(d)),
          "cp_combine_backward");
    return wrap_tuple(dy, dg);
}

// Experts of a stack of weights, 1 for a single matrix.
int64_t stack(const Tensor &t, const char *name) {
    if (t.dim() != 2 && t.dim() != 3) refuse(PyExc_ValueError, "%s must have 2 or 3 dimensions, got %d", name, (int)t.dim());
    const int64_t E = t.dim() == 3 ? t.size(0) : 1;
    if (E < 1 || E > CP_OPS_MAX_GROUPS) refuse(PyExc_ValueError, "%lld experts (1 to %d)", (long long)E, CP_OPS_MAX_GROUPS);
    return E;
}
int64_t group_of(PyObject *o) {
    const int64_t g = integer(o, "group_size");
    if (g != 32 && g != 64 && (g < 128 || g % 128 || g > CP_OPS_MAX_WIDTH))
        refuse(PyExc_ValueError, "groups of %lld (32, 64 or a multiple of 128)", (long long)g);
    return g;
}
std::vector<int64_t> with_rows(const Tensor &t, int64_t rows) {
    auto s = t.sizes().vec();
    s[s.size() - 2] = rows;
    return s;
}

// quantize_int4(w, group_size, symmetric) -> codes, scales, zeros
PyObject *quantize_int4(PyObject *const *a) {
    if (!THPVariable_Check(a[0]) || !THPVariable_Unpack(a[0]).is_cuda()) refuse(PyExc_TypeError, "w must be a device tensor");
    const Tensor &w = THPVariable_Unpack(a[0]);
    if (w.scalar_type() != at::kFloat && w.scalar_type() != at::kBFloat16)
        refuse(PyExc_ValueError, "w must be float32 or bfloat16, got %s", c10::toString(w.scalar_type()));
    const int64_t E = stack(w, "w"), g = group_of(a[1]), d = w.dim(), K = w.size(d - 2), N = w.size(d - 1);
    const bool symmetric = truth(a[2]);
    const c10::DeviceGuard guard(w.device());
    const auto u8 = w.options().dtype(at::kByte);
    const auto per = with_rows(w, (K + g - 1) / g);
    const Tensor q = at::empty(w.sizes(), u8), scales = at::empty(per, w.options());
    const Tensor zeros = symmetric ? Tensor() : at::empty(per, u8);
    check(cp_int4_quantize(code(w), K, N, (int32_t)E, g, w.data_ptr(), w.stride(d - 2), w.stride(d - 1), d == 3 ? w.stride(0) : 0,
                           (uint8_t *)q.data_ptr(), scales.data_ptr(), (uint8_t *)data(zeros), stream(w)),
          "cp_int4_quantize");
    return wrap_tuple(q, scales, zeros);
}

// pack_int4(codes, scales, zeros, group_size) -> bytes
PyObject *pack_int4(PyObject *const *a) {
    if (!THPVariable_Check(a[1]) || !THPVariable_Unpack(a[1]).is_cuda()) refuse(PyExc_TypeError, "scales must be a device tensor");
    const Tensor &scales = THPVariable_Unpack(a[1]);
    if (scales.scalar_type() != at::kFloat && scales.scalar_type() != at::kBFloat16)
        refuse(PyExc_ValueError, "scales must be float32 or bfloat16, got %s", c10::toString(scales.scalar_type()));
    const Tensor &q = tensor(a[0], "codes");
    const int64_t E = stack(q, "codes"), g = group_of(a[3]), d = q.dim(), K = q.size(d - 2), N = q.size(d - 1);
    const void *codes = vector(a[0], scales, q.sizes(), "codes", at::kByte);
    const auto per = with_rows(q, (K + g - 1) / g);
    vector(a[1], scales, per, "scales", scales.scalar_type());
    const void *zeros = a[2] == Py_None ? nullptr : vector(a[2], scales, per, "zeros", at::kByte);
    const int64_t n = cp_int4_bytes(code(scales), K, N, (int32_t)E, g);
    check(n, "cp_int4_bytes");
    const c10::DeviceGuard guard(scales.device());
    const Tensor packed = at::empty({n}, scales.options().dtype(at::kByte));
    check(cp_int4_pack(code(scales), K, N, (int32_t)E, g, (const uint8_t *)codes, scales.data_ptr(), (const uint8_t *)zeros,
                       packed.data_ptr(), stream(scales)),
          "cp_int4_pack");
    return wrap(packed);
}

// A packed weight's data: as many bytes as its sizes say.
const Tensor &packed_weight(PyObject *o, const Tensor &x, int64_t K, int64_t N, int64_t E, int64_t group) {
    const int64_t n = cp_int4_bytes(code(x), K, N, (int32_t)E, group);
    check(n, "cp_int4_bytes");
    const Tensor &t = like(o, x, {n}, "the packed weight", at::kByte);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "the packed weight must be contiguous");
    return t;
}

// linear_int4(x, packed, N, group, bias, residual, act, out)
PyObject *linear_int4(PyObject *const *a) {
    const Tensor &x = first(a[0], "x");
    const int64_t M = x.size(0), K = x.size(1), ldx = rows(x, "x"), N = integer(a[2], "N"), g = group_of(a[3]);
    const Tensor &w = packed_weight(a[1], x, K, N, 1, g);
    const void *bias = optional_vector(a[4], x, {N}, "bias");
    const Tensor *r = a[5] == Py_None ? nullptr : &like(a[5], x, {M, N}, "residual");
    const int64_t ldr = r ? rows(*r, "residual") : 0;
    const int act = activation(a[6]);
    const c10::DeviceGuard guard(x.device());
    const Tensor y = output(a[7], x, {M, N});
    const int64_t ldy = rows(y, "out");
    const Scratch ws(x, CP_OP_LINEAR_INT4, M, K, N, 0, true);
    check(cp_linear_int4(code(x), M, K, N, x.data_ptr(), ldx, w.data_ptr(), g, bias, r ? r->data_ptr() : nullptr, ldr,
                         act, y.data_ptr(), ldy, data(ws.t), ws.n, stream(x)),
          "cp_linear_int4");
    written(y);
    return wrap(y);
}

// grouped_linear_int4(x, packed, E, N, group, offsets, bias, act, out)
PyObject *grouped_linear_int4(PyObject *const *a) {
    const Tensor &x = first(a[0], "x");
    const int64_t T = x.size(0), K = x.size(1), ldx = rows(x, "x"), E = integer(a[2], "E"), N = integer(a[3], "N");
    const int64_t g = group_of(a[4]);
    const Tensor &w = packed_weight(a[1], x, K, N, E, g);
    const void *off = vector(a[5], x, {E + 1}, "offsets", at::kInt);
    const void *bias = optional_vector(a[6], x, {E, N}, "bias");
    const int act = activation(a[7]);
    const c10::DeviceGuard guard(x.device());
    const Tensor y = output(a[8], x, {T, N});
    const int64_t ldy = rows(y, "out");
    const Scratch ws(x, CP_OP_LINEAR_INT4, T, K, N, E, true);
    check(cp_grouped_linear_int4(code(x), T, K, N, (int32_t)E, x.data_ptr(), ldx, w.data_ptr(), g, (const int32_t *)off,
                                 bias, act, y.data_ptr(), ldy, data(ws.t), ws.n, stream(x)),
          "cp_grouped_linear_int4");
    written(y);
    return wrap(y);
}

// A gradient: float32 or bfloat16 elements that fill their memory, in any order.
const Tensor &dense(PyObject *o, const char *name) {
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) refuse(PyExc_TypeError, "%s must be device tensors", name);
    const Tensor &t = THPVariable_Unpack(o);
    if (t.scalar_type() != at::kFloat && t.scalar_type() != at::kBFloat16)
        refuse(PyExc_ValueError, "%s must be float32 or bfloat16, got %s", name, c10::toString(t.scalar_type()));
    if (!t.is_non_overlapping_and_dense())
        refuse(PyExc_ValueError, "%s must fill their memory (strides %s); call .contiguous()", name,
               shape_text(t.strides()).c_str());
    return t;
}

// The tensors of any iterable, which is gone through once; they live as long as this.
struct Sequence {
    PyObject *s;
    explicit Sequence(PyObject *o) {
        PyObject *items = PySequence_Fast(o, "gradients and out must be sequences of tensors");
        if (!items) throw Raised{};
        s = PySequence_Tuple(items);  // (a list is the caller's and can change)
        Py_DECREF(items);
        if (!s) throw Raised{};
    }
    ~Sequence() { Py_DECREF(s); }
    Sequence(const Sequence &) = delete;
    Py_ssize_t size() const { return PyTuple_GET_SIZE(s); }
    PyObject *operator[](Py_ssize_t i) const { return PyTuple_GET_ITEM(s, i); }
};

// clip_grad_norm(gradients, max_norm, out, scale) -> norm; out: None for in place
PyObject *clip_grad_norm(PyObject *const *a) {
    const Sequence grads(a[0]);
    std::optional<Sequence> outs;
    if (a[2] != Py_None) outs.emplace(a[2]);
    const double max_norm = number(a[1]);
    const bool scale = truth(a[3]);
    const Py_ssize_t n = grads.size();
    if (n == 0) refuse(PyExc_ValueError, "no gradients");
    const Tensor &x0 = dense(grads[0], "gradients");
    std::vector<int32_t> types(n), out_types(n);
    std::vector<const void *> from(n);
    std::vector<void *> to(n);
    std::vector<int64_t> numels(n);
    auto enter = [&](Py_ssize_t i, const Tensor &x, const Tensor &y) {
        if (x.device() != x0.device() || y.device() != x0.device())
            refuse(PyExc_ValueError, "gradients and out must be on one device");
        types[i] = code(x);
        from[i] = x.data_ptr();
        numels[i] = x.numel();
        out_types[i] = code(y);
        to[i] = y.data_ptr();
    };
    auto writable = [](const Tensor &t) {
        if (c10::GradMode::is_enabled() && t.requires_grad())
            refuse(PyExc_RuntimeError, "a tensor to write requires a gradient, which is not recorded here; pass .detach() or "
                                       "call under torch.no_grad()");
    };
    if (!outs) {
        for (Py_ssize_t i = 0; i < n; ++i) {
            const Tensor &x = dense(grads[i], "gradients");
            if (scale) writable(x);
            enter(i, x, x);
        }
    } else {
        if (outs->size() != n) refuse(PyExc_ValueError, "%zd gradients and %zd outputs", n, outs->size());
        for (Py_ssize_t i = 0; i < n; ++i) {
            const Tensor &x = dense(grads[i], "gradients"), &y = dense((*outs)[i], "out");
            bool same = x.sizes() == y.sizes();
            for (int64_t d = 0; same && d < x.dim(); ++d)
                same = x.numel() == 0 || x.size(d) == 1 || x.stride(d) == y.stride(d);
            if (!same)
                refuse(PyExc_ValueError, "out %zd must have its gradient's shape and strides: %s %s, got %s %s", i,
                       shape_text(x.sizes()).c_str(), shape_text(x.strides()).c_str(), shape_text(y.sizes()).c_str(),
                       shape_text(y.strides()).c_str());
            writable(y);
            enter(i, x, y);
        }
    }
    const c10::DeviceGuard guard(x0.device());
    const Tensor norm = at::empty({}, x0.options().dtype(at::kFloat));
    const Scratch ws(x0, CP_OP_CLIP_GRAD_NORM, n, 0, 0, 0, true);
    check(cp_clip_grad_norm(n, types.data(), from.data(), numels.data(), (float)max_norm, out_types.data(),
                            scale ? to.data() : nullptr, (float *)norm.data_ptr(), data(ws.t), ws.n, stream(x0)),
          "cp_clip_grad_norm");
    if (scale)
        for (Py_ssize_t i = 0; i < n; ++i) written(THPVariable_Unpack(outs ? (*outs)[i] : grads[i]));
    return wrap(norm);
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
                           CP_METHOD(route, 4),
                           CP_METHOD(route_backward, 6),
                           CP_METHOD(dispatch, 4),
                           CP_METHOD(combine, 5),
                           CP_METHOD(combine_backward, 7),
                           CP_METHOD(quantize_int4, 3),
                           CP_METHOD(pack_int4, 4),
                           CP_METHOD(linear_int4, 8),
                           CP_METHOD(grouped_linear_int4, 9),
                           CP_METHOD(clip_grad_norm, 4),
                           {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_cp_ops_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cp_ops_torch() { return PyModule_Create(&g_module); }
