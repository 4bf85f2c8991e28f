"""Feed-forward operators on torch tensors: linear layers with a fused epilogue,
linear layers grouped by expert, and layer normalisation, each with its
backward pass.

    y = act(x w + b) + residual
    y_t = act(x_t w_e + b_e)            rows sorted by expert
    y = (x - mean) rstd w + b

Binding of include/cp_ops.h: argument checks and marshalling only, every
arithmetic step runs in libcpchain.so, and there is no fallback.  All tensors
of a call are on one device and share one element type (float32 or bfloat16).
The work is enqueued on the device's current stream, outputs and scratch memory
come from PyTorch's allocator on that stream, and nothing is synchronised, so
the calls can be captured into a graph.  Rows must have unit stride; any row
stride that does not overlap is taken, and a weight may be a transposed view of
a stored [N][K] matrix.  Weight gradients come back in the weight's layout.
"""
import ctypes
import functools

import torch

from . import native as nat

ACT_NONE, ACT_GELU_TANH, ACT_RELU, ACT_SILU = 0, 1, 2, 3
ACTS = {"none": ACT_NONE, "gelu_tanh": ACT_GELU_TANH, "relu": ACT_RELU, "silu": ACT_SILU}
OP_LINEAR, OP_LINEAR_BACKWARD, OP_GROUPED_LINEAR, OP_GROUPED_LINEAR_BACKWARD, OP_LAYER_NORM_BACKWARD = range(5)
MAX_WIDTH = 4194304
MAX_GROUPS = 4096

# every symbol include/cp_ops.h declares
EXPORTS = ("cp_linear", "cp_linear_backward", "cp_grouped_linear", "cp_grouped_linear_backward", "cp_layer_norm",
           "cp_layer_norm_backward", "cp_ops_workspace", "cp_ops_last_error")

_lib = nat.lib()
_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


def _declare(name, restype, *argtypes):
    f = getattr(_lib, name)
    f.restype, f.argtypes = restype, list(argtypes)
    return f


_MAT, _TAIL = (_vp, _i64), (_vp, _i64, _vp)  # pointer and row stride; workspace, its bytes, stream
_SIZES = (_i32, _i64, _i64, _i64)            # dtype, M, K, N
_linear = _declare("cp_linear", ctypes.c_int, *_SIZES, *_MAT, *_MAT, _i32, _vp, *_MAT, _i32, *_MAT, *_MAT, *_TAIL)
_linear_backward = _declare("cp_linear_backward", ctypes.c_int, *_SIZES, *_MAT, *_MAT, *_MAT, _i32, *_MAT, _i32, *_MAT,
                            *_MAT, _vp, *_TAIL)
_grouped_linear = _declare("cp_grouped_linear", ctypes.c_int, *_SIZES, _i32, *_MAT, *_MAT, _i64, _i32, _vp, _vp, _i32,
                           *_MAT, *_MAT, *_TAIL)
_grouped_linear_backward = _declare("cp_grouped_linear_backward", ctypes.c_int, *_SIZES, _i32, *_MAT, *_MAT, *_MAT, _i64,
                                    _i32, _vp, *_MAT, _i32, *_MAT, *_MAT, _i64, _vp, *_TAIL)
_layer_norm = _declare("cp_layer_norm", ctypes.c_int, _i32, _i64, _i64, *_MAT, _vp, _vp, _f32, *_MAT, _vp, _vp, _vp)
_layer_norm_backward = _declare("cp_layer_norm_backward", ctypes.c_int, _i32, _i64, _i64, *_MAT, *_MAT, _vp, _vp, _vp,
                                *_MAT, _vp, _vp, *_TAIL)
_workspace = _declare("cp_ops_workspace", _i64, _i32, _i32, _i64, _i64, _i64, _i32, _i32)
_last_error = _declare("cp_ops_last_error", ctypes.c_char_p)

_CODES = {torch.float32: nat.CP_F32, torch.bfloat16: nat.CP_BF16}


def _check(rc, where):
    if rc < 0:
        raise nat.CpError(rc, where, _last_error().decode())
    return rc


@functools.lru_cache(maxsize=4096)
def workspace_bytes(op, dtype, M, K, N, E=0, aligned=False):
    """Bytes of scratch memory an operator takes (cp_ops_workspace)."""
    return _check(_workspace(op, dtype, M, K, N, E, aligned), "cp_ops_workspace")


def _like(t, x, shape, name, dtype=None):
    """t is a device tensor of x's device and type (or `dtype`) with this shape."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device != x.device:
        raise ValueError(f"{name} is on {t.device}, expected {x.device}")
    want = dtype or x.dtype
    if t.dtype != want or t.shape != shape:
        raise ValueError(f"{name} must be a {want} tensor of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    return t


def _first(x, dims, name):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if x.dtype not in _CODES:
        raise ValueError(f"{name} must be float32 or bfloat16, got {x.dtype}")
    if x.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {x.dim()}")
    return _CODES[x.dtype]


def _rows(t, name):
    """Row stride of a matrix with unit stride within its rows."""
    s0, s1 = t.stride()
    M, N = t.shape
    if s1 != 1 and N > 1 and M > 0:
        raise ValueError(f"{name} must have unit stride within a row (strides {t.stride()}); call .contiguous()")
    if s0 < N and M > 1:
        raise ValueError(f"the rows of {name} overlap (strides {t.stride()}); call .contiguous()")
    return s0


def _weight(w, name):
    """(row stride, stored transposed) of a weight matrix [K][N], or the last two dimensions of [E][K][N]."""
    s0, s1 = w.stride()[-2:]
    K, N = w.shape[-2:]
    if s1 == 1 and (s0 >= N or K <= 1) and N > 1:
        return s0, 0
    if (s0 == 1 or K <= 1) and (s1 >= K or N <= 1):
        return s1, 1
    if s1 == 1 or N <= 1:
        if s0 >= N or K <= 1:
            return s0, 0
    raise ValueError(f"{name} must be rows of unit stride that do not overlap, or the transpose of such "
                     f"(strides {w.stride()}); call .contiguous()")


def _vector(b, x, shape, name, dtype=None):
    _like(b, x, shape, name, dtype)
    if not b.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return b.data_ptr()


def _empty_weight(w, wt):
    """A gradient with w's layout."""
    if not wt:
        return torch.empty(w.shape, dtype=w.dtype, device=w.device)
    shape = (*w.shape[:-2], w.shape[-1], w.shape[-2])
    return torch.empty(shape, dtype=w.dtype, device=w.device).transpose(-1, -2)


def _elsewhere(x):
    """Whether the tensor's device is not the current one."""
    return x.get_device() != torch.cuda.current_device()


# The current stream's handle without a stream object around it: the calls below
# cost a few microseconds each, and the object alone takes three.
_stream = torch._C._cuda_getCurrentRawStream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _scratch(op, code, M, K, N, E, x, aligned):
    n = workspace_bytes(op, code, M, K, N, E, aligned)
    return (torch.empty(n, dtype=torch.uint8, device=x.device) if n else None), n


def linear(x, w, bias=None, residual=None, act=ACT_NONE, need_pre=False, out=None):
    """act(x w + bias) + residual: x [M][K], w [K][N], bias [N], residual [M][N].
    With need_pre returns (y, x w + bias), the second for linear_backward.  `out`
    may be the residual itself."""
    code = _first(x, 2, "x")
    if _elsewhere(x):
        with torch.cuda.device(x.device):
            return linear(x, w, bias, residual, act, need_pre, out)
    M, K = x.shape
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a matrix")
    N = w.shape[1]
    _like(w, x, (K, N), "w")
    ldw, wt = _weight(w, "w")
    b = None if bias is None else _vector(bias, x, (N,), "bias")
    ldr = 0 if residual is None else _rows(_like(residual, x, (M, N), "residual"), "residual")
    y = x.new_empty((M, N)) if out is None else _like(out, x, (M, N), "out")
    pre = torch.empty_like(y, memory_format=torch.contiguous_format) if need_pre else None
    xp, wp, ldx = x.data_ptr(), w.data_ptr(), _rows(x, "x")
    es = x.element_size()
    ws, n = _scratch(OP_LINEAR, code, M, K, N, 0, x, not ((xp | wp | (ldx | K | ldw | N) * es) & 15))
    _check(_linear(code, M, K, N, xp, ldx, wp, ldw, wt, b, _ptr(residual), ldr, act, y.data_ptr(),
                   N if out is None else _rows(y, "out"), _ptr(pre), N, _ptr(ws), n, _stream(x.get_device())),
           "cp_linear")
    return (y, pre) if need_pre else y


def linear_backward(dy, x, w, pre=None, act=ACT_NONE, need_x=True, need_w=True, need_bias=True):
    """Gradients (dx, dw, db) of linear for dy [M][N]; None for those not asked
    for.  `pre` is what linear returned with need_pre (not needed without an
    activation).  The residual's gradient is dy."""
    code = _first(dy, 2, "dy")
    if _elsewhere(dy):
        with torch.cuda.device(dy.device):
            return linear_backward(dy, x, w, pre, act, need_x, need_w, need_bias)
    M, N = dy.shape
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a matrix")
    K = w.shape[0]
    _like(w, dy, (K, N), "w")
    _like(x, dy, (M, K), "x")
    ldw, wt = _weight(w, "w")
    ldp = _backward_pre(pre, dy, act)
    dx = dy.new_empty((M, K)) if need_x else None
    dw = _empty_weight(w, wt) if need_w else None
    db = dy.new_empty(N) if need_bias else None
    dp, xp, wp, ldd, ldx = dy.data_ptr(), x.data_ptr(), w.data_ptr(), _rows(dy, "dy"), _rows(x, "x")
    ws, n = _scratch(OP_LINEAR_BACKWARD, code, M, K, N, 0, dy,
                     not ((dp | xp | wp | (ldd | ldx | ldw | K | N) * dy.element_size()) & 15))
    _check(_linear_backward(code, M, K, N, dp, ldd, xp, ldx, wp, ldw, wt, _ptr(pre), ldp, act, _ptr(dx), K, _ptr(dw),
                            K if wt else N, _ptr(db), _ptr(ws), n, _stream(dy.get_device())), "cp_linear_backward")
    return dx, dw, db


def _backward_pre(pre, dy, act):
    if act == ACT_NONE:
        return 0
    if pre is None:
        raise ValueError("pre is needed with an activation")
    return _rows(_like(pre, dy, dy.shape, "pre"), "pre")


def _experts(w, x, offsets):
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise ValueError("w must have 3 dimensions [E][K][N]")
    E = w.shape[0]
    if not isinstance(offsets, torch.Tensor) or offsets.dtype != torch.int32 or offsets.shape != (E + 1,) \
            or not offsets.is_contiguous() or offsets.device != x.device:
        raise ValueError(f"offsets must be a contiguous int32 tensor of {E + 1} elements on {x.device}")
    return E, w.stride(0)


def grouped_linear(x, w, offsets, bias=None, act=ACT_NONE, need_pre=False, out=None):
    """act(x_t w_e + bias_e) for rows sorted by expert: x [T][K], w [E][K][N],
    bias [E][N]; expert e has rows offsets[e] .. offsets[e + 1] - 1 (int32, on
    the device, never read by the host).  Rows from offsets[E] on give zeros."""
    code = _first(x, 2, "x")
    if _elsewhere(x):
        with torch.cuda.device(x.device):
            return grouped_linear(x, w, offsets, bias, act, need_pre, out)
    E, sw = _experts(w, x, offsets)
    T, K = x.shape
    N = w.shape[2]
    _like(w, x, (E, K, N), "w")
    ldw, wt = _weight(w, "w")
    b = None if bias is None else _vector(bias, x, (E, N), "bias")
    y = x.new_empty((T, N)) if out is None else _like(out, x, (T, N), "out")
    pre = torch.empty_like(y, memory_format=torch.contiguous_format) if need_pre else None
    xp, wp, ldx = x.data_ptr(), w.data_ptr(), _rows(x, "x")
    ws, n = _scratch(OP_GROUPED_LINEAR, code, T, K, N, E, x,
                     not ((xp | wp | (ldx | K | ldw | N | sw) * x.element_size()) & 15))
    _check(_grouped_linear(code, T, K, N, E, xp, ldx, wp, ldw, sw, wt, offsets.data_ptr(), b, act, y.data_ptr(),
                           N if out is None else _rows(y, "out"), _ptr(pre), N, _ptr(ws), n, _stream(x.get_device())),
           "cp_grouped_linear")
    return (y, pre) if need_pre else y


def grouped_linear_backward(dy, x, w, offsets, pre=None, act=ACT_NONE, need_x=True, need_w=True, need_bias=True):
    """Gradients (dx, dw, db) of grouped_linear for dy [T][N]; zeros for experts
    without rows and for rows without an expert."""
    code = _first(dy, 2, "dy")
    if _elsewhere(dy):
        with torch.cuda.device(dy.device):
            return grouped_linear_backward(dy, x, w, offsets, pre, act, need_x, need_w, need_bias)
    E, sw = _experts(w, dy, offsets)
    T, N = dy.shape
    K = w.shape[1]
    _like(w, dy, (E, K, N), "w")
    _like(x, dy, (T, K), "x")
    ldw, wt = _weight(w, "w")
    ldp = _backward_pre(pre, dy, act)
    dx = dy.new_empty((T, K)) if need_x else None
    dw = _empty_weight(w, wt) if need_w else None
    db = dy.new_empty((E, N)) if need_bias else None
    dp, xp, wp, ldd, ldx = dy.data_ptr(), x.data_ptr(), w.data_ptr(), _rows(dy, "dy"), _rows(x, "x")
    ws, n = _scratch(OP_GROUPED_LINEAR_BACKWARD, code, T, K, N, E, dy,
                     not ((dp | xp | wp | (ldd | ldx | ldw | K | N | sw) * dy.element_size()) & 15))
    _check(_grouped_linear_backward(code, T, K, N, E, dp, ldd, xp, ldx, wp, ldw, sw, wt, offsets.data_ptr(), _ptr(pre),
                                    ldp, act, _ptr(dx), K, _ptr(dw), K if wt else N, K * N, _ptr(db), _ptr(ws), n,
                                    _stream(dy.get_device())), "cp_grouped_linear_backward")
    return dx, dw, db


def layer_norm(x, weight=None, bias=None, eps=1e-5, out=None):
    """(y, mean, rstd) with y = (x - mean) rstd weight + bias over the rows of
    x [M][N]; mean and rstd are float32 [M].  `out` may be x."""
    code = _first(x, 2, "x")
    if _elsewhere(x):
        with torch.cuda.device(x.device):
            return layer_norm(x, weight, bias, eps, out)
    M, N = x.shape
    w = None if weight is None else _vector(weight, x, (N,), "weight")
    b = None if bias is None else _vector(bias, x, (N,), "bias")
    y = x.new_empty((M, N)) if out is None else _like(out, x, (M, N), "out")
    mean, rstd = torch.empty((2, M), dtype=torch.float32, device=x.device).unbind()
    _check(_layer_norm(code, M, N, x.data_ptr(), _rows(x, "x"), w, b, eps, y.data_ptr(),
                       N if out is None else _rows(y, "out"), mean.data_ptr(), rstd.data_ptr(),
                       _stream(x.get_device())), "cp_layer_norm")
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None, need_x=True, need_weight=True, need_bias=True):
    """Gradients (dx, dweight, dbias) of layer_norm for dy [M][N], from the mean
    and rstd it returned; None for those not asked for."""
    code = _first(dy, 2, "dy")
    if _elsewhere(dy):
        with torch.cuda.device(dy.device):
            return layer_norm_backward(dy, x, mean, rstd, weight, need_x, need_weight, need_bias)
    M, N = dy.shape
    _like(x, dy, (M, N), "x")
    m, r = _vector(mean, dy, (M,), "mean", torch.float32), _vector(rstd, dy, (M,), "rstd", torch.float32)
    w = None if weight is None else _vector(weight, dy, (N,), "weight")
    dx = dy.new_empty((M, N)) if need_x else None
    dw = dy.new_empty(N) if need_weight else None
    db = dy.new_empty(N) if need_bias else None
    ws, n = _scratch(OP_LAYER_NORM_BACKWARD, code, M, 0, N, 0, dy, True)
    _check(_layer_norm_backward(code, M, N, dy.data_ptr(), _rows(dy, "dy"), x.data_ptr(), _rows(x, "x"), m, r, w,
                                _ptr(dx), N, _ptr(dw), _ptr(db), _ptr(ws), n, _stream(dy.get_device())),
           "cp_layer_norm_backward")
    return dx, dw, db
