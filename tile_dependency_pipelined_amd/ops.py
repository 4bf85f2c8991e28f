"""Feed-forward operators on torch tensors: linear layers with a fused epilogue,
linear layers grouped by expert, layer normalisation, the router of an expert
layer and its rows' way to the experts and back, each with its backward pass;
linear layers with 4-bit weights; the gradients' norm and clipping.

    y = act(x w + b) + residual
    y_t = act(x_t w_e + b_e)            rows sorted by expert
    y = (x - mean) rstd w + b
    out_t = sum_j g_tj y[rows_tj] + residual_t
    w_kn = scale_gn (code_kn - zero_gn)

Every arithmetic step runs in libcpchain.so (include/cp_ops.h); the module
_cp_ops_torch checks the arguments and calls it.  There is no fallback: without the
built module the import of this one raises.  All tensors
of a call are on one device and share one element type (float32 or bfloat16).
The work is enqueued on the device's current stream, outputs and scratch memory
come from PyTorch's allocator on that stream, and nothing is synchronised, so
the calls can be captured into a graph.  Rows must have unit stride; any row
stride that does not overlap is taken, and a weight may be a transposed view of
a stored [N][K] matrix.  Weight gradients come back in the weight's layout.

No gradient is recorded, whatever the inputs require: results have no history, and
the *_backward functions are called by the program (or by its own
torch.autograd.Function).  A tensor given as `out` counts as changed in place,
so a gradient that needs its old values fails; one that requires a gradient is
refused while gradients are recorded, as for torch's own `out` arguments.  It may
share memory with an input only where its function says so.
"""
import ctypes
import os
from typing import NamedTuple, Optional

import torch  # noqa: F401  (the module below links to its libraries)

from . import native as nat

try:
    from . import _cp_ops_torch as _native
except ImportError as e:
    raise ImportError(f"{os.path.join(nat.PKG, '_cp_ops_torch.so')} is not built or does not fit this torch; run "
                      "`python -m tile_dependency_pipelined_amd.build`") from e

ACT_NONE, ACT_GELU_TANH, ACT_RELU, ACT_SILU = 0, 1, 2, 3
ACTS = {"none": ACT_NONE, "gelu_tanh": ACT_GELU_TANH, "relu": ACT_RELU, "silu": ACT_SILU}
OP_LINEAR, OP_LINEAR_BACKWARD, OP_GROUPED_LINEAR, OP_GROUPED_LINEAR_BACKWARD, OP_LAYER_NORM_BACKWARD = range(5)
OP_ROUTE, OP_CLIP_GRAD_NORM, OP_LINEAR_INT4 = 5, 6, 7
MAX_WIDTH = 4194304
MAX_GROUPS = 4096
MAX_ROUTED = 1024
MAX_CHOSEN = 32

# every symbol include/cp_ops.h declares
EXPORTS = ("cp_linear", "cp_linear_backward", "cp_grouped_linear", "cp_grouped_linear_backward", "cp_layer_norm",
           "cp_layer_norm_backward", "cp_route", "cp_route_backward", "cp_dispatch", "cp_combine", "cp_combine_backward",
           "cp_int4_quantize", "cp_int4_bytes", "cp_int4_pack", "cp_linear_int4", "cp_grouped_linear_int4",
           "cp_clip_grad_norm", "cp_ops_workspace", "cp_ops_last_error")

_workspace, _last_error = nat.lib().cp_ops_workspace, nat.lib().cp_ops_last_error
_workspace.restype = ctypes.c_int64
_workspace.argtypes = [ctypes.c_int32] * 2 + [ctypes.c_int64] * 3 + [ctypes.c_int32] * 2
_last_error.restype = ctypes.c_char_p


def _raise(code, where, detail):
    raise nat.CpError(code, where, detail)


_native.set_error(_raise)


def workspace_bytes(op, dtype, M, K, N, E=0, aligned=False):
    """Bytes of scratch memory an operator takes (cp_ops_workspace)."""
    n = _workspace(op, dtype, M, K, N, E, aligned)
    if n < 0:
        _raise(n, "cp_ops_workspace", _last_error().decode())
    return n


def linear(x, w, bias=None, residual=None, act=ACT_NONE, need_pre=False, out=None):
    """act(x w + bias) + residual: x [M][K], w [K][N], bias [N], residual [M][N].
    With need_pre returns (y, x w + bias), the second for linear_backward.  `out`
    may be the residual itself."""
    return _native.linear(x, w, bias, residual, act, need_pre, out)


def linear_backward(dy, x, w, pre=None, act=ACT_NONE, need_x=True, need_w=True, need_bias=True):
    """Gradients (dx, dw, db) of linear for dy [M][N]; None for those not asked
    for.  `pre` is what linear returned with need_pre (not needed without an
    activation).  The residual's gradient is dy."""
    return _native.linear_backward(dy, x, w, pre, act, need_x, need_w, need_bias)


def grouped_linear(x, w, offsets, bias=None, act=ACT_NONE, need_pre=False, out=None):
    """act(x_t w_e + bias_e) for rows sorted by expert: x [T][K], w [E][K][N],
    bias [E][N]; expert e has rows offsets[e] .. offsets[e + 1] - 1 (int32, on
    the device, never read by the host).  Rows from offsets[E] on give zeros."""
    return _native.grouped_linear(x, w, offsets, bias, act, need_pre, out)


def grouped_linear_backward(dy, x, w, offsets, pre=None, act=ACT_NONE, need_x=True, need_w=True, need_bias=True):
    """Gradients (dx, dw, db) of grouped_linear for dy [T][N]; zeros for experts
    without rows and for rows without an expert."""
    return _native.grouped_linear_backward(dy, x, w, offsets, pre, act, need_x, need_w, need_bias)


def layer_norm(x, weight=None, bias=None, eps=1e-5, out=None):
    """(y, mean, rstd) with y = (x - mean) rstd weight + bias over the rows of
    x [M][N]; mean and rstd are float32 [M].  `out` may be x."""
    return _native.layer_norm(x, weight, bias, eps, out)


def layer_norm_backward(dy, x, mean, rstd, weight=None, need_x=True, need_weight=True, need_bias=True):
    """Gradients (dx, dweight, dbias) of layer_norm for dy [M][N], from the mean
    and rstd it returned; None for those not asked for."""
    return _native.layer_norm_backward(dy, x, mean, rstd, weight, need_x, need_weight, need_bias)


class Routing(NamedTuple):
    """What route returns, for T tokens, E experts and k slots to a token.  The int32
    tensors share an allocation, gates and slopes another; the loss has its own."""
    experts: torch.Tensor  # int32 [T][k], largest logit first; -1: no expert
    gates: torch.Tensor    # float32 [T][k]; 0 without an expert
    rows: torch.Tensor     # int32 [T][k]: the slot's row in expert order; -1 without an expert
    counts: torch.Tensor   # int32 [E]: slots of each expert
    offsets: torch.Tensor  # int32 [E + 1]: where each expert's rows begin
    loss: torch.Tensor     # float32 []: the balance loss
    slopes: torch.Tensor   # float32 [E]: its derivative by any token's probability of an expert


def route(logits, k, normalize=False, valid=None):
    """The k experts with the largest of each token's logits [T][E], the lower
    index first among equals, as a Routing.  Gates are their softmax
    probabilities, with `normalize` divided by their sum.  A logit of -inf is
    never chosen; tokens for which `valid` (bool [T]) is False have no expert.
    The loss is E sum_e f_e P_e, f_e the share of the slots and P_e the mean
    probability of expert e over the tokens that have an expert."""
    return Routing._make(_native.route(logits, k, normalize, valid))


def route_backward(dgates, dloss, logits, experts, slopes, normalize=False):
    """Gradient of the logits for dgates (float32 [T][k]) and dloss (float32 [],
    on the device; each may be None), from what route was given and gave (a token's
    experts are different).  The counts are constants; tokens without an expert get
    zeros."""
    return _native.route_backward(dgates, dloss, logits, experts, slopes, normalize)


def dispatch(x, rows, offsets, out=None):
    """Rows of x [T][D] in expert order, [T k][D]: row rows[t][j] is x[t].  Rows
    from offsets[E] on are zero.  Its gradient is combine(d, rows)."""
    return _native.dispatch(x, rows, offsets, out)


def combine(y, rows, gates=None, residual=None, out=None):
    """sum_j gates[t][j] y[rows[t][j]] + residual[t]: y [T k][D] in expert order,
    gates float32 [T][k] (None: ones).  `out` may be the residual itself."""
    return _native.combine(y, rows, gates, residual, out)


def combine_backward(dout, y, rows, offsets, gates=None, need_y=True, need_gates=True):
    """Gradients (dy, dgates) of combine for dout [T][D]; None for those not asked
    for.  Rows of dy from offsets[E] on are zero.  The residual's is dout.  With other
    numbers of tokens dgates may be added up in another order."""
    return _native.combine_backward(dout, y, rows, offsets, gates, need_y, need_gates)


class Int4Weight(NamedTuple):
    """A weight [K][N] (or [E][K][N]) of 4-bit codes, as linear_int4 reads it."""
    data: torch.Tensor    # uint8: codes, scales and zero points, laid out by pack_int4
    shape: tuple
    group_size: int
    dtype: torch.dtype    # of the scales, and of the rows it is multiplied with

    def to(self, device):
        """The same on another device."""
        return self._replace(data=self.data.to(device))


def quantize_int4(w, group_size=128, symmetric=False):
    """4-bit codes of a finite weight [K][N] or [E][K][N] (any strides): (codes uint8,
    scales, zeros) with w ~ scale (code - zero), a scale and a zero point to each
    column's group_size consecutive k.  Symmetric: zeros None, which stands for 8."""
    return _native.quantize_int4(w, group_size, symmetric)


def pack_int4(codes, scales, zeros: Optional[torch.Tensor] = None, group_size=128):
    """Lays out codes (uint8 [K][N] or [E][K][N], 0 .. 15), scales (float32 or
    bfloat16, [ceil(K / group_size)][N] per expert) and zero points (uint8, 0 .. 15,
    shaped like the scales; None: 8) for linear_int4, once.  group_size is 32, 64 or
    a multiple of 128."""
    data = _native.pack_int4(codes, scales, zeros, group_size)
    return Int4Weight(data, tuple(codes.shape), group_size, scales.dtype)


def _check_int4(x, w, dims):
    if not isinstance(w, Int4Weight):
        raise TypeError("w must be an Int4Weight (pack_int4)")
    if len(w.shape) != dims:
        raise ValueError(f"w must have {dims} dimensions, got {w.shape}")
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a device tensor")
    if x.dtype != w.dtype or x.dim() != 2 or x.shape[1] != w.shape[-2]:
        raise ValueError(f"x must be {w.dtype} with rows of {w.shape[-2]}, got {x.dtype} {tuple(x.shape)}")


def linear_int4(x, w, bias=None, residual=None, act=ACT_NONE, out=None):
    """linear with a 4-bit weight (an Int4Weight [K][N]), for decoding and short
    prompts; x of the weight's type, finite.  `out` may be the residual itself."""
    _check_int4(x, w, 2)
    return _native.linear_int4(x, w.data, w.shape[1], w.group_size, bias, residual, act, out)


def grouped_linear_int4(x, w, offsets, bias=None, act=ACT_NONE, out=None):
    """grouped_linear with 4-bit weights (an Int4Weight [E][K][N])."""
    _check_int4(x, w, 3)
    return _native.grouped_linear_int4(x, w.data, w.shape[0], w.shape[2], w.group_size, offsets, bias, act, out)


def grad_norm(gradients):
    """Root of the sum of squares over all the tensors, float32 []; sums in 64 bits."""
    return _native.clip_grad_norm(gradients, float("inf"), None, False)


def clip_grad_norm(gradients, max_norm, out=None):
    """Scales the tensors (float32 and bfloat16, any mix, dense) by min(1, max_norm /
    (norm + 1e-6)) and returns the norm they had.  In place, or into `out`: a
    tensor of the same shape and strides for each, of either type.  Both may be any
    iterable, and are gone through once.  Nothing is read back to the host: a norm that
    is not finite shows in the norm and in the results."""
    return _native.clip_grad_norm(gradients, max_norm, out, True)
