"""Feed-forward operators on torch tensors: linear layers with a fused epilogue,
linear layers grouped by expert, and layer normalisation, each with its
backward pass.

    y = act(x w + b) + residual
    y_t = act(x_t w_e + b_e)            rows sorted by expert
    y = (x - mean) rstd w + b

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
MAX_WIDTH = 4194304
MAX_GROUPS = 4096

# every symbol include/cp_ops.h declares
EXPORTS = ("cp_linear", "cp_linear_backward", "cp_grouped_linear", "cp_grouped_linear_backward", "cp_layer_norm",
           "cp_layer_norm_backward", "cp_ops_workspace", "cp_ops_last_error")

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
