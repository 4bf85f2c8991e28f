"""Host tests of the feed-forward operators' C ABI: every declared symbol is
bound, constants agree with the binding, workspace sizes are host-only, and bad
arguments give the documented codes before anything is launched."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "cp_ops.h")

nat = pytest.importorskip("tile_dependency_pipelined_amd.native",
                          reason="libcpchain.so not built (python -m tile_dependency_pipelined_amd.build)")
from tile_dependency_pipelined_amd import ops  # noqa: E402

_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
_mat, _sizes, _tail = (_vp, _i64), (_i32, _i64, _i64, _i64), (_vp, _i64, _vp)
for _name, _args in (
        ("cp_linear", (*_sizes, *_mat, *_mat, _i32, _vp, *_mat, _i32, *_mat, *_mat, *_tail)),
        ("cp_linear_backward", (*_sizes, *_mat, *_mat, *_mat, _i32, *_mat, _i32, *_mat, *_mat, _vp, *_tail)),
        ("cp_grouped_linear", (*_sizes, _i32, *_mat, *_mat, _i64, _i32, _vp, _vp, _i32, *_mat, *_mat, *_tail)),
        ("cp_layer_norm", (_i32, _i64, _i64, *_mat, _vp, _vp, ctypes.c_float, *_mat, _vp, _vp, _vp)),
        ("cp_layer_norm_backward", (_i32, _i64, _i64, *_mat, *_mat, _vp, _vp, _vp, *_mat, _vp, _vp, *_tail))):
    getattr(nat.lib(), _name).argtypes = _args

P = 1 << 20  # a plausible, aligned address that no call below may touch


def source():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_symbols_bound():
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(cp_\w+)\s*\(", source(), flags=re.M))
    assert names == set(ops.EXPORTS)
    for n in names:
        assert hasattr(nat.lib(), n), n


def test_constants():
    src = source()
    for c, v in (("CP_ACT_RELU", ops.ACT_RELU), ("CP_ACT_SILU", ops.ACT_SILU), ("CP_OP_LINEAR", ops.OP_LINEAR),
                 ("CP_OP_LINEAR_BACKWARD", ops.OP_LINEAR_BACKWARD), ("CP_OP_GROUPED_LINEAR", ops.OP_GROUPED_LINEAR),
                 ("CP_OP_GROUPED_LINEAR_BACKWARD", ops.OP_GROUPED_LINEAR_BACKWARD),
                 ("CP_OP_LAYER_NORM_BACKWARD", ops.OP_LAYER_NORM_BACKWARD), ("CP_OPS_MAX_WIDTH", ops.MAX_WIDTH),
                 ("CP_OPS_MAX_GROUPS", ops.MAX_GROUPS)):
        m = re.search(rf"#define\s+{c}\s+(\d+)", src)
        assert m and int(m.group(1)) == v, c
    assert (ops.ACT_NONE, ops.ACT_GELU_TANH) == (nat.CP_ACT_NONE, nat.CP_ACT_GELU_TANH)


def test_workspace():
    for op in range(5):
        assert ops.workspace_bytes(op, nat.CP_BF16, 0, 0, 0, 1) >= 0
        assert ops.workspace_bytes(op, nat.CP_F32, 1000, 100, 100, 4) >= 0
    for args in ((9, nat.CP_BF16, 1, 1, 1, 1), (ops.OP_LINEAR, 7, 1, 1, 1, 0), (ops.OP_LINEAR, nat.CP_BF16, -1, 1, 1, 0),
                 (ops.OP_GROUPED_LINEAR, nat.CP_BF16, 1, 1, 1, 0),
                 (ops.OP_LINEAR, nat.CP_BF16, 1, 1, ops.MAX_WIDTH + 1, 0)):
        with pytest.raises(nat.CpError):
            ops.workspace_bytes(*args)


def linear(dtype=nat.CP_BF16, M=4, K=8, N=8, X=P, ldx=8, W=P, ldw=8, wt=0, bias=None, R=None, ldr=0, act=0, Y=P, ldy=8,
           pre=None, ldp=0, ws=P, n=1 << 30):
    return nat.lib().cp_linear(dtype, M, K, N, X, ldx, W, ldw, wt, bias, R, ldr, act, Y, ldy, pre, ldp, ws, n, None)


@pytest.mark.parametrize("change, code", [
    (dict(dtype=5), "UNSUPPORTED"), (dict(M=-1), "SHAPE"), (dict(N=ops.MAX_WIDTH + 1), "SHAPE"), (dict(M=1 << 31), "SHAPE"),
    (dict(act=9), "UNSUPPORTED"), (dict(act=-1), "UNSUPPORTED"), (dict(X=None), "INVALID_ARG"),
    (dict(W=None), "INVALID_ARG"), (dict(Y=None), "INVALID_ARG"), (dict(ldx=7), "SHAPE"), (dict(ldw=7), "SHAPE"),
    (dict(ldy=4), "SHAPE"), (dict(ldy=ops.MAX_WIDTH + 8), "SHAPE"), (dict(X=P + 1), "INVALID_ARG"),
    (dict(dtype=nat.CP_F32, W=P + 2), "INVALID_ARG"), (dict(bias=P + 1), "INVALID_ARG"), (dict(R=P, ldr=7), "SHAPE"),
    (dict(pre=P, ldp=1), "SHAPE"),
])
def test_linear_refusals(change, code):
    assert linear(**change) == getattr(nat, "CP_ERR_" + code)
    assert nat.lib().cp_ops_last_error()


def test_workspace_refusals():
    need = ops.workspace_bytes(ops.OP_LINEAR_BACKWARD, nat.CP_BF16, 64, 64, 64, aligned=True)
    assert need > 0

    def call(ws, n):
        return nat.lib().cp_linear_backward(nat.CP_BF16, 64, 64, 64, P, 64, P, 64, P, 64, 0, None, 0, 0, P, 64, P, 64, P,
                                            ws, n, None)
    assert call(None, need) == nat.CP_ERR_INVALID_ARG
    assert call(P, need - 1) == nat.CP_ERR_INVALID_ARG
    assert call(P + 16, need) == nat.CP_ERR_INVALID_ARG


def test_grouped_refusals():
    def call(E=2, off=P, sw=64, K=8, N=8):
        return nat.lib().cp_grouped_linear(nat.CP_BF16, 4, K, N, E, P, K, P, N, sw, 0, off, None, 0, P, N, None, 0, P,
                                           1 << 30, None)
    assert call(E=0) == nat.CP_ERR_SHAPE
    assert call(E=ops.MAX_GROUPS + 1) == nat.CP_ERR_SHAPE
    assert call(off=None) == nat.CP_ERR_INVALID_ARG
    assert call(off=P + 2) == nat.CP_ERR_INVALID_ARG
    assert call(sw=63) == nat.CP_ERR_SHAPE


def test_norm_refusals():
    lib = nat.lib()
    assert lib.cp_layer_norm(nat.CP_BF16, 4, 0, P, 8, None, None, 1e-5, P, 8, None, None, None) == nat.CP_ERR_SHAPE
    assert lib.cp_layer_norm(nat.CP_BF16, 4, 8, P, 8, None, None, -1.0, P, 8, None, None, None) == nat.CP_ERR_INVALID_ARG
    assert lib.cp_layer_norm(nat.CP_BF16, 4, 8, P, 8, None, None, float("nan"), P, 8, None, None,
                             None) == nat.CP_ERR_INVALID_ARG
    assert lib.cp_layer_norm(nat.CP_BF16, 4, 8, None, 8, None, None, 1e-5, P, 8, None, None, None) == nat.CP_ERR_INVALID_ARG
    assert lib.cp_layer_norm_backward(nat.CP_BF16, 4, 8, P, 8, P, 8, None, P, None, P, 8, None, None, P, 1 << 20,
                                      None) == nat.CP_ERR_INVALID_ARG
    assert lib.cp_layer_norm_backward(nat.CP_BF16, 4, 8, P, 8, P, 4, P, P, None, P, 8, None, None, P, 1 << 20,
                                      None) == nat.CP_ERR_SHAPE


def test_empty_calls_need_nothing():
    assert linear(M=0, X=None, Y=None, n=0, ws=None) == nat.CP_OK
    assert linear(N=0, W=None, Y=None, n=0, ws=None) == nat.CP_OK
    assert nat.lib().cp_layer_norm(nat.CP_F32, 0, 8, None, 8, None, None, 0.0, None, 8, None, None, None) == nat.CP_OK


def test_host_tensors_are_refused():
    import torch
    with pytest.raises(TypeError):
        ops.linear(torch.zeros(2, 2), torch.zeros(2, 2))
    with pytest.raises(TypeError):
        ops.layer_norm(torch.zeros(2, 2))
