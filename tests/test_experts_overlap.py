"""Host tests: outputs of the rows' way to the experts and back and of the clipping that
share memory with anything the kernels still read, or with each other, are refused
before a launch."""
import ctypes

import pytest

pytest.importorskip("torch")
nat = pytest.importorskip("tile_dependency_pipelined_amd.native",
                          reason="libcpchain.so not built (python -m tile_dependency_pipelined_amd.build)")
from tile_dependency_pipelined_amd import ops  # noqa: E402,F401

_p, _i, _l, _f = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
lib = nat.lib()
lib.cp_dispatch.argtypes = (_i, _l, _i, _l, _l, _p, _l, _p, _p, _p, _l, _p)
lib.cp_combine_backward.argtypes = (_i, _l, _i, _l, _l, _p, _l, _p, _l, _p, _p, _p, _p, _l, _p, _p)
lib.cp_clip_grad_norm.argtypes = (_l, _p, _p, _p, _f, _p, _p, _p, _p, _l, _p)
A, B, C, D, E, F, G = (n << 20 for n in range(1, 8))     # plausible addresses that no call below may touch


def refused(rc):
    assert rc == nat.CP_ERR_INVALID_ARG, rc
    assert b"overlaps" in lib.cp_ops_last_error()


# 4 tokens, 2 slots each, 8 rows of 8 fp32 elements: an output of 256 bytes, 32 of slots, 4 of the end
def dispatch(x=A, rows=B, end=C, out=D, ldo=8):
    return lib.cp_dispatch(nat.CP_F32, 4, 2, 8, 8, x, 8, rows, end, out, ldo, None)


@pytest.mark.parametrize("change", [dict(end=D), dict(end=D + 252), dict(end=D + 4 * 10 * 7 + 28, ldo=10), dict(rows=D + 252),
                                    dict(rows=D - 28), dict(x=D + 252)], ids=str)
def test_dispatch(change):
    refused(dispatch(**change))


def backward(dout=A, y=B, rows=C, end=D, gates=E, dy=F, dgates=G):
    return lib.cp_combine_backward(nat.CP_F32, 4, 2, 8, 8, dout, 8, y, 8, rows, end, gates, dy, 8, dgates, None)


@pytest.mark.parametrize("change", [
    dict(dy=A), dict(dy=B + 252), dict(rows=F), dict(end=F + 252), dict(gates=F + 252), dict(gates=F - 28), dict(dgates=F + 252),
    dict(dgates=A + 124), dict(dgates=B), dict(dgates=B + 252), dict(dgates=C), dict(dgates=E), dict(dgates=E + 28), dict(dgates=D - 28),
    dict(dgates=A + 124, dy=None), dict(dgates=C + 28, dy=None, end=None)], ids=str)
def test_combine_backward(change):
    refused(backward(**change))


def test_empty_outputs_are_not_refused():
    """Where there is nothing to write, nothing is shared (and nothing launched)."""
    assert lib.cp_dispatch(nat.CP_F32, 4, 2, 8, 0, A, 8, B, A, A, 8, None) == nat.CP_OK
    assert lib.cp_combine_backward(nat.CP_F32, 0, 2, 8, 0, A, 8, A, 8, A, A, A, A, 8, A, None) == nat.CP_OK
    assert lib.cp_combine_backward(nat.CP_F32, 4, 2, 8, 8, A, 8, None, 8, A, None, A, None, 8, None, None) == nat.CP_OK


@pytest.mark.parametrize("norm, outs", [(A, (C, D)), (A + 396, (C, D)), (B + 196, (C, D)), (C + 396, (C, D)), (D + 4, (C, D)),
                                        (B, (A, B)), (A, None), (B + 196, None)], ids=str)
def test_norm(norm, outs):
    """A gradient of 100 fp32 elements, one of 100 in bf16."""
    types = (_i * 2)(nat.CP_F32, nat.CP_BF16)
    refused(lib.cp_clip_grad_norm(2, types, (_p * 2)(A, B), (_l * 2)(100, 100), 1.0, types, None if outs is None else (_p * 2)(*outs),
                                  norm, E, 1 << 20, None))
