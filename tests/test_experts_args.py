"""Host tests of the C ABI of the router, the rows' way to the experts and back,
4-bit layers and clipping: constants agree with the binding, sizes are host-only,
and bad arguments give the documented codes before anything is launched."""
import ctypes
import re
import os

import pytest

pytest.importorskip("torch")
nat = pytest.importorskip("tile_dependency_pipelined_amd.native",
                          reason="libcpchain.so not built (python -m tile_dependency_pipelined_amd.build)")
from tile_dependency_pipelined_amd import ops  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # a plausible, aligned address that no call below may touch
Q = 1 << 30  # another, far from it
BF16, F32 = nat.CP_BF16, nat.CP_F32
_p, _i, _l, _f = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
lib = nat.lib()
for name, args in (
        ("cp_route", (_i, _l, _i, _i, _i, _p, _l, _p, _p, _p, _p, _p, _p, _p, _p, _p, _l, _p)),
        ("cp_route_backward", (_i, _l, _i, _i, _i, _p, _p, _p, _l, _p, _p, _p, _l, _p)),
        ("cp_dispatch", (_i, _l, _i, _l, _l, _p, _l, _p, _p, _p, _l, _p)),
        ("cp_combine", (_i, _l, _i, _l, _l, _p, _l, _p, _p, _p, _l, _p, _l, _p)),
        ("cp_combine_backward", (_i, _l, _i, _l, _l, _p, _l, _p, _l, _p, _p, _p, _p, _l, _p, _p)),
        ("cp_int4_quantize", (_i, _l, _l, _i, _l, _p, _l, _l, _l, _p, _p, _p, _p)),
        ("cp_int4_pack", (_i, _l, _l, _i, _l, _p, _p, _p, _p, _p)),
        ("cp_linear_int4", (_i, _l, _l, _l, _p, _l, _p, _l, _p, _p, _l, _i, _p, _l, _p, _l, _p)),
        ("cp_grouped_linear_int4", (_i, _l, _l, _l, _i, _p, _l, _p, _l, _p, _p, _i, _p, _l, _p, _l, _p)),
        ("cp_clip_grad_norm", (_l, _p, _p, _p, _f, _p, _p, _p, _p, _l, _p))):
    getattr(lib, name).argtypes = args
lib.cp_int4_bytes.argtypes = (_i, _l, _l, _i, _l)
lib.cp_int4_bytes.restype = _l


def refused(rc, code):
    assert rc == getattr(nat, "CP_ERR_" + code), rc
    assert lib.cp_ops_last_error()


def test_constants():
    src = open(os.path.join(ROOT, "include", "cp_ops.h")).read()
    for c, v in (("CP_OP_ROUTE", ops.OP_ROUTE), ("CP_OP_CLIP_GRAD_NORM", ops.OP_CLIP_GRAD_NORM),
                 ("CP_OP_LINEAR_INT4", ops.OP_LINEAR_INT4),
                 ("CP_OPS_MAX_ROUTED", ops.MAX_ROUTED), ("CP_OPS_MAX_CHOSEN", ops.MAX_CHOSEN)):
        m = re.search(rf"#define\s+{c}\s+(\d+)", src)
        assert m and int(m.group(1)) == v, c


def test_sizes():
    for T in (0, 1, 64, 1000, 1 << 20, 1 << 30):
        assert ops.workspace_bytes(ops.OP_ROUTE, BF16, T, 0, 100) <= 256 * (2 * 100 + 1) * 4 + 256
    assert ops.workspace_bytes(ops.OP_CLIP_GRAD_NORM, BF16, 1000, 0, 0) > 0
    assert lib.cp_int4_bytes(BF16, 128, 16, 1, 128) == 1024 + 64
    assert lib.cp_int4_bytes(BF16, 129, 17, 3, 64) == 3 * (4 * 1024 + 2 * 3 * 16 * 4)
    assert lib.cp_int4_bytes(F32, 0, 5, 1, 32) == 0
    for args in ((7, 8, 8, 1, 32), (BF16, -1, 8, 1, 32), (BF16, 8, ops.MAX_WIDTH + 1, 1, 32), (BF16, 8, 8, 0, 32),
                 (BF16, 8, 8, ops.MAX_GROUPS + 1, 32), (BF16, 8, 8, 1, 0), (BF16, 8, 8, 1, 16), (BF16, 8, 8, 1, 96),
                 (BF16, 8, 8, 1, -128), (BF16, 8, 8, 1, 192)):
        assert lib.cp_int4_bytes(*args) < 0


def route(dtype=BF16, T=4, E=8, k=2, logits=P, ld=8, experts=P, gates=P, rows=P, counts=P, offsets=P, loss=P, slopes=P, ws=P,
          n=1 << 30):
    return lib.cp_route(dtype, T, E, k, 0, logits, ld, None, experts, gates, rows, counts, offsets, loss, slopes, ws, n, None)


@pytest.mark.parametrize("change, code", [
    (dict(dtype=5), "UNSUPPORTED"), (dict(E=0), "SHAPE"), (dict(E=1025), "SHAPE"), (dict(k=0), "SHAPE"), (dict(k=9), "SHAPE"),
    (dict(E=64, k=33, ld=64), "SHAPE"), (dict(T=-1), "SHAPE"), (dict(T=(1 << 29) + 1), "SHAPE"), (dict(logits=None), "INVALID_ARG"),
    (dict(logits=P + 1), "INVALID_ARG"), (dict(ld=7), "SHAPE"), (dict(experts=None), "INVALID_ARG"),
    (dict(gates=P + 2), "INVALID_ARG"), (dict(rows=None), "INVALID_ARG"), (dict(counts=None), "INVALID_ARG"),
    (dict(offsets=P + 1), "INVALID_ARG"), (dict(loss=None), "INVALID_ARG"), (dict(slopes=None), "INVALID_ARG"),
    (dict(T=100000, ws=None), "INVALID_ARG"), (dict(T=100000, n=64), "INVALID_ARG"), (dict(T=100000, ws=P + 4), "INVALID_ARG"),
])
def test_route_refusals(change, code):
    refused(route(**change), code)


def test_route_backward_refusals():
    def call(T=4, E=8, k=2, dg=P, dl=P, x=P, ld=8, experts=P, slopes=P, d=Q, ldd=8):
        return lib.cp_route_backward(BF16, T, E, k, 0, dg, dl, x, ld, experts, slopes, d, ldd, None)
    for change, code in ((dict(E=2000), "SHAPE"), (dict(k=9), "SHAPE"), (dict(x=None), "INVALID_ARG"), (dict(d=None), "INVALID_ARG"),
                         (dict(ldd=3), "SHAPE"), (dict(experts=None), "INVALID_ARG"), (dict(slopes=None), "INVALID_ARG"),
                         (dict(dg=P + 1), "INVALID_ARG"), (dict(dl=P + 1), "INVALID_ARG"), (dict(d=P + 8), "INVALID_ARG"),
                         (dict(d=P, ldd=16), "INVALID_ARG")):
        refused(call(**change), code)
    assert call(T=0, x=None, d=None, experts=None) == nat.CP_OK


def test_exchange_refusals():
    def dispatch(dtype=BF16, T=4, k=2, R=8, D=8, x=P, ldx=8, rows=P, end=P, out=Q, ldo=8):
        return lib.cp_dispatch(dtype, T, k, R, D, x, ldx, rows, end, out, ldo, None)
    for change, code in ((dict(dtype=3), "UNSUPPORTED"), (dict(k=0), "SHAPE"), (dict(k=33), "SHAPE"), (dict(T=1 << 30), "SHAPE"),
                         (dict(R=-1), "SHAPE"), (dict(R=(1 << 30) + 1), "SHAPE"), (dict(D=ops.MAX_WIDTH + 1), "SHAPE"),
                         (dict(x=None), "INVALID_ARG"), (dict(x=P + 1), "INVALID_ARG"), (dict(ldx=7), "SHAPE"),
                         (dict(rows=None), "INVALID_ARG"), (dict(end=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"),
                         (dict(out=P + 16), "INVALID_ARG"), (dict(ldo=4), "SHAPE")):
        refused(dispatch(**change), code)
    assert dispatch(T=0, R=0, x=None, rows=None, end=None, out=None) == nat.CP_OK
    assert dispatch(D=0, x=None, out=None) == nat.CP_OK

    def combine(y=P, ldy=8, rows=P, gates=P, res=None, ldr=8, out=Q, ldo=8, T=4):
        return lib.cp_combine(F32, T, 2, 8, 8, y, ldy, rows, gates, res, ldr, out, ldo, None)
    for change, code in ((dict(y=None), "INVALID_ARG"), (dict(ldy=1), "SHAPE"), (dict(rows=P + 2), "INVALID_ARG"),
                         (dict(gates=P + 2), "INVALID_ARG"), (dict(res=Q, ldr=16), "INVALID_ARG"), (dict(res=Q + 32), "INVALID_ARG"),
                         (dict(out=P + 32), "INVALID_ARG"), (dict(ldr=2, res=P), "SHAPE")):
        refused(combine(**change), code)
    assert combine(T=0, rows=None, out=None) == nat.CP_OK

    def backward(d=P, y=P, rows=P, end=P, dy=Q, lddy=8, dg=P):
        return lib.cp_combine_backward(F32, 4, 2, 8, 8, d, 8, y, 8, rows, end, None, dy, lddy, dg, None)
    for change, code in ((dict(d=None), "INVALID_ARG"), (dict(y=None), "INVALID_ARG"), (dict(end=None), "INVALID_ARG"),
                         (dict(dy=P), "INVALID_ARG"), (dict(lddy=7), "SHAPE"), (dict(dg=P + 2), "INVALID_ARG")):
        refused(backward(**change), code)
    assert backward(dy=None, dg=None, y=None, end=None) == nat.CP_OK


def test_int4_refusals():
    def call(dtype=BF16, M=4, K=64, N=8, X=P, ldx=64, w=Q, group=32, bias=None, R=None, ldr=8, act=0, Y=P << 2, ldy=8, ws=P, n=1 << 50):
        return lib.cp_linear_int4(dtype, M, K, N, X, ldx, w, group, bias, R, ldr, act, Y, ldy, ws, n, None)
    for change, code in ((dict(dtype=2), "UNSUPPORTED"), (dict(group=48), "UNSUPPORTED"), (dict(act=4), "UNSUPPORTED"),
                         (dict(M=-1), "SHAPE"), (dict(K=ops.MAX_WIDTH + 1), "SHAPE"), (dict(X=None), "INVALID_ARG"),
                         (dict(ldx=63), "SHAPE"), (dict(w=None), "INVALID_ARG"), (dict(w=Q + 8), "INVALID_ARG"),
                         (dict(bias=P + 1), "INVALID_ARG"), (dict(Y=Q + 64), "INVALID_ARG"), (dict(Y=P), "INVALID_ARG"),
                         (dict(ldy=7), "SHAPE"), (dict(K=9000, ldx=9000, ws=None), "INVALID_ARG"),
                         (dict(K=9000, ldx=9000, ws=P, n=64), "INVALID_ARG"), (dict(R=(P << 2) + 8), "INVALID_ARG"),
                         (dict(M=1 << 30, N=ops.MAX_WIDTH, ldy=ops.MAX_WIDTH, Y=1 << 60), "SHAPE")):
        refused(call(**change), code)
    assert call(M=0, X=None, Y=None, w=None) == nat.CP_OK

    def grouped(E=2, off=P, Y=P << 2):
        return lib.cp_grouped_linear_int4(BF16, 4, 64, 8, E, P, 64, Q, 32, off, None, 0, Y, 8, None, 0, None)
    for change, code in ((dict(E=0), "SHAPE"), (dict(E=-1), "SHAPE"), (dict(E=ops.MAX_GROUPS + 1), "SHAPE"),
                         (dict(off=None), "INVALID_ARG"), (dict(off=P + 2), "INVALID_ARG")):
        refused(grouped(**change), code)
    assert lib.cp_int4_pack(BF16, 64, 8, 1, 32, P, P, None, Q + 4, None) == nat.CP_ERR_INVALID_ARG
    assert lib.cp_int4_pack(BF16, 64, 8, 1, 32, None, P, None, Q, None) == nat.CP_ERR_INVALID_ARG
    assert lib.cp_int4_pack(BF16, 64, 8, 1, 32, Q + 16, P, None, Q, None) == nat.CP_ERR_INVALID_ARG
    assert lib.cp_int4_quantize(BF16, 64, 8, 1, 32, P, -8, 1, 0, P, P, None, None) == nat.CP_ERR_SHAPE
    assert lib.cp_int4_quantize(BF16, 64, 8, 1, 32, P + 1, 8, 1, 0, P, P, None, None) == nat.CP_ERR_INVALID_ARG


def test_clip_refusals():
    def call(grads, outs=None, numels=None, types=None, out_types=None, most=1.0, norm=P, ws=P, n=1 << 30):
        k = len(grads)
        ints = lambda v, t=_i: (t * max(k, 1))(*v)  # noqa: E731
        return lib.cp_clip_grad_norm(k, ints(types or [F32] * k), ints(grads, _p), ints(numels or [100] * k, _l), most,
                                     ints(out_types or types or [F32] * k), None if outs is None else ints(outs, _p), norm, ws, n,
                                     None)
    for args, code in (((dict(grads=[P], most=-1.0)), "INVALID_ARG"), (dict(grads=[P], most=float("nan")), "INVALID_ARG"),
                       (dict(grads=[P], norm=None), "INVALID_ARG"), (dict(grads=[P], ws=None), "INVALID_ARG"),
                       (dict(grads=[P], n=8), "INVALID_ARG"), (dict(grads=[None]), "INVALID_ARG"),
                       (dict(grads=[P], types=[4]), "UNSUPPORTED"), (dict(grads=[P], outs=[P], out_types=[4]), "UNSUPPORTED"),
                       (dict(grads=[P], numels=[-1]), "SHAPE"), (dict(grads=[P + 1]), "INVALID_ARG"),
                       (dict(grads=[P], outs=[None]), "INVALID_ARG"), (dict(grads=[P], outs=[P + 4]), "INVALID_ARG"),
                       (dict(grads=[P, P], outs=[P, P]), "INVALID_ARG"), (dict(grads=[P], outs=[P], out_types=[BF16]), "INVALID_ARG"),
                       (dict(grads=[P, P + 400], outs=[Q, P]), "INVALID_ARG"),
                       (dict(grads=[P, P + 396], outs=[P, P + 396]), "INVALID_ARG"),
                       (dict(grads=[Q, P], outs=[P + 396, Q + 4096]), "INVALID_ARG")):
        refused(call(**args), code)
