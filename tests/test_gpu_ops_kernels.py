"""GPU tests of every kernel of the linear layers (the calls in ops_kernels.py) and
of the norm's backward pass in place, through the C entry points: rows that are
longer than the matrix, scratch memory of exactly the size asked for, and nothing
written but the outputs.

Inputs lie in buffers filled with NaN, so do the rows without an expert and what
belongs to an idle expert: none of that may reach a result.  Tolerances are those of
test_gpu_ops.py; the formulas are computed on the device in 64 bits.  A second
run has to give the same bits."""
import ctypes
import math
import sys

import pytest
from ops_kernels import CASES

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

E32 = 2.0 ** -24
U = {1: 2.0 ** -8, 0: 2.0 ** -24}
DTYPES = {1: torch.bfloat16, 0: torch.float32}
ACTS = ("none", "gelu_tanh", "relu", "silu")
vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


@pytest.fixture(scope="module")
def lib():
    from tile_dependency_pipelined_amd import ops
    from tile_dependency_pipelined_amd import native as nat
    assert torch.cuda.is_available()
    f, m = nat.lib(), (vp, i64)
    f.cp_linear.argtypes = (i32, i64, i64, i64, *m, *m, i32, vp, *m, i32, *m, *m, *m, vp)
    f.cp_grouped_linear.argtypes = (i32, i64, i64, i64, i32, *m, *m, i64, i32, vp, vp, i32, *m, *m, *m, vp)
    f.cp_linear_backward.argtypes = (i32, i64, i64, i64, *m, *m, *m, i32, *m, i32, *m, *m, vp, *m, vp)
    f.cp_grouped_linear_backward.argtypes = (i32, i64, i64, i64, i32, *m, *m, *m, i64, i32, vp, *m, i32, *m, *m, i64, vp, *m, vp)
    f.cp_layer_norm_backward.argtypes = (i32, i64, i64, *m, *m, vp, vp, vp, *m, vp, vp, *m, vp)
    return f, ops


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def stream():
    return torch.cuda.current_stream().cuda_stream


class Box:
    """A matrix (or a stack of them) `shift` elements into a buffer of `fill`, `pad` elements between its rows."""

    def __init__(self, shape, dtype, pad=8, shift=8, fill=float("nan")):
        self.ld = max(shape[-1], 1) + pad
        self.stride = self.ld * shape[-2] + pad
        n = self.stride * (shape[0] if len(shape) == 3 else 1)
        self.fill = fill
        self.buf = torch.full((shift + n + 64,), fill, dtype=dtype, device="cuda")
        strides = (self.stride, self.ld, 1)[3 - len(shape):]
        self.t = self.buf.as_strided(shape, strides, shift)

    @property
    def p(self):
        return self.t.data_ptr()

    def inside_only(self):
        """Nothing but the matrix was written (its values are lost)."""
        self.t.fill_(self.fill)
        return bool((self.buf == self.fill).all())


def scratch(ops, op, dtype, M, K, N, E, aligned):
    n = ops.workspace_bytes(op, dtype, M, K, N, E, aligned)
    buf = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    return buf, n


def randn(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def act(z, a):
    if a == 1:
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if a == 2:
        return z.clamp(min=0)
    return z * torch.sigmoid(z) if a == 3 else z


def act_grad(z, a):
    if a == 2:  # (zero at zero)
        return (z > 0).double()
    z = z.clone().requires_grad_(True)
    act(z, a).sum().backward()
    return z.grad


def close(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {got[i].item()} "
                             f"want {want[i].item()} tol {tol[i].item()}")


def offsets(M, E):
    """Rows of E experts: one idle, the last rows of several filling less than half a tile of 256, some rows
    without an expert."""
    if M < 8:
        return [0] * (E - 1) + [max(M - 1, 1), max(M - 1, 1)] if E > 1 else [0, M]
    a = M * 2 // 5 // 256 * 256 + 88 if M >= 700 else M * 2 // 5
    last = M - min(10, M // 8)
    if E == 2:
        return [0, a, last]
    b = a + (M // 3 // 256 * 256 + 20 if M >= 1500 else M // 4)
    return [0, a, a, b, b + (last - b) // 2, last]


def values(case):
    """Inputs as boxes, and the spans of rows with their experts."""
    op, dtype, M, K, N, E, wt, a, parts, aligned = case[:10]
    g = torch.Generator(device="cuda").manual_seed(M + K + N)
    d, shift = DTYPES[dtype], 8 if aligned else 1
    spans = [(0, M, 0)]
    off = None
    if E:
        off = offsets(M, E)
        assert len(off) == E + 1 and off == sorted(off) and off[-1] <= M
        spans = [(off[e], off[e + 1], e) for e in range(E)]

    def box(*shape, std=1.0):
        b = Box(shape, d, 8, shift)
        if len(shape) == 3:
            for e in range(shape[0]):
                if spans[e][0] < spans[e][1]:  # (an idle expert's stay NaN)
                    b.t[e].copy_(randn(g, *shape[1:], std=std))
        else:
            n = off[-1] if E else shape[0]
            b.t[:n].copy_(randn(g, n, shape[1], std=std))
        return b
    return g, d, shift, off, spans, box


@pytest.mark.parametrize("case", [c for c in CASES if c[0] == "forward"], ids=lambda c: "-".join(map(str, c[:10])))
def test_forward(lib, case):
    f, ops = lib
    op, dtype, M, K, N, E, wt, a, parts, aligned = case[:10]
    i = CASES.index(case)
    a = (1, 3, 2, 0)[i % 4]
    say("forward", case, "act", a)
    g, d, shift, off, spans, box = values(case)
    lead = (E,) if E else ()
    x, w = box(M, K), box(*lead, *((N, K) if wt else (K, N)), std=K ** -0.5)
    has_r, has_b = not E and bool(parts & 1), bool(parts & 4)
    r = box(M, N) if has_r else None
    b = None
    if has_b:
        b = torch.full((max(E, 1) * N + 8,), float("nan"), dtype=d, device="cuda")[8 - shift % 8:]
        b = b[:max(E, 1) * N].view(max(E, 1), N)
        for s, t, e in spans:
            if s < t:
                b[e] = randn(g, N).to(d)
    doff = torch.tensor(off, dtype=torch.int32, device="cuda") if E else None
    ws, n = scratch(ops, ops.OP_GROUPED_LINEAR if E else ops.OP_LINEAR, dtype, M, K, N, E, aligned)
    # every third with results off 16 bytes: the epilogue by single elements
    outs = [(Box((M, N), d, 8, shift if i % 3 else 3, 7.0), Box((M, N), d, 8, shift if i % 3 else 3, 7.0)) for _ in range(2)]
    for y, pre in outs:
        bias = b.data_ptr() if has_b else None
        if E:
            rc = f.cp_grouped_linear(dtype, M, K, N, E, x.p, x.ld, w.p, w.ld, w.stride, wt, doff.data_ptr(), bias, a, y.p, y.ld,
                                     pre.p, pre.ld, ws.data_ptr(), n, stream())
        else:
            rc = f.cp_linear(dtype, M, K, N, x.p, x.ld, w.p, w.ld, wt, bias, r.p if r else None, r.ld if r else 0, a, y.p,
                             y.ld, pre.p, pre.ld, ws.data_ptr(), n, stream())
        assert rc == 0, f.cp_ops_last_error()
    assert bool((ws[n:] == 0xA5).all()), "wrote past the scratch memory"
    (y, pre), (y2, pre2) = outs
    assert torch.equal(y.t, y2.t) and torch.equal(pre.t, pre2.t), "not the same bits"
    for s, t, e in spans:
        if s == t:
            continue
        xd, wd = x.t[s:t].double(), (w.t[e] if E else w.t).double()
        wd = wd.t() if wt else wd
        z = xd @ wd
        size = xd.abs() @ wd.abs()
        if has_b:
            z, size = z + b[e].double(), size + b[e].double().abs()
        want = act(z, a)
        zt = (K + 8) * E32 * size
        ty = 1.2 * zt + (0 if a == 0 else 2.0 ** -20 * (1 + z.abs()))
        if has_r:
            want, ty = want + r.t.double(), ty + 4 * E32 * r.t.double().abs()
        close(pre.t[s:t], z, zt + 1.01 * U[dtype] * z.abs(), f"pre {e}")
        close(y.t[s:t], want, ty + (1.01 * U[dtype] + 4 * E32) * want.abs(), f"y {e}")
    if E:
        assert not y.t[off[-1]:].any() and not pre.t[off[-1]:].any(), "rows without an expert"
    assert y.inside_only() and pre.inside_only() and y2.inside_only() and pre2.inside_only(), "wrote outside"


@pytest.mark.parametrize("case", [c for c in CASES if c[0] == "backward"], ids=lambda c: "-".join(map(str, c[:10])))
def test_backward(lib, case):
    f, ops = lib
    op, dtype, M, K, N, E, wt, a, parts, aligned = case[:10]
    i = CASES.index(case)
    if a:
        a = (1, 3, 2)[i % 3]
    say("backward", case, "act", a)
    g, d, shift, off, spans, box = values(case)
    lead = (E,) if E else ()
    dy, x, w = box(M, N), box(M, K), box(*lead, *((N, K) if wt else (K, N)), std=N ** -0.5)
    pre = box(M, N, std=2.0)
    doff = torch.tensor(off, dtype=torch.int32, device="cuda") if E else None
    ws, n = scratch(ops, ops.OP_GROUPED_LINEAR_BACKWARD if E else ops.OP_LINEAR_BACKWARD, dtype, M, K, N, E, aligned)
    so = shift if i % 3 else 3
    need_x, need_w, need_b = bool(parts & 1), bool(parts & 2), bool(parts & 4)
    runs = []
    for _ in range(2):
        dx, dw = Box((M, K), d, 8, so, 7.0), Box((*lead, *((N, K) if wt else (K, N))), d, 8, so, 7.0)
        db = Box((max(E, 1), N), d, 0, so, 7.0)
        px, pw, pb = dx.p if need_x else None, dw.p if need_w else None, db.p if need_b else None
        if E:
            rc = f.cp_grouped_linear_backward(dtype, M, K, N, E, dy.p, dy.ld, x.p, x.ld, w.p, w.ld, w.stride, wt, doff.data_ptr(),
                                              pre.p, pre.ld, a, px, dx.ld, pw, dw.ld, dw.stride, pb, ws.data_ptr(), n, stream())
        else:
            rc = f.cp_linear_backward(dtype, M, K, N, dy.p, dy.ld, x.p, x.ld, w.p, w.ld, wt, pre.p, pre.ld, a, px, dx.ld, pw,
                                      dw.ld, pb, ws.data_ptr(), n, stream())
        assert rc == 0, f.cp_ops_last_error()
        runs.append((dx, dw, db))
    assert bool((ws[n:] == 0xA5).all()), "wrote past the scratch memory"
    assert all(torch.equal(p.t, q.t) for p, q in zip(*runs)), "not the same bits"
    dx, dw, db = runs[0]
    u = 1.01 * U[dtype]
    ut = U[1] if a and dtype == 1 else 0.0  # dZ rounded for the products
    for s, t, e in spans:
        if s == t:
            if need_w:
                assert not dw.t[e].any(), "idle expert's weight"
            if need_b:
                assert not db.t[e].any(), "idle expert's bias"
            continue
        yd, xd, wd, zd = dy.t[s:t].double(), x.t[s:t].double(), (w.t[e] if E else w.t).double(), pre.t[s:t].double()
        wd = wd.t() if wt else wd
        dz = yd * act_grad(zd, a) if a else yd
        zt = yd.abs() * 2.0 ** -20 * (1 + zd.abs()) if a else torch.zeros_like(yd)
        et = zt + (ut + 2 * E32) * dz.abs()
        if need_x:
            want = dz @ wd.t()
            close(dx.t[s:t], want, (et + (N + 8) * E32 * dz.abs()) @ wd.abs().t() + u * want.abs(), f"dx {e}")
        if need_w:
            want = xd.t() @ dz
            tol = xd.abs().t() @ (et + (t - s + 8) * E32 * dz.abs()) + u * want.abs()
            got = dw.t[e] if E else dw.t
            close(got.t() if wt else got, want, tol, f"dw {e}")
        if need_b:
            want = dz.sum(0)
            tol = (zt + (t - s + 10) * E32 * dz.abs()).sum(0) + u * want.abs()
            close(db.t[e], want, tol, f"db {e}")
    if E and need_x:
        assert not dx.t[off[-1]:].any(), "rows without an expert"
    for dx, dw, db in runs:
        assert dx.inside_only() and dw.inside_only() and db.inside_only(), "wrote outside"


# Rows held in registers by waves and by blocks, one and several to a block, and
# rows that are not (8192 elements in fp32 or unaligned, 16384 else, are the longest).
@pytest.mark.parametrize("dtype", [1, 0])
@pytest.mark.parametrize("aligned", [1, 0])
@pytest.mark.parametrize("M, N", [(1, 8), (3, 504), (40, 512), (700, 1000), (300, 4096), (1, 8192), (300, 8192), (5, 8200),
                                  (300, 12288), (9, 16384), (7, 16392), (270, 20008)])
def test_norm_backward_in_place(lib, M, N, aligned, dtype):
    f, ops = lib
    say("norm backward in place", M, N, aligned, dtype)
    g = torch.Generator(device="cuda").manual_seed(M + N)
    d, shift = DTYPES[dtype], 8 if aligned else 1
    x0, dy0 = randn(g, M, N).to(d), randn(g, M, N).to(d)
    w = Box((1, N), d, 0, shift)
    w.t.copy_(randn(g, 1, N))
    mean, rstd = randn(g, M), randn(g, M).abs() + 0.5
    buf, n = scratch(ops, ops.OP_LAYER_NORM_BACKWARD, dtype, M, 0, N, 0, 1)
    results = []
    for where in ("apart", "dy", "x", "apart"):
        x, dy = Box((M, N), d, 8, shift, 7.0), Box((M, N), d, 8, shift, 7.0)
        x.t.copy_(x0)
        dy.t.copy_(dy0)
        dx = {"dy": dy, "x": x}.get(where) or Box((M, N), d, 8, shift, 7.0)
        dw, db = Box((1, N), d, 0, 3, 7.0), Box((1, N), d, 0, 3, 7.0)
        rc = f.cp_layer_norm_backward(dtype, M, N, dy.p, dy.ld, x.p, x.ld, mean.data_ptr(), rstd.data_ptr(), w.p, dx.p, dx.ld,
                                      dw.p, db.p, buf.data_ptr(), n, stream())
        assert rc == 0, f.cp_ops_last_error()
        results.append([t.t.clone() for t in (dx, dw, db)])
        for t, was in ((x, x0), (dy, dy0)):
            assert t is dx or torch.equal(t.t, was)
            assert t.inside_only()
        assert dx.inside_only() and dw.inside_only() and db.inside_only(), "wrote outside"
    assert bool((buf[n:] == 0xA5).all()), "wrote past the scratch memory"
    for r in results[1:]:
        assert all(torch.equal(p, q) for p, q in zip(r, results[0]))
    xh = (x0.double() - mean.double()[:, None]) * rstd.double()[:, None]
    gy = dy0.double() * w.t.double()
    s0, s1 = gy.mean(1, keepdim=True), (gy * xh).mean(1, keepdim=True)
    want = rstd.double()[:, None] * (gy - s0 - xh * s1)
    n_, r = (N + 16) * E32, rstd.double()[:, None]
    txh = 4 * E32 * ((x0.double().abs() + mean.double().abs()[:, None]) * r)
    ts0, ts1 = n_ * gy.abs().mean(1, keepdim=True), (n_ * (gy * xh).abs() + gy.abs() * txh).mean(1, keepdim=True)
    size = gy.abs() + gy.abs().mean(1, keepdim=True) + (xh * s1).abs()
    u = 1.01 * U[dtype]
    close(results[0][0], want, r * (ts0 + xh.abs() * ts1 + txh * s1.abs() + 8 * E32 * size) + u * want.abs(), "dx")
    p = dy0.double() * xh
    want = p.sum(0, keepdim=True)
    close(results[0][1], want, ((M + 16) * E32 * p.abs() + dy0.double().abs() * txh).sum(0, keepdim=True) + u * want.abs(), "dw")
    want = dy0.double().sum(0, keepdim=True)
    close(results[0][2], want, (M + 16) * E32 * dy0.double().abs().sum(0, keepdim=True) + u * want.abs(), "db")


@pytest.mark.parametrize("dtype", [1, 0])
@pytest.mark.parametrize("M", [1, 2, 12, 40, 300])
def test_infinities_in_a_row_of_the_gradient(lib, M, dtype):
    """An infinite dY, pre-activation or X spoils what its row and column enter and nothing else."""
    f, ops = lib
    say("infinities", M, dtype)
    d, K, N, row = DTYPES[dtype], 96, 80, M // 2
    g = torch.Generator(device="cuda").manual_seed(M)
    x, w, dy, pre = (randn(g, *s).to(d) for s in ((M, K), (K, N), (M, N), (M, N)))
    clean = ops.linear_backward(dy, x, w, pre=pre, act=ops.ACT_SILU)
    dy2 = dy.clone()
    dy2[row, 5] = float("inf")
    dx, dw, db = ops.linear_backward(dy2, x, w, pre=pre, act=ops.ACT_SILU)
    assert not dx[row].isfinite().any()
    keep, cols = [m for m in range(M) if m != row], [c for c in range(N) if c != 5]
    assert torch.equal(dx[keep], clean[0][keep])
    assert not dw[:, 5].isfinite().any() and torch.equal(dw[:, cols], clean[1][:, cols])
    assert not db[5].isfinite().any() and torch.equal(db[cols], clean[2][cols])
    # far out the derivative of an activation is 0 or 1, and stays finite
    pre2 = pre.clone()
    pre2[row, 7], pre2[row, 9] = float("inf"), float("-inf")
    one = ops.linear_backward(dy, x, w, pre=pre2, act=ops.ACT_SILU)
    pre2[row, 7], pre2[row, 9] = 200.0, -200.0
    assert all(torch.equal(p, q) for p, q in zip(one, ops.linear_backward(dy, x, w, pre=pre2, act=ops.ACT_SILU)))
    x2 = x.clone()
    x2[row, 3] = float("nan")
    dx, dw, db = ops.linear_backward(dy, x2, w, pre=pre, act=ops.ACT_SILU)
    assert torch.equal(dx, clean[0]) and torch.equal(db, clean[2]) and dw[3].isnan().all()
    assert torch.equal(dw[[k for k in range(K) if k != 3]], clean[1][[k for k in range(K) if k != 3]])
