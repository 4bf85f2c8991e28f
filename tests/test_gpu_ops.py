"""GPU tests of the feed-forward operators against the formulas in 64 bits.

Tolerances are element-wise bounds on the rounding of the stated algorithm.
With u the unit roundoff of the stored type (2^-8 bf16, 2^-24 fp32) and
e = 2^-24 that of the fp32 sums:
  - a sum of K products is off by at most (K + 8) e sum |a||b|;
  - an activation or its derivative has a slope below 1.2 and is itself off by
    at most 2^-20 (1 + |z|): the exponential's argument is rounded, the rest
    is a few operations;
  - bf16 products of dZ use dZ rounded to bf16: u sum |dz||w|;
  - the stored value is rounded once: u |y| (with a factor 1.01 for second order);
  - a row's mean and deviation are sums of N terms, so their relative error is
    below (N + 8) e, and a normalised value's below a small multiple of that.
Inputs sit in larger buffers filled with NaN, outputs in buffers whose
surroundings have to stay as they were."""
import math
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

E32 = 2.0 ** -24
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
C0 = math.sqrt(2 / math.pi)
ACTS = ("none", "gelu_tanh", "relu", "silu")


@pytest.fixture(scope="module")
def ops():
    from tile_dependency_pipelined_amd import ops as o
    assert torch.cuda.is_available()
    return o


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def place(t, dtype, pad=0, shift=0):
    """t on the GPU inside a NaN-filled buffer: `pad` elements after each row, `shift` before the first."""
    ld = t.shape[-1] + pad
    buf = torch.full((shift + max(math.prod(t.shape[:-1]), 1) * ld + 16,), float("nan"), dtype=dtype, device="cuda")
    strides = [1]
    n = ld
    for s in reversed(t.shape[:-1]):
        strides.insert(0, n)
        n *= s
    v = buf.as_strided(t.shape, strides, shift)
    v.copy_(t.to(dtype))
    return v


def data(g, *shape, dtype, std=1.0):
    """Values of the element type, as doubles on the host."""
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * std).to(dtype).double()


def act(z, a):
    if a == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(C0 * (z + 0.044715 * z ** 3)))
    if a == "relu":
        return z.clamp(min=0)
    if a == "silu":
        return z * torch.sigmoid(z)
    return z


def grad(z, a):
    z = z.clone().requires_grad_(True)
    if z.numel() == 0:
        return torch.ones_like(z)
    act(z, a).sum().backward()
    return z.grad


def close(got, want, tol, what):
    got = got.detach().double().cpu()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= tol)
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {got[i]} want {want[i]} "
                             f"tol {tol[i] if torch.is_tensor(tol) else tol}")


def forward_tol(x, w, b, z, y, a, name):
    K = x.shape[1]
    size = x.abs() @ w.abs() + (b.abs() if b is not None else 0)
    zt = (K + 8) * E32 * size
    return 1.2 * zt + (0 if a == "none" else 2.0 ** -20 * (1 + z.abs())) + 1.01 * U[name] * y.abs() + 4 * E32 * y.abs(), \
        zt + 1.01 * U[name] * z.abs()


SIZES = [  # M, K, N: one token to several tiles, whole and ragged, aligned and not
    (1, 8, 8), (1, 1, 1), (1, 256, 512), (1, 1000, 200), (2, 7, 3), (5, 64, 72), (13, 264, 136), (16, 2048, 128),
    (17, 65, 33), (31, 128, 1), (64, 64, 64), (100, 72, 264), (128, 512, 256), (130, 130, 130), (257, 192, 520),
    (300, 1001, 65), (513, 40, 96), (520, 2056, 520), (3, 0, 5), (0, 8, 8), (4, 8, 0),
]


@pytest.mark.parametrize("name", ["bf16", "f32"])
@pytest.mark.parametrize("wt", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_linear(ops, size, wt, name):
    M, K, N = size
    i = SIZES.index(size) + (7 if wt else 0)
    a, has_b, has_r, pad, shift = ACTS[i % 4], i % 3 != 0, i % 2 == 0, (0, 8, 3)[i % 3], (0, 0, 8, 1)[i % 4]
    say(f"linear {size} wt={wt} {name} act={a} pad={pad} shift={shift}")
    g = torch.Generator().manual_seed(i)
    d = dt(name)
    x, w = data(g, M, K, dtype=d), data(g, K, N, dtype=d, std=max(K, 1) ** -0.5)
    b = data(g, N, dtype=d) if has_b else None
    r = data(g, M, N, dtype=d) if has_r else None
    dw = place(w.t().contiguous(), d, pad, shift).t() if wt else place(w, d, pad, shift)
    out = torch.full((M + 2, N + 5), 7.0, dtype=d, device="cuda")
    y, pre = ops.linear(place(x, d, pad, shift), dw, None if b is None else place(b, d, 0, shift),
                        residual=None if r is None else place(r, d, pad, shift), act=ops.ACTS[a], need_pre=True,
                        out=out[1:M + 1, 2:N + 2])
    z = x @ w + (b if has_b else 0)
    want = act(z, a) + (r if has_r else 0)
    ty, tz = forward_tol(x, w, b, z, want, a, name)
    close(y, want, ty + (U[name] * 0 if r is None else 4 * E32 * r.abs()), "y")
    close(pre, z, tz, "pre")
    keep = out.clone()
    keep[1:M + 1, 2:N + 2] = 7.0
    assert bool((keep == 7.0).all()), "wrote outside the output"


@pytest.mark.parametrize("name", ["bf16", "f32"])
@pytest.mark.parametrize("wt", [False, True])
@pytest.mark.parametrize("size", [s for s in SIZES if s != (520, 2056, 520)], ids=lambda s: "x".join(map(str, s)))
def test_linear_backward(ops, size, wt, name):
    M, K, N = size
    i = SIZES.index(size) + (5 if wt else 0)
    a, pad, shift = ACTS[i % 4], (0, 8, 3)[i % 3], (0, 0, 8, 1)[i % 4]
    say(f"linear_backward {size} wt={wt} {name} act={a} pad={pad} shift={shift}")
    g = torch.Generator().manual_seed(100 + i)
    d = dt(name)
    x, w = data(g, M, K, dtype=d), data(g, K, N, dtype=d, std=max(N, 1) ** -0.5)
    dy, pre = data(g, M, N, dtype=d), data(g, M, N, dtype=d, std=2.0)
    dw_in = place(w.t().contiguous(), d, pad, shift).t() if wt else place(w, d, pad, shift)
    dx, dw, db = ops.linear_backward(place(dy, d, pad, shift), place(x, d, pad, shift), dw_in,
                                     pre=None if a == "none" else place(pre, d, pad, shift), act=ops.ACTS[a])
    check_backward(x, w, dy, pre, a, name, dx, dw, db)
    assert (dw.stride(0) == 1 or K <= 1) if wt and N > 1 and K > 1 else True


def check_backward(x, w, dy, pre, a, name, dx, dw, db):
    M, N = dy.shape
    K = w.shape[0]
    gz = grad(pre, a)
    dz = dy * gz
    zt = dy.abs() * 2.0 ** -20 * (1 + pre.abs()) if a != "none" else torch.zeros_like(dy)
    ut = U[name] if a != "none" and name == "bf16" else 0.0     # dZ rounded for the products
    et = zt + (ut + 2 * E32) * dz.abs()
    u = 1.01 * U[name]
    if dx is not None:
        want = dz @ w.t()
        close(dx, want, et @ w.abs().t() + (N + 8) * E32 * (dz.abs() @ w.abs().t()) + u * want.abs(), "dx")
    if dw is not None:
        want = x.t() @ dz
        close(dw, want, x.abs().t() @ et + (M + 8) * E32 * (x.abs().t() @ dz.abs()) + u * want.abs(), "dw")
    if db is not None:
        want = dz.sum(0)
        close(db, want, (zt + 2 * E32 * dz.abs()).sum(0) + (M + 8) * E32 * dz.abs().sum(0) + u * want.abs(), "db")


@pytest.mark.parametrize("need", [(True, False, False), (False, True, False), (False, False, True), (False, False, False)])
def test_linear_backward_subsets(ops, need):
    say(f"linear_backward subset {need}")
    g = torch.Generator().manual_seed(3)
    d = torch.bfloat16
    x, w, dy, pre = (data(g, *s, dtype=d) for s in ((40, 72), (72, 56), (40, 56), (40, 56)))
    out = ops.linear_backward(dy.to("cuda", d), x.to("cuda", d), w.to("cuda", d), pre=pre.to("cuda", d), act=ops.ACT_SILU,
                              need_x=need[0], need_w=need[1], need_bias=need[2])
    assert [o is not None for o in out] == list(need)
    check_backward(x, w, dy, pre, "silu", "bf16", *out)


def test_linear_residual_in_place_and_repeatable(ops):
    say("linear with out = residual")
    g = torch.Generator().manual_seed(5)
    d = torch.bfloat16
    x, w, r = (data(g, *s, dtype=d).to("cuda", d) for s in ((200, 512), (512, 264), (200, 264)))
    y = ops.linear(x, w, residual=r, act=ops.ACT_GELU_TANH)
    again = ops.linear(x, w, residual=r, act=ops.ACT_GELU_TANH)
    assert torch.equal(y, again)
    ops.linear(x, w, residual=r, act=ops.ACT_GELU_TANH, out=r)
    assert torch.equal(y, r)


@pytest.mark.parametrize("name", ["bf16", "f32"])
@pytest.mark.parametrize("M", [1, 3, 40, 300])
def test_linear_special_values(ops, M, name):
    """Infinities and NaN of an input row or weight column stay in that row or column; huge finite
    pre-activations have finite activations and derivatives."""
    say(f"special values M={M} {name}")
    d = dt(name)
    x, w = torch.ones(M, 96, dtype=d, device="cuda"), torch.ones(96, 80, dtype=d, device="cuda")
    x[M - 1, 5] = float("nan")
    w[3, 7] = float("inf")
    y = ops.linear(x, w, act=ops.ACT_RELU).float()
    assert y[M - 1].isnan().all()
    for m in (0, M - 2):
        if 0 <= m < M - 1:
            assert y[m, 7].item() == float("inf")
            rest = torch.cat([y[m, :7], y[m, 8:]])
            assert (rest == 96).all()
    big = torch.tensor([[1e30, -1e30, 3e19, -3e19, 60.0, -60.0, 0.0, 1.0]], dtype=d, device="cuda")
    one = torch.eye(8, dtype=d, device="cuda")
    for a in ("gelu_tanh", "silu"):
        out = ops.linear(big, one, act=ops.ACTS[a]).double().cpu()[0]
        want = act(big.double().cpu()[0].clamp(-100, 1e38), a)
        assert out.isfinite().all()
        assert torch.allclose(out, want, rtol=2.0 ** -8, atol=1e-10), (a, out, want)
        dx = ops.linear_backward(torch.ones_like(big), big, one, pre=big, act=ops.ACTS[a])[0].double().cpu()[0]
        assert torch.allclose(dx[:6], torch.tensor([1, 0, 1, 0, 1, 0], dtype=torch.float64), atol=1e-10), (a, dx)


OFFSETS = {  # rows, offsets
    "one": (37, [0, 37]),
    "idle": (300, [0, 0, 5, 5, 140, 299, 299, 300]),
    "single_rows": (9, list(range(10))),
    "tail_without_expert": (200, [0, 10, 150, 160]),
    "all_in_last": (130, [0, 0, 0, 0, 130]),
    "none": (20, [0, 0, 0]),
    "decode": (16, [0, 0, 2, 6, 7, 12, 15, 16, 16]),
    "no_rows": (0, [0, 0, 0]),
    "many_experts": (333, sorted([0, 333] + [(i * 97) % 331 for i in range(129)])),
    "sixty_four": (100, [0] + [min(100, 2 * i) for i in range(64)]),
    "malformed": (90, [5, 30, 10, 200, 60, -3]),
    "wide": (700, [0, 260, 300, 650, 700]),
    "long": (3000, [0, 1500, 1500, 2990]),
}


def spans(T, off):
    out, last = [], 0
    for o in off[1:]:
        end = max(last, min(max(o, 0), T))
        out.append((last, end))
        last = end
    return out, last


@pytest.mark.parametrize("name", ["bf16", "f32"])
@pytest.mark.parametrize("kn", [(64, 128), (72, 40), (33, 65), (512, 136)], ids=str)
@pytest.mark.parametrize("case", OFFSETS)
def test_grouped(ops, case, kn, name):
    T, off = OFFSETS[case]
    K, N = kn
    i = list(OFFSETS).index(case) + K
    a, wt, has_b, pad, shift = ACTS[i % 4], i % 2 == 1, i % 3 != 0, (0, 8, 3)[i % 3], (0, 8, 1)[i % 3]
    say(f"grouped {case} {kn} {name} act={a} wt={wt} pad={pad} shift={shift}")
    E, d = len(off) - 1, dt(name)
    g = torch.Generator().manual_seed(i)
    x, w = data(g, T, K, dtype=d), data(g, E, K, N, dtype=d, std=K ** -0.5)
    b = data(g, E, N, dtype=d) if has_b else None
    doff = torch.tensor(off, dtype=torch.int32, device="cuda")
    dwt = place(w.transpose(1, 2).contiguous(), d, pad, shift).transpose(1, 2) if wt else place(w, d, pad, shift)
    y, pre = ops.grouped_linear(place(x, d, pad, shift), dwt, doff, None if b is None else b.to("cuda", d),
                                act=ops.ACTS[a], need_pre=True)
    where, last = spans(T, off)
    z, ty, tz = torch.zeros(T, N, dtype=torch.float64), torch.zeros(T, N), torch.zeros(T, N)
    for e, (p, q) in enumerate(where):
        be = b[e] if has_b else None
        z[p:q] = x[p:q] @ w[e] + (be if has_b else 0)
        ty[p:q], tz[p:q] = forward_tol(x[p:q], w[e], be, z[p:q], act(z[p:q], a), a, name)
    close(pre, z, tz, "pre")
    close(y, act(z, a), ty, "y")
    assert not y[last:].any() and not pre[last:].any()

    dy, zin = data(g, T, N, dtype=d), data(g, T, N, dtype=d, std=2.0)
    dx, dw, db = ops.grouped_linear_backward(place(dy, d, pad, shift), place(x, d, pad, shift), dwt, doff,
                                             pre=place(zin, d, pad, shift), act=ops.ACTS[a])
    assert not dx[last:].any()
    for e, (p, q) in enumerate(where):
        if p == q:
            assert not dw[e].any() and not db[e].any(), e
        else:
            check_backward(x[p:q], w[e], dy[p:q], zin[p:q], a, name, dx[p:q], dw[e], db[e])


NORM = [(1, 1), (1, 8), (3, 7), (5, 64), (2, 512), (9, 513), (4, 1024), (7, 1000), (1, 8192), (600, 264), (33, 4099),
        (3, 8193), (2, 16384), (2, 20001), (3, 40000), (0, 16), (1100, 40), (1, 9000), (1, 16392), (1, 33000), (16, 512),
        (17, 482), (2, 4096), (2, 4097), (40, 12296), (5, 6000), (260, 5000)]


@pytest.mark.parametrize("name", ["bf16", "f32"])
@pytest.mark.parametrize("size", NORM, ids=str)
def test_layer_norm(ops, size, name):
    M, N = size
    i = NORM.index(size)
    pad, shift, has_w, has_b = (0, 8, 3)[i % 3], (0, 8, 1)[i % 3], i % 4 != 1, i % 4 != 2
    say(f"layer_norm {size} {name} pad={pad} shift={shift}")
    g = torch.Generator().manual_seed(i)
    d, eps = dt(name), 1e-5
    x = data(g, M, N, dtype=d) + 3.0 * data(g, M, 1, dtype=d)
    x = x.to(d).double()
    w = data(g, N, dtype=d) if has_w else None
    b = data(g, N, dtype=d) if has_b else None
    dw_, db_ = (None if t is None else place(t, d, 0, shift) for t in (w, b))
    px = place(x, d, pad, shift)
    y, mean, rstd = ops.layer_norm(px, dw_, db_, eps=eps)
    mu = x.mean(1, keepdim=True)
    var = ((x - mu) ** 2).mean(1, keepdim=True)
    rs = (var + eps) ** -0.5
    xh = (x - mu) * rs
    wv, bv = (w if has_w else torch.ones(N, dtype=torch.float64)), (b if has_b else torch.zeros(N, dtype=torch.float64))
    # relative error of the sums, and what the rounded mean does to a deviation
    n = (N + 16) * E32
    off = n * x.abs().mean(1, keepdim=True) if M else mu
    close(mean, mu[:, 0], off[:, 0] + E32 * mu[:, 0].abs(), "mean")
    rel = n + 2 * off * off / (var + eps) + 8 * E32
    close(rstd, rs[:, 0], (rel * rs)[:, 0], "rstd")
    want = xh * wv + bv
    # a deviation of two close values is exact, otherwise off by its rounding
    tx = off * rs + xh.abs() * (rel + 4 * E32)
    close(y, want, tx * wv.abs() + (1.01 * U[name] + 4 * E32) * want.abs() + 4 * E32 * bv.abs(), "y")

    dy = data(g, M, N, dtype=d)
    m32, r32 = mu[:, 0].float(), rs[:, 0].float()
    dx, dw, db = ops.layer_norm_backward(place(dy, d, pad, shift), px, m32.cuda(), r32.cuda(), dw_)
    xh = (x - m32.double()[:, None]) * r32.double()[:, None]
    gy = dy * wv
    txh = 4 * E32 * ((x.abs() + m32.double().abs()[:, None]) * r32.double()[:, None])
    s1 = (gy * xh).mean(1, keepdim=True)
    want = r32.double()[:, None] * (gy - gy.mean(1, keepdim=True) - xh * s1)
    ts0 = n * gy.abs().mean(1, keepdim=True) if M else mu
    ts1 = (n * (gy * xh).abs() + gy.abs() * txh).mean(1, keepdim=True) if M else mu
    size_ = gy.abs() + gy.abs().mean(1, keepdim=True) + (xh * s1).abs() if M else gy
    tol = r32.double()[:, None] * (ts0 + xh.abs() * ts1 + txh * s1.abs() + 8 * E32 * size_) + 1.01 * U[name] * want.abs()
    close(dx, want, tol, "dx")
    want = (dy * xh).sum(0)
    close(dw, want, ((M + 16) * E32 * (dy * xh).abs() + dy.abs() * txh).sum(0) + 1.01 * U[name] * want.abs(), "dw")
    want = dy.sum(0)
    close(db, want, (M + 16) * E32 * dy.abs().sum(0) + 1.01 * U[name] * want.abs(), "db")


def test_layer_norm_in_place_and_subsets(ops):
    say("layer_norm in place, backward subsets")
    g = torch.Generator().manual_seed(9)
    d = torch.bfloat16
    x, dy = (data(g, 50, 600, dtype=d).to("cuda", d) for _ in range(2))
    w = data(g, 600, dtype=d).to("cuda", d)
    y, mean, rstd = ops.layer_norm(x, w)
    full = ops.layer_norm_backward(dy, x, mean, rstd, w)
    for need in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1), (0, 0, 0)):
        part = ops.layer_norm_backward(dy, x, mean, rstd, w, need_x=need[0], need_weight=need[1], need_bias=need[2])
        for p, f, n in zip(part, full, need):
            assert (p is None) == (not n) and (p is None or torch.equal(p, f))
    x2 = x.clone()
    assert torch.equal(ops.layer_norm(x2, w, out=x2)[0], y) and torch.equal(x2, y)


def test_layer_norm_special_rows(ops):
    """A constant row has deviation zero, a row with NaN or infinity spoils only itself."""
    say("layer_norm special rows")
    for d in (torch.bfloat16, torch.float32):
        x = torch.randn(5, 300, device="cuda").to(d)
        clean = ops.layer_norm(x)[0]
        x[1] = 3.0
        x[2, 7] = float("nan")
        x[3, 9] = float("inf")
        y, mean, rstd = ops.layer_norm(x, eps=1e-5)
        assert not y[1].any() and abs(rstd[1].item() * 1e-5 ** 0.5 - 1) < 1e-5
        assert y[2].isnan().all() and y[3].isnan().all()
        assert torch.equal(y[0], clean[0]) and torch.equal(y[4], clean[4])


def test_gradients_against_differences(ops):
    """Central differences of sum(y dy) in fp32: truncation is O(h^2) of third derivatives below 2, rounding
    about K e |f| / h; both are below 2e-3 of the gradients' size at h = 2^-6."""
    say("differences")
    g = torch.Generator().manual_seed(11)
    M, K, N, h = 6, 20, 12, 2.0 ** -6
    x, w, b, dy = (torch.randn(*s, generator=g).cuda() for s in ((M, K), (K, N), (N,), (M, N)))
    w *= K ** -0.5

    def f(x, w, b):
        return (ops.linear(x, w, b, act=ops.ACT_GELU_TANH).double() * dy.double()).sum().item()
    _, pre = ops.linear(x, w, b, act=ops.ACT_GELU_TANH, need_pre=True)
    grads = ops.linear_backward(dy, x, w, pre=pre, act=ops.ACT_GELU_TANH)
    for k, t in enumerate((x, w, b)):
        for j in range(0, t.numel(), 7):
            p, q = [u.clone() for u in (x, w, b)], [u.clone() for u in (x, w, b)]
            p[k].view(-1)[j] += h
            q[k].view(-1)[j] -= h
            assert abs((f(*p) - f(*q)) / (2 * h) - grads[k].reshape(-1)[j].item()) < 2e-3 * 4, (k, j)

    def fn(x, w, b):
        return (ops.layer_norm(x, w, b)[0].double() * dx_.double()).sum().item()
    x, w, b, dx_ = (torch.randn(*s, generator=g).cuda() for s in ((4, 24), (24,), (24,), (4, 24)))
    _, mean, rstd = ops.layer_norm(x, w, b)
    grads = ops.layer_norm_backward(dx_, x, mean, rstd, w)
    for k, t in enumerate((x, w, b)):
        for j in range(0, t.numel(), 5):
            p, q = [u.clone() for u in (x, w, b)], [u.clone() for u in (x, w, b)]
            p[k].view(-1)[j] += h
            q[k].view(-1)[j] -= h
            assert abs((fn(*p) - fn(*q)) / (2 * h) - grads[k].reshape(-1)[j].item()) < 2e-3 * 4, (k, j)

    off = torch.tensor([0, 2, 2, 5], dtype=torch.int32, device="cuda")
    x, w, b, dy = (torch.randn(*s, generator=g).cuda() for s in ((6, K), (3, K, N), (3, N), (6, N)))
    w *= K ** -0.5

    def fg(x, w, b):
        return (ops.grouped_linear(x, w, off, b, act=ops.ACT_SILU).double() * dy.double()).sum().item()
    _, pre = ops.grouped_linear(x, w, off, b, act=ops.ACT_SILU, need_pre=True)
    grads = ops.grouped_linear_backward(dy, x, w, off, pre=pre, act=ops.ACT_SILU)
    for k, t in enumerate((x, w, b)):
        for j in range(0, t.numel(), 11):
            p, q = [u.clone() for u in (x, w, b)], [u.clone() for u in (x, w, b)]
            p[k].view(-1)[j] += h
            q[k].view(-1)[j] -= h
            assert abs((fg(*p) - fg(*q)) / (2 * h) - grads[k].reshape(-1)[j].item()) < 2e-3 * 4, (k, j)


def test_streams_and_graphs(ops):
    """A call on another stream, and replays of a captured step between eager work."""
    say("streams and graphs")
    g = torch.Generator().manual_seed(13)
    d = torch.bfloat16
    x, w, r = (data(g, *s, dtype=d).to("cuda", d) for s in ((24, 1024), (1024, 512), (24, 512)))
    nw = data(g, 1024, dtype=d).to("cuda", d)
    off = torch.tensor([0, 9, 9, 24], dtype=torch.int32, device="cuda")
    we = data(g, 3, 1024, 512, dtype=d).to("cuda", d)

    def step():
        n, mean, rstd = ops.layer_norm(x, nw)
        y, pre = ops.linear(n, w, residual=r, act=ops.ACT_SILU, need_pre=True)
        dx, dw, db = ops.linear_backward(y, n, w, pre=pre, act=ops.ACT_SILU)
        z = ops.grouped_linear(n, we, off)
        dn = ops.layer_norm_backward(dx, x, mean, rstd, nw)
        return [y, dx, dw, db, z, *dn]
    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for rep in range(4):
        for t in got:
            t.fill_(float("nan"))
        ops.linear(torch.randn(24, 1024, device="cuda").to(d), w)  # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), rep


def test_rows_beyond_32_bits(ops):
    """Row and expert offsets past 2^31 elements: only the last rows and the last expert hold values, and
    theirs are the only results that are not zero."""
    say("offsets past 32 bits")
    g = torch.Generator().manual_seed(17)
    d = torch.bfloat16
    M, K, N = 530_000, 4096, 8   # x: 2.17e9 elements
    x = torch.zeros(M, K, dtype=d, device="cuda")
    tail = data(g, 3, K, dtype=d)
    x[-3:] = tail.to("cuda", d)
    w = data(g, K, N, dtype=d, std=K ** -0.5)
    want = tail @ w
    tol = (K + 8) * E32 * (tail.abs() @ w.abs()) + 1.01 * U["bf16"] * want.abs()
    y = ops.linear(x, w.to("cuda", d))
    close(y[-3:], want, tol, "linear")
    assert not y[:-3].any()
    off = torch.tensor([0, 5, M], dtype=torch.int32, device="cuda")
    we = torch.stack([torch.zeros_like(w), w]).to("cuda", d)
    close(ops.grouped_linear(x, we, off)[-3:], want, tol, "grouped rows")
    n = ops.layer_norm(x)[0]
    xh = (tail - tail.mean(1, keepdim=True)) / (tail.var(1, unbiased=False, keepdim=True) + 1e-5).sqrt()
    assert (n[-3:].double().cpu() - xh).abs().max() < 4 * U["bf16"] * xh.abs().max()
    assert not n[:-3].any()
    dy = torch.zeros(M, N, dtype=d, device="cuda")
    dt_ = data(g, 3, N, dtype=d)
    dy[-3:] = dt_.to("cuda", d)
    dx, dw, db = ops.linear_backward(dy, x, w.to("cuda", d))
    check_backward(tail, w, dt_, torch.zeros_like(dt_), "none", "bf16", dx[-3:], None, None)
    want = tail.t() @ dt_
    close(dw, want, (M + 8) * E32 * (tail.abs().t() @ dt_.abs()) + 1.01 * U["bf16"] * want.abs(), "dw")
    assert not dx[:-3].any()
    del x, n, dx, y
    E, K, N = 35, 8192, 8192     # w: 2.35e9 elements
    we = torch.zeros(E, K, N, dtype=d, device="cuda")
    w = torch.randn(K, N, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") * K ** -0.5
    we[-1] = w.to(d)
    xs = data(g, 4, K, dtype=d)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = 4
    got = ops.grouped_linear(xs.to("cuda", d), we, off)
    wd = we[-1].double()
    xd = xs.cuda()
    want = xd @ wd
    close(got, want.cpu(), ((K + 8) * E32 * (xd.abs() @ wd.abs()) + 1.01 * U["bf16"] * want.abs()).cpu(), "last expert")


def test_refusals(ops):
    say("refusals")
    d = torch.bfloat16
    x, w = torch.zeros(4, 8, dtype=d, device="cuda"), torch.zeros(8, 16, dtype=d, device="cuda")
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    bad = [
        (TypeError, lambda: ops.linear(x.cpu(), w)),
        (ValueError, lambda: ops.linear(x, w.float())),
        (ValueError, lambda: ops.linear(x.half(), w.half())),
        (ValueError, lambda: ops.linear(x, w[:7])),
        (ValueError, lambda: ops.linear(x[0], w)),
        (ValueError, lambda: ops.linear(x, w, bias=torch.zeros(15, dtype=d, device="cuda"))),
        (ValueError, lambda: ops.linear(x, w, bias=torch.zeros(16, dtype=d))),
        (ValueError, lambda: ops.linear(x, w, residual=torch.zeros(4, 15, dtype=d, device="cuda"))),
        (ValueError, lambda: ops.linear(x, w, out=torch.zeros(4, 15, dtype=d, device="cuda"))),
        (ValueError, lambda: ops.linear(torch.zeros(8, 4, dtype=d, device="cuda").t(), w)),
        (ValueError, lambda: ops.linear(torch.zeros(1, 8, dtype=d, device="cuda").expand(4, 8), w)),
        (ValueError, lambda: ops.linear(x, torch.zeros(16, 32, dtype=d, device="cuda")[::2, ::2])),
        (RuntimeError, lambda: ops.linear(x, w, act=17)),
        (ValueError, lambda: ops.linear_backward(torch.zeros(4, 16, dtype=d, device="cuda"), x, w, act=ops.ACT_SILU)),
        (ValueError, lambda: ops.grouped_linear(x, w, off)),
        (ValueError, lambda: ops.grouped_linear(x, w[None], off.long())),
        (ValueError, lambda: ops.grouped_linear(x, w[None], off.cpu())),
        (ValueError, lambda: ops.grouped_linear(x, w[None], torch.zeros(3, dtype=torch.int32, device="cuda"))),
        (ValueError, lambda: ops.layer_norm(x, torch.zeros(7, dtype=d, device="cuda"))),
        (RuntimeError, lambda: ops.layer_norm(x, eps=-1.0)),
        (RuntimeError, lambda: ops.layer_norm(torch.zeros(3, 0, dtype=d, device="cuda"))),
        (ValueError, lambda: ops.layer_norm_backward(x, x, torch.zeros(4, dtype=d, device="cuda"),
                                                     torch.zeros(4, device="cuda"))),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            say("not refused:", i)


# More than one round of large tiles, the last one at most half full, with
# ragged edges: its tiles are computed in halves, some of them without a row.
# Compared at some rows, with those on both sides of the halves' borders.
def some_rows(M):
    return sorted({r for r in range(0, M, 23)} | {r for k in range(0, M + 1, 128) for r in (k - 1, k) if 0 <= r < M} | {M - 1})


@pytest.mark.parametrize("wt", [False, True])
def test_linear_rounds(ops, wt):
    M, K, N = 4200, 2056, 4312
    g = torch.Generator().manual_seed(11 + wt)
    d = torch.bfloat16
    x, w, b, r = (data(g, *s, dtype=d, std=sd) for s, sd in (((M, K), 1), ((K, N), K ** -0.5), ((N,), 1), ((M, N), 1)))
    dw = place(w.t().contiguous(), d, 8).t() if wt else place(w, d, 8)
    y, pre = ops.linear(place(x, d, 8), dw, b.to("cuda", d), residual=place(r, d, 8), act=ops.ACTS["gelu_tanh"], need_pre=True)
    s = some_rows(M)
    z = x[s] @ w + b
    want = act(z, "gelu_tanh") + r[s]
    ty, tz = forward_tol(x[s], w, b, z, want, "gelu_tanh", "bf16")
    close(y[s], want, ty + 4 * E32 * r[s].abs(), "y")
    close(pre[s], z, tz, "pre")


@pytest.mark.parametrize("wt", [False, True])
def test_linear_gradient_rounds(ops, wt):
    M, K, N = 2056, 4200, 4312
    g = torch.Generator().manual_seed(21 + wt)
    d = torch.bfloat16
    x, w, dy = data(g, M, K, dtype=d), data(g, K, N, dtype=d, std=N ** -0.5), data(g, M, N, dtype=d)
    dw_in = place(w.t().contiguous(), d, 8).t() if wt else place(w, d, 8)
    for need_x, need_w in ((False, True), (True, True)):
        dx, dw, _ = ops.linear_backward(place(dy, d, 8), place(x, d, 8), dw_in, need_x=need_x, need_w=need_w)
        s = some_rows(K)
        check_backward(x[:, s], w[s], dy, dy, "none", "bf16", None if dx is None else dx[:, s], dw[s], None)


@pytest.mark.parametrize("wt", [False, True])
def test_grouped_rounds(ops, wt):
    T, K, N, off = 4400, 2056, 4312, [0, 700, 700, 1900, 3180, 4390]
    g = torch.Generator().manual_seed(31 + wt)
    E, d = len(off) - 1, torch.bfloat16
    x, w, b = data(g, T, K, dtype=d), data(g, E, K, N, dtype=d, std=K ** -0.5), data(g, E, N, dtype=d)
    doff = torch.tensor(off, dtype=torch.int32, device="cuda")
    dwt = place(w.transpose(1, 2).contiguous(), d).transpose(1, 2) if wt else place(w, d)
    y, pre = ops.grouped_linear(place(x, d, 8), dwt, doff, b.to("cuda", d), act=ops.ACTS["silu"], need_pre=True)
    for e in range(E):
        s = [off[e] + r for r in some_rows(off[e + 1] - off[e])] if off[e + 1] > off[e] else []
        z = x[s] @ w[e] + b[e]
        ty, tz = forward_tol(x[s], w[e], b[e], z, act(z, "silu"), "silu", "bf16")
        close(y[s], act(z, "silu"), ty, f"y {e}")
        close(pre[s], z, tz, f"pre {e}")
    assert not y[off[-1]:].any() and not pre[off[-1]:].any()


# Widths around the units of 16 bytes and the threads of a row, in rows that are
# not aligned, surrounded by NaN; also in place, and nothing else is written.
@pytest.mark.parametrize("name", ["bf16", "f32"])
@pytest.mark.parametrize("N", [2, 8, 9, 15, 23, 505, 511, 517, 1025, 2047, 2051, 4095, 8185, 8193, 12287, 12289, 16383])
def test_layer_norm_odd_widths(ops, N, name):
    M, eps, d = 5, 1e-5, dt(name)
    say(f"layer_norm odd width {N} {name}")
    g = torch.Generator().manual_seed(N)
    x, w, b = data(g, M, N, dtype=d), data(g, N, dtype=d), data(g, N, dtype=d)
    px = place(x, d, 3, 1)
    y, mean, rstd = ops.layer_norm(px, place(w, d, 0, 1), place(b, d, 0, 1), eps=eps)
    mu = x.mean(1, keepdim=True)
    var = ((x - mu) ** 2).mean(1, keepdim=True)
    rs = (var + eps) ** -0.5
    xh = (x - mu) * rs
    n = (N + 16) * E32
    off = n * x.abs().mean(1, keepdim=True)
    rel = n + 2 * off * off / (var + eps) + 8 * E32
    close(mean, mu[:, 0], off[:, 0] + E32 * mu[:, 0].abs(), "mean")
    close(rstd, rs[:, 0], (rel * rs)[:, 0], "rstd")
    want = xh * w + b
    close(y, want, (off * rs + xh.abs() * (rel + 4 * E32)) * w.abs() + (1.01 * U[name] + 4 * E32) * want.abs()
          + 4 * E32 * b.abs(), "y")
    box = torch.full((M + 2, N + 3), 7.0, dtype=d, device="cuda")
    inside = box[1:M + 1, 1:N + 1]
    inside.copy_(px)
    ops.layer_norm(inside, place(w, d, 0, 1), place(b, d, 0, 1), eps=eps, out=inside)
    assert torch.equal(inside, y)
    inside.fill_(7.0)
    assert bool((box == 7.0).all()), "wrote outside the rows"
