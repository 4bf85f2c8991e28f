"""GPU tests of the router, the rows' way to the experts and back, 4-bit linear
layers and gradient clipping against the formulas in 64 bits.

Tolerances are element-wise bounds on the rounding of the stated algorithm, with
e = 2^-24 the unit roundoff of the fp32 sums and u that of the stored type (2^-8
bf16, 2^-24 fp32):
  - a probability: the logit's distance d from the largest is rounded (|d| e), the
    exponential is within 4 e, its sum over E within (E + 8) e, two more roundings:
    relative (|d| + E + 16) e; below 2^-126 it may be 0;
  - the sum of probabilities over T tokens is within (T + 8) e on top of theirs;
  - a sum of n products is within (n + 8) e sum |a||b|;
  - a 4-bit product: per group of G two sums of G products with factors up to 31
    (sum x (16 + q) and (16 + z) sum x), so 62 (G + 8) e s sum |x|, three times the
    products for fp32; then the sum over groups and waves;
  - activations as in test_gpu_ops.py; a stored value is rounded once, 1.01 u |y|.
Inputs sit in larger buffers filled with NaN, outputs in buffers whose surroundings
have to stay as they were."""
import math
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

E32 = 2.0 ** -24
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
C0 = math.sqrt(2 / math.pi)
ACTS = ("none", "gelu_tanh", "relu", "silu")
NAMES = ["bf16", "f32"]


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
    strides, n = [1], ld
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


def close(got, want, tol, what):
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~((got - want).abs() <= tol)
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {got[i]} want {want[i]} "
                             f"tol {tol[i] if torch.is_tensor(tol) else tol}")


def same(got, want, what):
    assert torch.equal(got.cpu().long(), want.long()), what


# ------------------------------------------------------------------- router

def softmax(x):
    live = (x > -math.inf).any(1)
    p = torch.zeros_like(x)
    p[live] = torch.softmax(x[live], 1)
    return p


def routing(x, k, normalize, valid=None):
    """The documented result, token by token; with it the bound of the gates."""
    T, E = x.shape
    x = x.clone()
    if valid is not None:
        x[~valid] = -math.inf
    p = softmax(x)
    v, order = torch.sort(x, dim=1, descending=True, stable=True)
    used = v[:, :k] > -math.inf
    experts = torch.where(used, order[:, :k], -1)
    gates = torch.gather(p, 1, order[:, :k]) * used
    far = torch.where(used, v[:, :1] - v[:, :k], torch.zeros_like(gates))
    rel = (far + E + 16) * E32
    if normalize:
        gates = gates / gates.sum(1, keepdim=True).clamp(min=1e-300)
        rel = 2 * rel.amax(1, keepdim=True) + 8 * E32 if T else rel
    rows = torch.full((T, k), -1, dtype=torch.long)
    counts = torch.bincount(experts[experts >= 0], minlength=E)
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)])
    at = offsets[:-1].tolist()
    for t, row in enumerate(experts.tolist()):
        for j, e in enumerate(row):
            if e >= 0:
                rows[t, j] = at[e]
                at[e] += 1
    n = max(int(used[:, 0].sum()), 1) if T else 1
    slopes = counts.double() * E / (n * n * k)
    return dict(experts=experts, gates=gates, rows=rows, counts=counts, offsets=offsets, loss=(slopes * p.sum(0)).sum(),
                slopes=slopes, tol=gates * rel + 2.0 ** -126)


ROUTES = [  # T, E, k: no token to several blocks of them, each width of the lanes, whole and ragged
    (0, 8, 2), (1, 1, 1), (1, 8, 2), (16, 8, 2), (5, 3, 3), (63, 16, 4), (65, 17, 4), (200, 60, 6), (256, 64, 8), (257, 65, 8),
    (320, 128, 8), (300, 129, 5), (1000, 256, 8), (700, 300, 32), (130, 512, 3), (129, 513, 7), (300, 1024, 32), (5000, 12, 2),
    (16500, 33, 4), (40000, 5, 1), (100, 20, 3), (128, 32, 4), (128, 33, 4),
]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("size", ROUTES, ids=lambda s: "x".join(map(str, s)))
def test_route(ops, size, name):
    T, E, k = size
    i = ROUTES.index(size) + NAMES.index(name)
    normalize, pad, shift = i % 2 == 0, (0, 8, 3)[i % 3], (0, 1, 8)[i % 3]
    say(f"route {size} {name} normalize={normalize} pad={pad} shift={shift}")
    g = torch.Generator().manual_seed(i)
    x = data(g, T, E, dtype=dt(name), std=2.0)
    if i % 4 == 1:
        x = (x * 2).round() / 2                     # many ties
    if i % 3 == 2:
        x[torch.rand(T, E, generator=g) < 0.4] = -math.inf
    valid = torch.rand(T, generator=g) < 0.7 if i % 3 == 1 else None
    r = ops.route(place(x, dt(name), pad, shift), k, normalize=normalize, valid=None if valid is None else valid.cuda())
    want = routing(x, k, normalize, valid)
    for what in ("experts", "rows", "counts", "offsets"):
        same(getattr(r, what), want[what], what)
    close(r.gates, want["gates"], want["tol"], "gates")
    close(r.slopes, want["slopes"], 1.01 * E32 * want["slopes"], "slopes")
    far = 12.0 + (x[x > -math.inf].abs().max().item() if (x > -math.inf).any() else 0)
    close(r.loss, want["loss"], (T + 2 * far + E + 40) * E32 * want["loss"], "loss")


@pytest.mark.parametrize("name", NAMES)
def test_route_special_rows(ops, name):
    say("route special rows", name)
    inf, nan = math.inf, math.nan
    x = torch.tensor([[-inf] * 4, [0.0, -0.0, 0.0, -0.0], [nan, 1.0, 2.0, 3.0], [1.0, inf, inf, 0.0], [-inf, -inf, 5.0, -inf],
                      [-nan, -inf, -inf, nan], [1e30, -1e30, 1e30, 0.0], [-200.0, 0.0, -300.0, -inf]])
    r = ops.route(x.to(dt(name)).cuda(), 2)
    assert r.experts.tolist() == [[-1, -1], [0, 1], [0, 3], [1, 2], [2, -1], [0, 3], [0, 2], [1, 0]]
    gates = r.gates.cpu()
    assert gates[0].tolist() == [0.0, 0.0] and gates[1].tolist() == [0.25, 0.25] and gates[4].tolist() == [1.0, 0.0]
    assert gates[[2, 3, 5]].isnan().all()
    assert gates[6].tolist() == [0.5, 0.5] and gates[7].tolist() == [1.0, 0.0]
    assert r.rows[0].tolist() == [-1, -1] and r.counts.tolist() == [5, 3, 3, 2] and r.offsets.tolist() == [0, 5, 8, 11, 13]
    assert r.loss.isnan()
    # nothing but padding
    r = ops.route(torch.full((70, 5), nan, dtype=dt(name), device="cuda"), 3, normalize=True,
                  valid=torch.zeros(70, dtype=torch.bool, device="cuda"))
    assert (r.experts == -1).all() and (r.rows == -1).all() and not r.gates.any() and not r.counts.any()
    assert not r.offsets.any() and r.loss.item() == 0 and not r.slopes.any()


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("size", ROUTES, ids=lambda s: "x".join(map(str, s)))
def test_route_backward(ops, size, name):
    T, E, k = size
    i = ROUTES.index(size) + NAMES.index(name)
    normalize, pad, shift = i % 2 == 1, (0, 3, 8)[i % 3], (1, 0, 8)[i % 3]
    say(f"route backward {size} {name} normalize={normalize}")
    g = torch.Generator().manual_seed(100 + i)
    x = data(g, T, E, dtype=dt(name), std=2.0)
    if i % 3 == 2:
        x[torch.rand(T, E, generator=g) < 0.4] = -math.inf
    valid = torch.rand(T, generator=g) < 0.7 if i % 3 == 1 else None
    r = routing(x, k, normalize, valid)
    dg = torch.randn(T, k, generator=g, dtype=torch.float32) if i % 5 else None
    dl = torch.tensor(0.7 * T, dtype=torch.float32) if i % 7 else None
    got = ops.route_backward(None if dg is None else dg.cuda(), None if dl is None else dl.cuda(), place(x, dt(name), pad, shift),
                             r["experts"].int().cuda(), r["slopes"].float().cuda(), normalize=normalize)
    has = r["experts"] >= 0
    live = has.any(1, keepdim=True) if T else torch.zeros(T, 1, dtype=torch.bool)
    p = softmax(x) * live
    c = (r["slopes"].float().double() * dl.double() if dl is not None else torch.zeros(E).double()).expand(T, E)
    d = torch.zeros(T, E, dtype=torch.float64)
    s = torch.zeros(T, E, dtype=torch.float64)
    s.scatter_add_(1, r["experts"].clamp(min=0), has.double())
    if dg is not None:
        d.scatter_add_(1, r["experts"].clamp(min=0), dg.double() * has)
    if normalize:
        q = p * s / (p * s).sum(1, keepdim=True).clamp(min=1e-300)
        want = p * (c - (p * c).sum(1, keepdim=True)) + q * (d - (q * d).sum(1, keepdim=True))
        size_ = p * (c + (p * c).sum(1, keepdim=True)) + q * (d.abs() + (q * d.abs()).sum(1, keepdim=True))
    else:
        want = p * ((c + d) - (p * (c + d)).sum(1, keepdim=True))
        size_ = p * (c + d.abs() + (p * (c + d.abs())).sum(1, keepdim=True))
    # each probability within (spread + E + 16) e; three of them in a product, sums over E; in all fewer than this many roundings
    spread = 2 * x[x > -math.inf].abs().max().item() if (x > -math.inf).any() else 0
    close(got, want, (4 * (spread + E) + 100) * E32 * size_ + 1.01 * U[name] * want.abs() + 2.0 ** -126, "dlogits")


def test_route_gradient_against_differences(ops):
    """Central differences of the kernel's own gates and loss, in fp32, at logits far enough apart for the choice to stay."""
    say("route differences")
    T, E, k, h = 6, 9, 3, 2.0 ** -6
    g = torch.Generator().manual_seed(3)
    x = torch.stack([torch.randperm(E, generator=g) * 0.25 for _ in range(T)]).float()
    dg, dl = torch.randn(T, k, generator=g), torch.tensor(2.0)
    for normalize in (False, True):
        def f(z):
            r = ops.route(z.cuda(), k, normalize=normalize)
            return (r.gates.cpu().double() * dg.double()).sum() + dl.double() * r.loss.cpu().double()
        r = ops.route(x.cuda(), k, normalize=normalize)
        got = ops.route_backward(dg.cuda(), dl.cuda(), x.cuda(), r.experts, r.slopes, normalize=normalize).cpu().double()
        want = torch.zeros(T, E, dtype=torch.float64)
        for t in range(T):
            for e in range(E):
                a, b = x.clone(), x.clone()
                a[t, e] += h
                b[t, e] -= h
                want[t, e] = (f(a) - f(b)) / (2 * h)
        # truncation h^2 / 6 times a third derivative below 8 for |dg| < 4; roundings 100 e / h
        close(got, want, 8 * h * h / 6 * 4 + 400 * E32 / h, f"differences, normalize={normalize}")


# ------------------------------------------------- rows to experts and back

MOVES = [  # T, E, k, D
    (0, 4, 2, 16), (1, 1, 1, 1), (1, 8, 2, 4096), (7, 5, 3, 33), (64, 8, 2, 8), (65, 8, 8, 17), (300, 16, 1, 200), (129, 60, 6, 520),
    (33, 64, 32, 96), (500, 8, 2, 1000), (40, 4, 4, 8200), (2100, 6, 3, 136), (9, 5, 2, 0), (2049, 5, 2, 1040),
]


def moved(g, T, E, k, i):
    """Slots of a random router, some tokens without an expert and some with too few."""
    x = torch.randn(T, E, generator=g, dtype=torch.float64)
    if i % 2:
        x[torch.rand(T, E, generator=g) < 0.3] = -math.inf
    return routing(x, k, False, torch.rand(T, generator=g) < 0.8 if i % 3 else None)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("size", MOVES, ids=lambda s: "x".join(map(str, s)))
def test_exchange(ops, size, name):
    T, E, k, D = size
    i = MOVES.index(size) + NAMES.index(name)
    pad, shift = (0, 8, 3)[i % 3], (0, 8, 1)[i % 3]
    say(f"exchange {size} {name} pad={pad} shift={shift}")
    g = torch.Generator().manual_seed(i)
    d, u = dt(name), U[name]
    r = moved(g, T, E, k, i)
    R, rows = T * k, r["rows"]
    drows, doff = rows.int().cuda(), r["offsets"].int().cuda()
    token, slot = (rows >= 0).nonzero(as_tuple=True)
    at = rows[token, slot]
    # dispatch
    x = data(g, T, D, dtype=d)
    out = torch.full((R + 2, D + 5), 7.0, dtype=d, device="cuda")
    got = ops.dispatch(place(x, d, pad, shift), drows, doff, out=out[1:R + 1, 2:D + 2])
    want = torch.zeros(R, D, dtype=torch.float64)
    want[at] = x[token]
    assert torch.equal(got.double().cpu(), want), "dispatch"
    keep = out.clone()
    keep[1:R + 1, 2:D + 2] = 7.0
    assert bool((keep == 7.0).all()), "dispatch wrote outside the output"
    # combine; rows that no slot names hold NaN, and so do gates without a slot
    y = data(g, R, D, dtype=d)
    named = torch.zeros(R, dtype=torch.bool)
    named[at] = True
    gates = torch.rand(T, k, generator=g, dtype=torch.float32)
    bad = gates.clone()
    bad[rows < 0] = math.nan
    res = data(g, T, D, dtype=d) if i % 2 else None
    yn = y.clone()
    yn[~named] = math.nan
    for gated in (True, False):
        w = gates.double()[token, slot][:, None] if gated else 1.0
        want = torch.zeros(T, D, dtype=torch.float64).index_add(0, token, y[at] * w)
        size_ = torch.zeros(T, D, dtype=torch.float64).index_add(0, token, (y[at] * w).abs())
        if res is not None:
            want, size_ = want + res, size_ + res.abs()
        out = torch.full((T + 2, D + 5), 7.0, dtype=d, device="cuda")
        got = ops.combine(place(yn, d, pad, shift), drows, bad.cuda() if gated else None,
                          residual=None if res is None else place(res, d, pad, shift), out=out[1:T + 1, 3:D + 3])
        close(got, want, (k + 8) * E32 * size_ + 1.01 * u * want.abs(), "combine")
        keep = out.clone()
        keep[1:T + 1, 3:D + 3] = 7.0
        assert bool((keep == 7.0).all()), "combine wrote outside the output"
        if res is not None:     # onto the residual itself
            box = place(res, d, pad, shift)
            assert torch.equal(ops.combine(place(yn, d), drows, bad.cuda() if gated else None, residual=box, out=box), got)
    # its gradients
    do = data(g, T, D, dtype=d)
    dy, dg = ops.combine_backward(place(do, d, pad, shift), place(yn, d, pad, shift), drows, doff, bad.cuda())
    want = torch.zeros(R, D, dtype=torch.float64)
    want[at] = do[token] * gates.double()[token, slot][:, None]
    close(dy, want, (1.01 * u + 2 * E32) * want.abs() + 2.0 ** -133, "dy")
    wg = torch.zeros(T, k, dtype=torch.float64)
    wg[token, slot] = (do[token] * y[at]).sum(1)
    tol = torch.zeros(T, k, dtype=torch.float64)
    tol[token, slot] = (D + 8) * E32 * (do[token] * y[at]).abs().sum(1)
    close(dg, wg, tol, "dgates")
    # one at a time, and without gates
    assert torch.equal(ops.combine_backward(do.to(d).cuda(), y.to(d).cuda(), drows, doff, bad.cuda(), need_gates=False)[0], dy)
    none, only = ops.combine_backward(do.to(d).cuda(), y.to(d).cuda(), drows, doff, None, need_y=False)
    assert none is None and torch.equal(only, dg)
    assert torch.equal(ops.combine_backward(do.to(d).cuda(), y.to(d).cuda(), drows, doff)[0], ops.dispatch(do.to(d).cuda(), drows, doff))


@pytest.mark.parametrize("name", NAMES)
def test_exchange_any_rows(ops, name):
    """Entries out of range are no slots; rows before the end that nothing names are left as they were."""
    say("exchange any rows", name)
    d = dt(name)
    x = torch.arange(1, 13, dtype=torch.float32).view(3, 4).to(d).cuda()
    rows = torch.tensor([[0, 6], [-5, 2 ** 31 - 1], [3, -2 ** 31]], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    out = torch.full((6, 4), 9.0, dtype=d, device="cuda")
    ops.dispatch(x, rows, off, out=out)
    assert out.float().tolist() == [[1, 2, 3, 4], [9] * 4, [9] * 4, [9, 10, 11, 12], [9] * 4, [0] * 4]
    for end, zeros in ((-7, 6), (0, 6), (6, 0), (2 ** 31 - 1, 0)):
        out.fill_(9.0)
        ops.dispatch(x, torch.full((3, 2), -1, dtype=torch.int32, device="cuda"),
                     torch.tensor([0, end], dtype=torch.int32, device="cuda"), out=out)
        assert (out[:6 - zeros] == 9).all() and not out[6 - zeros:].any()
    y = torch.full((4, 4), 2.0, dtype=d, device="cuda")     # fewer rows than slots
    assert ops.combine(y, rows).float().tolist() == [[2.0] * 4, [0.0] * 4, [2.0] * 4]
    dy, dg = ops.combine_backward(x, y, rows, torch.tensor([4], dtype=torch.int32, device="cuda"))
    assert dg.tolist() == [[20.0, 0.0], [0.0, 0.0], [84.0, 0.0]]
    assert dy[0].tolist() == [1, 2, 3, 4] and dy[3].tolist() == [9, 10, 11, 12]


# ------------------------------------------------------------- 4-bit weights

def codes(g, *shape, group, dtype, zeros):
    *lead, K, N = shape
    G = -(-K // group)
    q = torch.randint(0, 16, shape, generator=g, dtype=torch.uint8)
    s = ((0.5 + torch.rand(*lead, G, N, generator=g, dtype=torch.float64)) * 0.2 * max(K, 1) ** -0.5).to(dtype).double()
    z = torch.randint(0, 16, (*lead, G, N), generator=g, dtype=torch.uint8) if zeros else None
    return q, s, z


def weight(q, s, z, group):
    """The weight, and its scales spread over k."""
    spread = torch.arange(q.shape[-2]) // group
    sk = s[..., spread, :]
    zk = z.double()[..., spread, :] if z is not None else 8.0
    return sk * (q.double() - zk), sk


def int4_tol(x, w, sk, b, z, y, a, group, name):
    G, parts = min(group, 128), 1 if name == "bf16" else 3
    size = x.abs() @ w.abs() + (b.abs() if b is not None else 0)
    zt = 62 * parts * (G + 8) * E32 * (x.abs() @ sk) + (x.shape[1] // 32 + 32) * E32 * size
    return 1.2 * zt + (0 if a == "none" else 2.0 ** -20 * (1 + z.abs())) + (1.01 * U[name] + 4 * E32) * y.abs()


INT4 = [  # M, K, N, group
    (1, 128, 16, 128), (1, 1, 1, 32), (1, 4096, 512, 128), (1, 1000, 200, 64), (2, 65, 33, 32), (3, 300, 17, 256), (5, 64, 72, 64),
    (16, 2048, 144, 128), (17, 264, 136, 32), (13, 4300, 9000, 128), (31, 128, 1, 128), (33, 40, 24, 64), (64, 512, 264, 32),
    (65, 1001, 65, 64), (130, 384, 200, 384), (300, 200, 130, 128), (3, 0, 5, 32), (0, 8, 8, 32), (4, 8, 0, 32),
    (1, 4200, 40, 32), (5, 9001, 40, 128), (16, 8200, 33, 64), (40, 2048, 64, 128), (33, 2100, 100, 32), (100, 9000, 72, 64),
    (320, 1300, 2064, 128),
]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("size", INT4, ids=lambda s: "x".join(map(str, s)))
def test_linear_int4(ops, size, name):
    M, K, N, group = size
    i = INT4.index(size) + NAMES.index(name)
    a, zeros, has_b, has_r = ACTS[i % 4], i % 2 == 0, i % 3 != 0, i % 5 < 2
    pad, shift = (0, 8, 3)[i % 3], (0, 0, 8, 1)[i % 4]
    say(f"int4 {size} {name} zeros={zeros} act={a} pad={pad} shift={shift}")
    g = torch.Generator().manual_seed(i)
    d = dt(name)
    x = data(g, M, K, dtype=d) + (1.0 if i % 2 else 0.0)
    x = x.to(d).double()
    q, s, z = codes(g, K, N, group=group, dtype=d, zeros=zeros)
    b = data(g, N, dtype=d) if has_b else None
    r = data(g, M, N, dtype=d) if has_r else None
    w, sk = weight(q, s, z, group)
    packed = ops.pack_int4(q.cuda(), s.to(d).cuda(), None if z is None else z.cuda(), group_size=group)
    out = torch.full((M + 2, N + 5), 7.0, dtype=d, device="cuda")
    y = ops.linear_int4(place(x, d, pad, shift), packed, None if b is None else place(b, d, 0, shift),
                        residual=None if r is None else place(r, d, pad, shift), act=ops.ACTS[a], out=out[1:M + 1, 2:N + 2])
    pre = x @ w + (b if has_b else 0)
    want = act(pre, a) + (r if has_r else 0)
    close(y, want, int4_tol(x, w, sk, b, pre, want, a, group, name) + (0 if r is None else 4 * E32 * r.abs()), "y")
    keep = out.clone()
    keep[1:M + 1, 2:N + 2] = 7.0
    assert bool((keep == 7.0).all()), "wrote outside the output"
    if has_r:
        box = place(r, d, pad, shift)
        assert torch.equal(ops.linear_int4(place(x, d), packed, None if b is None else b.to(d).cuda(), residual=box,
                                           act=ops.ACTS[a], out=box), y)


GROUPED = [  # K, N, group, rows of each expert, rows behind
    (128, 64, 128, [1], 0), (200, 136, 64, [3, 0, 5, 1], 0), (512, 96, 32, [0, 0, 17, 2, 0], 3), (72, 40, 128, [100, 0, 90, 70], 0),
    (9000, 40, 128, [3, 0, 2], 4), (4600, 24, 32, [1, 20], 2), (2048, 64, 64, [40, 25], 9),
    (384, 130, 128, [2] * 70, 1), (64, 24, 32, [0, 0], 2), (1024, 9000, 128, [1, 4, 0, 2], 0), (136, 72, 64, [300], 20),
]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("case", range(len(GROUPED)))
def test_grouped_linear_int4(ops, case, name):
    K, N, group, counts, behind = GROUPED[case]
    i = case + NAMES.index(name)
    a, zeros, has_b = ACTS[i % 4], i % 2 == 0, i % 3 != 0
    say(f"grouped int4 {K}x{N} group {group} {counts[:6]} {name} zeros={zeros} act={a}")
    g = torch.Generator().manual_seed(i)
    d, E, T = dt(name), len(counts), sum(counts) + behind
    x = data(g, T, K, dtype=d)
    q, s, z = codes(g, E, K, N, group=group, dtype=d, zeros=zeros)
    b = data(g, E, N, dtype=d) if has_b else None
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32)
    packed = ops.pack_int4(q.cuda(), s.to(d).cuda(), None if z is None else z.cuda(), group_size=group)
    y = ops.grouped_linear_int4(place(x, d, 3, 1), packed, off.cuda(), None if b is None else b.to(d).cuda(), act=ops.ACTS[a])
    want, tol = torch.zeros(T, N, dtype=torch.float64), torch.zeros(T, N, dtype=torch.float64)
    for e, c in enumerate(counts):
        if c:
            t = slice(int(off[e]), int(off[e]) + c)
            w, sk = weight(q[e], s[e], None if z is None else z[e], group)
            be = b[e] if has_b else None
            pre = x[t] @ w + (be if has_b else 0)
            want[t] = act(pre, a)
            tol[t] = int4_tol(x[t], w, sk, be, pre, want[t], a, group, name)
    close(y, want, tol, "y")
    # offsets of any content stay in range, by the rule of grouped_linear
    wild = torch.tensor(([5, -3] + [2 ** 31 - 1, 1] * E)[:E + 1], dtype=torch.int32, device="cuda")
    wk = torch.zeros(E, K, N, dtype=d, device="cuda")
    for e in range(E):
        wk[e] = weight(q[e], s[e], None if z is None else z[e], group)[0].to(d).cuda()
    ones = torch.ones(T, K, dtype=d, device="cuda")
    same_rows = ops.grouped_linear(ones, wk, wild, act=ops.ACT_NONE).float().abs().sum(1) == 0
    assert torch.equal(ops.grouped_linear_int4(ones, packed, wild).float().abs().sum(1) == 0, same_rows)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("size", [(1, 1, 32), (100, 33, 32), (256, 40, 64), (300, 17, 128), (700, 8, 256), (0, 4, 32)])
def test_quantize_int4(ops, size, name):
    K, N, group = size
    say("quantize", size, name)
    g = torch.Generator().manual_seed(K)
    d = dt(name)
    w = data(g, 2, K, N, dtype=d) + 0.3
    w = w.to(d).double()
    w[0, :, 0] = 0.0
    for stored in (w.to(d).cuda(), w.to(d).transpose(1, 2).contiguous().cuda().transpose(1, 2)):
        for symmetric in (False, True):
            q, s, z = ops.quantize_int4(stored, group_size=group, symmetric=symmetric)
            assert q.shape == w.shape and (z is None) == symmetric and int(q.max() if K else 0) <= 15
            back, sk = weight(q.cpu(), s.double().cpu(), None if z is None else z.cpu(), group)
            # half a step; the zero point's rounding moves the range by another half, the scale's by 15 u of a step
            steps = 0.5 if symmetric else 1.0
            assert bool(((back - w).abs() <= (steps + 16 * U[name]) * sk + 1e-30).all())
            if K:
                assert not back[0, :, 0].any()
    one = ops.quantize_int4(w[1].to(d).cuda(), group_size=group)
    two = ops.quantize_int4(w.to(d).cuda(), group_size=group)
    assert torch.equal(one[0], two[0][1]) and torch.equal(one[1], two[1][1]) and torch.equal(one[2], two[2][1])


def test_int4_against_bf16_layer(ops):
    """A quantised layer and linear with the same weight in fp32: the same within both bounds."""
    say("int4 against linear")
    g = torch.Generator().manual_seed(5)
    x, w = data(g, 40, 640, dtype=torch.float32), data(g, 640, 200, dtype=torch.float32, std=0.04)
    q, s, z = ops.quantize_int4(w.float().cuda(), group_size=64)
    back, sk = weight(q.cpu(), s.double().cpu(), z.cpu(), 64)
    y = ops.linear_int4(x.float().cuda(), ops.pack_int4(q, s, z, group_size=64))
    want = ops.linear(x.float().cuda(), back.float().cuda()).double().cpu()
    close(y, want, int4_tol(x, back, sk, None, want, want, "none", 64, "f32") + 700 * E32 * (x.abs() @ back.abs()), "y")


def test_beyond_32_bits(ops):
    """Rows, codes, logits and gradients behind 2^31 elements (4-bit codes: bytes): the same as in small tensors."""
    say("beyond 32 bits")
    d = torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(6)
    # experts' codes: the last of 70, 67 MB each
    K, N, E = 8192, 16384, 70
    q = torch.zeros(E, K, N, dtype=torch.uint8, device="cuda")
    s = torch.zeros(E, K // 128, N, dtype=d, device="cuda")
    q[-1] = torch.randint(0, 16, (K, N), generator=g, device="cuda", dtype=torch.uint8)
    s[-1] = 0.01
    x = torch.randn(5, K, generator=g, device="cuda").to(d)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = 5
    one = ops.grouped_linear_int4(x, ops.pack_int4(q[-1:].clone(), s[-1:].clone()), torch.tensor([0, 5], dtype=torch.int32, device="cuda"))
    w = ops.pack_int4(q, s)
    assert w.data.numel() > 1 << 32
    del q, s
    assert torch.equal(ops.grouped_linear_int4(x, w, off), one) and one.float().abs().sum() > 0
    del w
    # rows of a large expert buffer
    T, k, D = 140000, 2, 8192
    rows = torch.randperm(T * k, generator=g, device="cuda").int().view(T, k)
    x = torch.randn(T, D, generator=g, device="cuda", dtype=d)
    gates = torch.rand(T, k, generator=g, device="cuda")
    end = torch.tensor([T * k], dtype=torch.int32, device="cuda")
    y = ops.dispatch(x, rows, end)
    assert y.numel() > 1 << 31
    last = rows.max(1).values.argsort(descending=True)[:50]
    assert torch.equal(y[rows[last].long()], x[last][:, None].expand(-1, k, -1))
    small = torch.arange(100, dtype=torch.int32, device="cuda").view(50, 2)
    part = y[rows[last].long()].reshape(100, D)
    assert torch.equal(ops.combine(y, rows, gates)[last], ops.combine(part, small, gates[last].contiguous()))
    dy, dg = ops.combine_backward(x, y, rows, end, gates)
    sy, sg = ops.combine_backward(x[last].contiguous(), part, small, torch.tensor([100], dtype=torch.int32, device="cuda"),
                                  gates[last].contiguous())
    assert torch.equal(dy[rows[last].long()].reshape(100, D), sy)
    # (a token's dot product is split over waves where tokens are few: another order of the same sum)
    assert bool(((dg[last] - sg).abs() <= 2 * (D + 8) * E32 * (x[last].float().abs()[:, None] * part.float().abs().view(50, 2, D)).sum(2)).all())
    del x, y, dy
    # logits
    T, E = 1 << 22, 520
    x = torch.zeros(T, E, dtype=d, device="cuda")
    x[-64:] = torch.randn(64, E, generator=g, device="cuda")
    r, tail = ops.route(x, 3), ops.route(x[-64:], 3)
    assert torch.equal(r.experts[-64:], tail.experts) and torch.equal(r.gates[-64:], tail.gates)
    assert r.experts[:-64].amax().item() == 2 and r.offsets[-1].item() == 3 * T
    assert torch.equal(r.rows[:-64, 1], torch.arange(T - 64, device="cuda", dtype=torch.int32) + r.offsets[1])
    dg = torch.randn(T, 3, generator=g, device="cuda")
    assert torch.equal(ops.route_backward(dg, None, x, r.experts, r.slopes)[-64:],
                       ops.route_backward(dg[-64:].contiguous(), None, x[-64:], tail.experts, tail.slopes))
    del x
    # gradients
    x = torch.zeros((1 << 31) + 1000, dtype=d, device="cuda")
    x[-1], x[5] = 3.0, 4.0
    assert ops.clip_grad_norm([x], 1.0).item() == 5.0
    assert abs(x[-1].item() - 0.6) < 0.6 * 2 ** -8 + 1e-6 and abs(x[5].item() - 0.8) < 0.8 * 2 ** -8 + 1e-6


# ----------------------------------------------------------------- clipping

def gradients(g, shapes, kinds):
    """Tensors of very different sizes, some of them views, as dense as they are."""
    out = []
    for i, (n, kind) in enumerate(zip(shapes, kinds)):
        d = dt(kind)
        if i % 4 == 1 and n > 1:        # off 16 bytes
            t = torch.zeros(n + 3, dtype=d, device="cuda")[1:n + 1]
        elif i % 4 == 2 and n % 6 == 0:  # a transposed weight's gradient
            t = torch.zeros(n // 6, 6, dtype=d, device="cuda").t()
        else:
            t = torch.zeros(n, dtype=d, device="cuda")
        t.copy_((torch.randn(t.shape, generator=g, dtype=torch.float64) * 10.0 ** (i % 5 - 2)).to(d))
        out.append(t)
    return out


CLIPS = [[1], [0, 5, 0], [7, 6, 12, 1000], [65536], [65537], [100000, 3, 0, 12345, 777777, 60000], [17] * 96, [17, 30, 6] * 70, [5, 0, 4097, 2048, 2049] * 33,
         [1 << 20, 1 << 22, 99999, 1], [0, 0]]


@pytest.mark.parametrize("case", range(len(CLIPS)))
def test_clip(ops, case):
    shapes = CLIPS[case]
    say("clip", shapes[:6], len(shapes))
    g = torch.Generator().manual_seed(case)
    kinds = [NAMES[(i + case) % 3 % 2] for i in range(len(shapes))]
    xs = gradients(g, shapes, kinds)
    ref = [x.double().cpu() for x in xs]
    norm = math.sqrt(math.fsum(float((x * x).sum()) for x in ref))
    got = ops.grad_norm(xs)
    assert got.shape == () and abs(got.item() - norm) <= 2 * E32 * norm
    assert all(torch.equal(a.double().cpu(), b) for a, b in zip(xs, ref))
    for most in (0.5 * norm, 0.0, 2.0 * norm + 1.0, math.inf):
        f = min(1.0, most / (norm + 1e-6)) if most < math.inf else 1.0
        for to in (NAMES[case % 2], None):
            if to is None:
                outs, back = [x.clone(memory_format=torch.preserve_format) for x in xs], None
                back = ops.clip_grad_norm(outs, most)
            else:
                outs = [torch.full_like(x, 7.0, dtype=dt(to), memory_format=torch.preserve_format) for x in xs]
                back = ops.clip_grad_norm(xs, most, out=outs)
            assert torch.equal(back, got)
            for x, o in zip(ref, outs):
                u = 2.0 ** -8 if o.dtype == torch.bfloat16 else 2.0 ** -24
                if f == 1.0:
                    assert torch.equal(o.cpu(), x.to(o.dtype))
                else:
                    close(o, x * f, (1.01 * u + 6 * E32) * (x * f).abs() + 2.0 ** -133, "scaled")


def test_clip_special_values(ops):
    say("clip special values")
    big = torch.full((100000,), 1e30, device="cuda")        # squares beyond fp32
    tiny = torch.full((5,), 1e-30, device="cuda")
    n = ops.grad_norm([big, tiny]).item()
    assert abs(n - 1e30 * math.sqrt(1e5)) < 1e-6 * n
    assert abs(ops.grad_norm([tiny]).item() - 1e-30 * math.sqrt(5)) < 1e-36
    out = [torch.zeros_like(big)]
    ops.clip_grad_norm([big], 1.0, out=out)
    assert abs(out[0].double().norm().item() - 1.0) < 1e-5
    for bad, factor in ((math.inf, 0.0), (math.nan, math.nan)):
        for n in (10, 200000):
            x = torch.ones(n, device="cuda")
            x[n // 2] = bad
            norm = ops.clip_grad_norm([x], 1.0)
            assert norm.item() == bad or (math.isnan(bad) and norm.isnan())
            assert x[n // 2].isnan() and (x[0].item() == factor or (math.isnan(factor) and x[0].isnan()))
            ops.clip_grad_norm([x], math.inf)


# ------------------------------------------------------------------ together

def step(ops, x, wr, w1, w2, dy, packed, k):
    """A routed block's forward and backward pass, a decode pass, and clipping."""
    logits = ops.linear(x, wr)
    r = ops.route(logits, k, normalize=True)
    rows = ops.dispatch(x, r.rows, r.offsets)
    h, z = ops.grouped_linear(rows, w1, r.offsets, act=ops.ACT_SILU, need_pre=True)
    o = ops.grouped_linear(h, w2, r.offsets)
    y = ops.combine(o, r.rows, r.gates, residual=x)
    do, dg = ops.combine_backward(dy, o, r.rows, r.offsets, r.gates)
    dh, dw2, _ = ops.grouped_linear_backward(do, h, w2, r.offsets, need_bias=False)
    dr, dw1, _ = ops.grouped_linear_backward(dh, rows, w1, r.offsets, pre=z, act=ops.ACT_SILU, need_bias=False)
    dl = ops.route_backward(dg, torch.ones((), device="cuda"), logits, r.experts, r.slopes, normalize=True)
    dxr, dwr, _ = ops.linear_backward(dl, x, wr, need_bias=False)
    dx = ops.combine(dr, r.rows, residual=dxr)
    norm = ops.clip_grad_norm([dw1, dw2, dwr], 0.1)
    q = ops.grouped_linear_int4(rows, packed, r.offsets, act=ops.ACT_SILU)
    return (*r, y, dx, dw1, dw2, dwr, norm, q)


def test_streams_and_graphs(ops):
    """The same bits on another stream, and in replays of a captured step between eager work."""
    say("streams and graphs")
    d = torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(9)

    def normal(*s, std=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * std).to(d)
    T, D, H, E, k = 700, 136, 200, 6, 2
    x, wr, w1, w2, dy = normal(T, D), normal(D, E), normal(E, D, H, std=0.1), normal(E, H, D, std=0.1), normal(T, D)
    packed = ops.pack_int4(*ops.quantize_int4(w1, group_size=32), group_size=32)
    want = [v.clone() for v in step(ops, x, wr, w1, w2, dy, packed, k)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(ops, x, wr, w1, w2, dy, packed, k)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(ops, x, wr, w1, w2, dy, packed, k)
    for i in range(3):
        for v in held:
            v.zero_()
        step(ops, normal(T, D), wr, w1, w2, dy, packed, k)  # eager work between the replays
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), i


def test_results_repeat(ops):
    """Sums whose order could depend on timing: the same bits every time."""
    say("repeats")
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(30000, 100, generator=g, device="cuda")
    r = ops.route(x, 4)
    grads = [torch.randn(n, generator=g, device="cuda") for n in (5000001, 333, 70000)]
    n = ops.grad_norm(grads)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(ops.route(x, 4), r))
        assert torch.equal(ops.grad_norm(grads), n)


# -------------------------------------------------------- outputs and refusals

def test_out_is_marked_as_written(ops):
    say("versions")
    d = torch.bfloat16
    x = torch.ones(4, 8, dtype=d, device="cuda")
    rows = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    w = ops.pack_int4(*ops.quantize_int4(torch.ones(8, 8, dtype=d, device="cuda"), group_size=32), group_size=32)
    w3 = ops.pack_int4(*ops.quantize_int4(torch.ones(1, 8, 8, dtype=d, device="cuda"), group_size=32), group_size=32)
    off4 = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    calls = {(8, 8): [lambda o: ops.dispatch(x, rows, off, out=o), lambda o: ops.clip_grad_norm([o], 1.0),
                      lambda o: ops.clip_grad_norm([torch.ones_like(o)], 1.0, out=[o])],
             (4, 8): [lambda o: ops.combine(torch.ones(8, 8, dtype=d, device="cuda"), rows, out=o),
                      lambda o: ops.linear_int4(x, w, out=o), lambda o: ops.grouped_linear_int4(x, w3, off4, out=o)]}
    for shape, fs in calls.items():
        for f in fs:
            buf = torch.zeros(*shape, dtype=d, device="cuda")
            before = buf._version
            f(buf)
            assert buf._version > before
            leaf = torch.zeros(*shape, dtype=d, device="cuda", requires_grad=True)
            with pytest.raises(RuntimeError):
                f(leaf)
            with torch.no_grad():
                f(leaf)


def test_routing_tensors_are_ordinary(ops):
    """They come from one allocation: each is written, copied and differentiated like any other."""
    say("routing tensors")
    x = torch.randn(300, 40, device="cuda")
    r, want = ops.route(x, 4), ops.route(x, 4)
    r.counts.add_(1)
    r.experts.fill_(-7)
    r.loss.zero_()
    for name in ("gates", "rows", "offsets", "slopes"):
        assert torch.equal(getattr(r, name), getattr(want, name)), name
    for v in want:
        assert v.is_contiguous() and v._version == 0 and torch.equal(v.clone().cpu(), v.cpu()) and not v._is_view()
    gates = want.gates.requires_grad_()
    (gates * 3).sum().backward()
    assert (gates.grad == 3).all()
    assert not ops.route_backward(None, None, x, want.experts, want.slopes).any()
    with torch.inference_mode():
        assert torch.equal(ops.route(x, 4).rows, want.rows)


def test_refusals(ops):
    say("refusals")
    d = torch.bfloat16

    def new(*s, dtype=d):
        return torch.zeros(s, dtype=dtype, device="cuda")
    i32, f32 = torch.int32, torch.float32
    x, rows, off = new(4, 8), new(4, 2, dtype=i32), new(3, dtype=i32)
    y, gates = new(8, 8), new(4, 2, dtype=f32)
    q, s = new(64, 8, dtype=torch.uint8), new(2, 8)
    w = ops.pack_int4(q, s, group_size=32)
    x64 = new(4, 64)
    w3 = ops.pack_int4(q[None], s[None], group_size=32)
    for error, call in [
        (TypeError, lambda: ops.route(torch.zeros(4, 8), 2)),
        (ValueError, lambda: ops.route(new(4, 8, dtype=torch.float16), 2)),
        (ValueError, lambda: ops.route(new(8), 2)),
        (ValueError, lambda: ops.route(x, 0)),
        (ValueError, lambda: ops.route(x, 9)),
        (ValueError, lambda: ops.route(x, (1 << 32) + 1)),
        (ValueError, lambda: ops.route(new(4, 64), 33)),
        (ValueError, lambda: ops.route(new(2, 1025), 2)),
        (ValueError, lambda: ops.route(new(2, 0), 1)),
        (ValueError, lambda: ops.route(x, 2, valid=new(4))),
        (ValueError, lambda: ops.route(x, 2, valid=new(5, dtype=torch.bool))),
        (ValueError, lambda: ops.route(new(8, 4).t(), 2)),
        (ValueError, lambda: ops.route_backward(gates, None, x, rows[:3], None)),
        (ValueError, lambda: ops.route_backward(gates.to(d), None, x, rows, None)),
        (ValueError, lambda: ops.route_backward(gates, new(1, dtype=f32), x, rows, new(8, dtype=f32))),
        (ValueError, lambda: ops.route_backward(gates, new(dtype=f32), x, rows, new(7, dtype=f32))),
        (ValueError, lambda: ops.route_backward(gates, None, x, rows.long(), None)),
        (ValueError, lambda: ops.dispatch(x, rows.long(), off)),
        (ValueError, lambda: ops.dispatch(x, rows[:3], off)),
        (ValueError, lambda: ops.dispatch(x, rows, off.long())),
        (ValueError, lambda: ops.dispatch(x, rows, new(0, dtype=i32))),
        (ValueError, lambda: ops.dispatch(x, rows, off, out=new(8, 9))),
        (ValueError, lambda: ops.dispatch(x, rows, off.cpu())),
        (RuntimeError, lambda: ops.dispatch(y[:4], rows, off, out=y)),
        (RuntimeError, lambda: ops.dispatch(x, new(4, 33, dtype=i32), off)),
        (ValueError, lambda: ops.combine(y, rows, gates.to(d))),
        (ValueError, lambda: ops.combine(y, rows, gates[:3])),
        (ValueError, lambda: ops.combine(y, rows, residual=new(3, 8))),
        (ValueError, lambda: ops.combine(y, rows.t())),
        (RuntimeError, lambda: ops.combine(y, rows, out=y[2:6])),
        (ValueError, lambda: ops.combine_backward(x, new(8, 7), rows, off, gates)),
        (ValueError, lambda: ops.combine_backward(x, y.float(), rows, off, gates)),
        (ValueError, lambda: ops.quantize_int4(x, group_size=16)),
        (ValueError, lambda: ops.quantize_int4(x, group_size=96)),
        (ValueError, lambda: ops.quantize_int4(x.half())),
        (TypeError, lambda: ops.quantize_int4(torch.zeros(4, 4))),
        (ValueError, lambda: ops.quantize_int4(new(8))),
        (ValueError, lambda: ops.pack_int4(q.int(), s, group_size=32)),
        (ValueError, lambda: ops.pack_int4(q, s, group_size=64)),
        (ValueError, lambda: ops.pack_int4(q, s, s, group_size=32)),
        (ValueError, lambda: ops.pack_int4(q.t(), s, group_size=32)),
        (TypeError, lambda: ops.linear_int4(x64, q)),
        (TypeError, lambda: ops.linear_int4(None, w)),
        (TypeError, lambda: ops.linear_int4(x64.cpu(), w)),
        (ValueError, lambda: ops.linear_int4(x64[0], w)),
        (ValueError, lambda: ops.linear_int4(x64.float(), w)),
        (ValueError, lambda: ops.linear_int4(new(4, 65), w)),
        (ValueError, lambda: ops.linear_int4(x64, w3)),
        (ValueError, lambda: ops.linear_int4(x64, w._replace(data=w.data[1:]))),
        (ValueError, lambda: ops.linear_int4(x64, w._replace(group_size=64))),
        (ValueError, lambda: ops.linear_int4(x64, w, bias=new(7))),
        (ValueError, lambda: ops.linear_int4(x64, w, act=1 << 32)),
        (RuntimeError, lambda: ops.linear_int4(x64, w, act=9)),
        (RuntimeError, lambda: ops.linear_int4(x64, w, out=x64[:, :8])),
        (ValueError, lambda: ops.grouped_linear_int4(x64, w, off)),
        (ValueError, lambda: ops.grouped_linear_int4(x64, w3, off)),
        (ValueError, lambda: ops.grouped_linear_int4(x64, w3, off[:2].long())),
        (ValueError, lambda: ops.grad_norm([])),
        (TypeError, lambda: ops.grad_norm([None])),
        (TypeError, lambda: ops.grad_norm(3)),
        (TypeError, lambda: ops.grad_norm([torch.zeros(3)])),
        (ValueError, lambda: ops.grad_norm([new(4, 4)[:, :2]])),
        (ValueError, lambda: ops.grad_norm([new(4).half()])),
        (RuntimeError, lambda: ops.clip_grad_norm([x], -1.0)),
        (RuntimeError, lambda: ops.clip_grad_norm([x], math.nan)),
        (RuntimeError, lambda: ops.clip_grad_norm([x, x], 1.0)),
        (RuntimeError, lambda: ops.clip_grad_norm([y[:4], y[3:]], 1.0)),
        (RuntimeError, lambda: ops.clip_grad_norm([x, y], 1.0, out=[y[:4], new(8, 8)])),
        (ValueError, lambda: ops.clip_grad_norm([x], 1.0, out=[])),
        (ValueError, lambda: ops.clip_grad_norm([x], 1.0, out=[new(8, 4)])),
        (ValueError, lambda: ops.clip_grad_norm([x], 1.0, out=[new(8, 4).t()])),
    ]:
        with pytest.raises(error):
            call()
    assert ops.clip_grad_norm([x, x.clone()], 1.0, out=[x, new(4, 8)]).item() == 0.0
    assert ops.grad_norm([x, x]).item() == 0.0    # read only: the same tensor twice is taken twice
