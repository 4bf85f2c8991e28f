"""GPU tests of the feed-forward operators at row counts whose launches would have
2^32 threads or more with one thread or block to a fixed number of rows.  A
grid's dimension holds fewer, so such a launch is made in parts or over two
dimensions, and its results have to be those of any other.

Sizes of up to 69 GB; inputs are random where the whole result is compared, by
ranges of rows on the device in 64 bits, and otherwise zero but for some rows.
Tolerances are those of test_gpu_ops.py: with e = 2^-24 and u the unit roundoff
of the stored type, a sum of K products is off by at most (K + 8) e sum |a||b|,
a row's mean and deviation by (N + 16) e relative, the stored value by u."""
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

E32 = 2.0 ** -24
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ops():
    from tile_dependency_pipelined_amd import ops as o
    assert torch.cuda.is_available()
    yield o
    torch.cuda.empty_cache()


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def parts(M, step=1 << 23):
    return [slice(r, min(r + step, M)) for r in range(0, M, step)]


def check_norm(x, w, b, eps, y, mean, rstd, name):
    N = x.shape[1]
    w, b = w.double(), b.double()
    for s in parts(x.shape[0]):
        v = x[s].double()
        mu = v.mean(1, keepdim=True)
        var = ((v - mu) ** 2).mean(1, keepdim=True)
        rs = (var + eps) ** -0.5
        n = (N + 16) * E32
        off = n * v.abs().mean(1, keepdim=True)
        rel = n + 2 * off * off / (var + eps) + 8 * E32
        assert bool(((mean[s].double() - mu[:, 0]).abs() <= off[:, 0] + E32 * mu[:, 0].abs()).all()), ("mean", s)
        assert bool(((rstd[s].double() - rs[:, 0]).abs() <= (rel * rs)[:, 0]).all()), ("rstd", s)
        xh = (v - mu) * rs
        want = xh * w + b
        tol = (off * rs + xh.abs() * (rel + 4 * E32)) * w.abs() + (1.01 * U[name] + 4 * E32) * want.abs() + 4 * E32 * b.abs()
        assert bool(((y[s].double() - want).abs() <= tol).all()), ("y", s)


# Narrow rows: 4 elements, far more rows than blocks of 1024 threads fit a grid;
# 8 elements (a unit of 16 bytes in bf16), more than waves fit.
@pytest.mark.parametrize("name, M, N", [("bf16", (1 << 22) + 3, 4), ("bf16", (1 << 26) + 5, 8), ("f32", (1 << 26) + 5, 4),
                                        ("bf16", (1 << 26) + 5, 3)])
def test_layer_norm_of_many_rows(ops, name, M, N):
    say(f"layer_norm {M} x {N} {name}")
    g = torch.Generator(device="cuda").manual_seed(N)
    x = torch.empty(M, N, dtype=DTYPES[name], device="cuda")
    for s in parts(M):
        x[s] = torch.randn(x[s].shape, generator=g, device="cuda") + 2.0
    w, b = (torch.randn(N, generator=g, device="cuda").to(x.dtype) for _ in range(2))
    y, mean, rstd = ops.layer_norm(x, w, b, eps=1e-3)
    check_norm(x, w, b, 1e-3, y, mean, rstd, name)


@pytest.mark.parametrize("N", range(1, 8))
def test_layer_norm_narrower_than_a_unit(ops, N):
    """Rows of fewer elements than 16 bytes hold, with NaN around them, and in place."""
    say(f"layer_norm 1003 x {N} bf16")
    g = torch.Generator(device="cuda").manual_seed(N)
    box = torch.full((1005, N + 3), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = box[1:-1, 2:2 + N]
    x.copy_(torch.randn(1003, N, generator=g, device="cuda") + 1.0)
    w, b = (torch.randn(N, generator=g, device="cuda").to(x.dtype) for _ in range(2))
    y, mean, rstd = ops.layer_norm(x, w, b, eps=1e-3)
    check_norm(x, w, b, 1e-3, y, mean, rstd, "bf16")
    ops.layer_norm(x, w, b, eps=1e-3, out=x)
    assert torch.equal(x, y)
    x.fill_(float("nan"))
    assert bool(box.isnan().all()), "wrote outside the rows"


def test_layer_norm_backward_of_many_long_rows(ops):
    """Rows that do not fit the registers, a block of 1024 threads each."""
    M, N, some = (1 << 22) + 3, 8193, [0, 1, (1 << 22) - 2, (1 << 22) - 1, 1 << 22, (1 << 22) + 2]
    say(f"layer_norm_backward {M} x {N} bf16")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")  # dy as well: two inputs may be the same
    v = torch.randn(len(some), N, generator=g, device="cuda").to(x.dtype)
    x[some] = v
    mean, rstd = torch.full((M,), 0.25, device="cuda"), torch.full((M,), 0.5, device="cuda")
    dx = ops.layer_norm_backward(x, x, mean, rstd, need_weight=False, need_bias=False)[0]
    v = v.double()
    xh = (v - 0.25) * 0.5
    s0, s1 = v.mean(1, keepdim=True), (v * xh).mean(1, keepdim=True)
    want = 0.5 * (v - s0 - xh * s1)
    n = (N + 16) * E32
    tol = 0.5 * (n * v.abs().mean(1, keepdim=True) + xh.abs() * n * (v * xh).abs().mean(1, keepdim=True)
                 + 8 * E32 * (v.abs() + s0.abs() + (xh * s1).abs())) + 1.01 * U["bf16"] * want.abs()
    assert bool(((dx[some].double() - want).abs() <= tol).all())
    dx[some] = 0.0
    # a row of zeros has the gradient zero
    assert not any(bool(dx[s].any()) for s in parts(M, 1 << 18))


def check_product(x, w, b, y, name):
    w, b = w.double(), b.double()
    for s in parts(x.shape[0]):
        v = x[s].double()
        want = v @ w + b
        tol = (x.shape[1] + 8) * E32 * (v.abs() @ w.abs() + b.abs()) + 1.01 * U[name] * want.abs()
        assert bool(((y[s].double() - want).abs() <= tol).all()), s


def test_linear_of_many_unaligned_rows(ops):
    """The copies that put rows of 14 bytes into whole units, four rows to a block."""
    M, K, N = (1 << 26) + 5, 7, 8
    say(f"linear {M} x {K} x {N} bf16")
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    for s in parts(M):
        x[s] = torch.randn(x[s].shape, generator=g, device="cuda")
    w, b = torch.randn(K, N, generator=g, device="cuda").to(x.dtype), torch.randn(N, generator=g, device="cuda").to(x.dtype)
    check_product(x, w, b, ops.linear(x, w, b), "bf16")
    off = torch.tensor([0, 3, M], dtype=torch.int32, device="cuda")
    y = ops.grouped_linear(x, torch.stack([w, -w]), off, torch.stack([b, -b]))
    check_product(x[:3], w, b, y[:3], "bf16")
    check_product(x[3:], w, b, -y[3:], "bf16")


def test_linear_of_a_billion_rows(ops):
    """64 x 64 tiles, the cheapest for such narrow products, are more than a grid holds."""
    M, K, N = 1 << 30, 4, 8
    say(f"linear {M} x {K} x {N} fp32")
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.zeros(M, K, device="cuda")
    some = [0, 1, 4095, M // 2 - 1, M // 2, M - 2, M - 1]
    x[some] = torch.randn(len(some), K, generator=g, device="cuda")
    w, b = torch.randn(K, N, generator=g, device="cuda"), torch.zeros(N, device="cuda")
    y = ops.linear(x, w, b)
    check_product(x[some], w, b, y[some], "f32")
    y[some] = 0.0
    assert not any(bool(y[s].any()) for s in parts(M, 1 << 26))


@pytest.mark.parametrize("act", ["none", "relu"])
def test_bias_gradient_of_many_rows(ops, act):
    """A block to each 32 rows: small integers, whose sums are exact."""
    M, N = (1 << 29) + 5, 3
    say(f"bias gradient {M} x {N} bf16 {act}")
    dy = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    some = [0, 31, 32, 1 << 28, (1 << 29) - 1, 1 << 29, M - 1]
    dy[some] = torch.tensor([[i + 1.0, 2.0 * i, -i - 3.0] for i in range(len(some))], device="cuda").to(dy.dtype)
    want = dy[some].float().sum(0)
    x, w = torch.zeros(M, 1, dtype=dy.dtype, device="cuda"), torch.zeros(1, N, dtype=dy.dtype, device="cuda")
    pre = None if act == "none" else torch.ones(M, N, dtype=dy.dtype, device="cuda")
    db = ops.linear_backward(dy, x, w, pre=pre, act=ops.ACTS[act], need_x=False, need_w=False)[2]
    assert torch.equal(db.float(), want)
