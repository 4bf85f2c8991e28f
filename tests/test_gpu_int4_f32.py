"""GPU tests of 4-bit layers of fp32 rows where the weight is small beside its codes: a
code that equals its zero point is a weight of 0 and adds nothing, so the result is as
good as that of the weight itself.

Tolerance: each product of x (three bf16 parts of 8 bits) with a code less its zero point
(5 bits) is exact, and so is every sum over them while it is of one part and fits 24
bits; else a sum of n terms is within n e of the sum of their magnitudes, e = 2^-24,
n = 3 K; scaling, the sum over groups and waves and the output add K / 32 + 40."""
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
E32 = 2.0 ** -24


@pytest.fixture(scope="module")
def ops():
    from tile_dependency_pipelined_amd import ops as o
    assert torch.cuda.is_available()
    return o


def say(*a):
    print(*a, file=sys.stderr, flush=True)


SIZES = [(1, 128, 32, 128), (1, 4096, 64, 128), (3, 1000, 40, 32), (13, 2100, 33, 64), (16, 9001, 48, 128), (17, 512, 64, 32),
         (40, 1300, 72, 64), (100, 2048, 136, 128), (300, 4097, 130, 256)]


@pytest.mark.parametrize("zeros", [True, False], ids=["zeros", "symmetric"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_weights_of_zero(ops, size, zeros):
    M, K, N, group = size
    say("int4 fp32 zero weights", size, zeros)
    g = torch.Generator().manual_seed(K + zeros)
    G = -(-K // group)
    x = torch.rand(M, K, generator=g) + 0.5             # of one sign, as behind an activation
    s = (0.5 + torch.rand(G, N, generator=g)) * 0.02
    z = torch.randint(0, 16, (G, N), generator=g, dtype=torch.uint8) if zeros else None
    spread = torch.arange(K) // group
    zk = z[spread] if zeros else torch.full((K, N), 8, dtype=torch.uint8)
    q = zk.clone()
    at = torch.randint(0, K, (N,), generator=g)         # one weight of every other column is not 0
    cols = torch.arange(0, N, 2)
    q[at[cols], cols] = torch.randint(0, 16, (len(cols),), generator=g, dtype=torch.uint8)
    w = s.double()[spread] * (q.double() - zk.double())
    y = ops.linear_int4(x.cuda(), ops.pack_int4(q.cuda(), s.cuda(), None if z is None else z.cuda(), group_size=group))
    y = y.double().cpu()
    want, size_ = x.double() @ w, x.double().abs() @ w.abs()
    assert not y[:, 1::2].any()
    assert bool(((y - want).abs() <= (3 * K + K / 32 + 40) * E32 * size_).all())
    # a single product: three exact partial products and few roundings
    assert bool(((y - want).abs() <= 8 * E32 * size_).all())


def test_experts_of_zero_weights(ops):
    say("int4 fp32 zero weights by expert")
    g = torch.Generator().manual_seed(2)
    counts, K, N, group = [3, 0, 40, 1], 300, 56, 32
    z = torch.randint(0, 16, (4, -(-K // group), N), generator=g, dtype=torch.uint8)
    s = torch.rand(z.shape, generator=g) + 0.5
    q = z[:, torch.arange(K) // group]
    x = torch.rand(sum(counts) + 2, K, generator=g) + 0.5
    off = torch.tensor([0, 3, 3, 43, 44], dtype=torch.int32)
    y = ops.grouped_linear_int4(x.cuda(), ops.pack_int4(q.cuda().contiguous(), s.cuda(), z.cuda(), group_size=group), off.cuda())
    assert not y.any()


# A group of 128 is a sum of 384 products, each step of which is off by e / sqrt(3) of the sum
# so far, in the mean; with the errors of groups independent of each other and the sum so far at most
# as large as the group's (centred codes, so that both grow alike), sqrt(384 / 3) e = 11.3 e of the
# result's 2-norm.  Adding up 32 groups gives sqrt(32 / 3) e more, together 11.8 e.  Half as much again.
@pytest.mark.parametrize("shift", [0.0, 3.0])
@pytest.mark.parametrize("M, K, N", [(1, 4096, 512), (13, 4096, 512), (64, 2048, 256)])
def test_error_of_the_sum(ops, M, K, N, shift):
    say("int4 fp32 error", M, K, N, shift)
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, K, generator=g) + shift
    q = torch.randint(0, 16, (K, N), generator=g, dtype=torch.uint8)
    z = torch.randint(5, 11, (K // 128, N), generator=g, dtype=torch.uint8)
    s = torch.full((K // 128, N), 2.0 ** -6)
    want = x.double() @ (2.0 ** -6 * (q.double() - z.double()[torch.arange(K) // 128]))
    y = ops.linear_int4(x.cuda(), ops.pack_int4(q.cuda(), s.cuda(), z.cuda(), group_size=128)).double().cpu()
    err = ((y - want).norm() / want.norm()).item()
    say(f"off {err:.2e}")
    assert err <= 18 * E32
