"""GPU tests of `out` arguments and of what autograd sees: a tensor that a call
writes is marked as changed, one that requires a gradient is refused while
gradients are recorded, and `out` may share memory only where the operator
allows it."""
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ops():
    from tile_dependency_pipelined_amd import ops as o
    assert torch.cuda.is_available()
    return o


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def calls(ops, d=torch.bfloat16):
    """Each call with `out`: a function of the tensor to write."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = (torch.randn(*s, generator=g, device="cuda").to(d) for s in ((24, 64), (64, 64)))
    off = torch.tensor([0, 10, 24], dtype=torch.int32, device="cuda")
    return {"linear": lambda out: ops.linear(x, w, out=out),
            "grouped_linear": lambda out: ops.grouped_linear(x, torch.stack([w, w]), off, out=out),
            "layer_norm": lambda out: ops.layer_norm(x, out=out)[0]}


@pytest.mark.parametrize("name", ["linear", "grouped_linear", "layer_norm"])
def test_out_is_marked_as_written(ops, name):
    say("version", name)
    call = calls(ops)[name]
    buf = torch.zeros(24, 64, dtype=torch.bfloat16, device="cuda")
    before = buf._version
    assert call(buf).data_ptr() == buf.data_ptr()
    assert buf._version > before
    # a tensor saved for a gradient and then overwritten: the gradient is refused, not wrong
    leaf = torch.ones_like(buf, requires_grad=True)
    y = (leaf * buf).sum()
    call(buf)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


@pytest.mark.parametrize("name", ["linear", "grouped_linear", "layer_norm"])
def test_out_that_requires_a_gradient(ops, name):
    say("requires_grad", name)
    call = calls(ops)[name]
    want = call(None)
    buf = torch.zeros(24, 64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    with pytest.raises(RuntimeError, match="out"):
        call(buf)
    assert not buf.detach().any()
    with torch.no_grad():
        call(buf)
    assert torch.equal(buf.detach(), want)


@pytest.mark.parametrize("name", ["linear", "grouped_linear", "layer_norm"])
def test_out_made_in_inference_mode(ops, name):
    """Such tensors have no version; autograd cannot have saved them."""
    say("inference", name)
    call = calls(ops)[name]
    want = call(None)
    with torch.inference_mode():
        buf = torch.zeros(24, 64, dtype=torch.bfloat16, device="cuda")
        call(buf)
    assert torch.equal(buf, want)
    buf2 = call(buf)
    assert torch.equal(buf2, want)


def test_out_that_overlaps_an_input(ops):
    """Refused: other workgroups still read what such a call writes."""
    say("overlap")
    d = torch.bfloat16
    M = N = K = 64
    pool = torch.zeros(4 * M, 4 * N, dtype=d, device="cuda")
    x, w, r = (torch.randn(M, N, device="cuda").to(d) for _ in range(3))
    b = torch.zeros(N, dtype=d, device="cuda")
    off = torch.tensor([0, 40, 64], dtype=torch.int32, device="cuda")
    w2 = torch.stack([w, w])
    shifted = pool[1:M + 1, :N]
    bad = [
        lambda: ops.linear(x, w, out=x),
        lambda: ops.linear(x, w, out=w),
        lambda: ops.linear(x, w.t(), out=w),
        lambda: ops.linear(pool[:M, :K], w, out=pool[M - 1:2 * M - 1, :N]),
        lambda: ops.linear(pool[:M, :K], w, out=pool[:M, K - 1:K - 1 + N]),
        lambda: ops.linear(x, w, residual=pool[:M, :N], out=shifted),
        lambda: ops.linear(x[:1], w, b, out=b[None]),
        lambda: ops.grouped_linear(x, w2, off, out=x),
        lambda: ops.grouped_linear(x, w2, off, out=w2[1]),
        lambda: ops.layer_norm(pool[:M, :N], out=shifted),
        lambda: ops.layer_norm(x, w[0], out=w),
        lambda: ops.layer_norm(x, None, w[63], out=w),
    ]
    for i, call in enumerate(bad):
        say("overlap", i)
        with pytest.raises(RuntimeError, match="overlap"):
            call()


def test_out_beside_an_input(ops):
    """Views of one buffer that share no element, and the tensors that `out` may be."""
    say("views side by side")
    d = torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(3)
    M, N = 40, 64
    pool = torch.randn(2 * M, 3 * N, generator=g, device="cuda").to(d)
    w = torch.randn(N, N, generator=g, device="cuda").to(d)
    for x, out in ((pool[:M, :N], pool[:M, N:2 * N]), (pool[:M, :N], pool[M:, :N]), (pool[::2, :N], pool[1::2, :N]),
                   (pool[::2, :N], pool[1::2, N:2 * N])):
        want = ops.linear(x.clone(), w)
        ops.linear(x, w, out=out)
        assert torch.equal(out, want)
        want = ops.layer_norm(x.clone())[0]
        ops.layer_norm(x, out=out)
        assert torch.equal(out, want)
    x, r = pool[:M, :N], pool[:M, N:2 * N]
    want = ops.linear(x, w, residual=r.clone())
    ops.linear(x, w, residual=r, out=r)
    assert torch.equal(r, want)
    want = ops.layer_norm(x.clone())[0]
    ops.layer_norm(x, out=x)
    assert torch.equal(x, want)
