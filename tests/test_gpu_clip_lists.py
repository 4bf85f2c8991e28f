"""GPU tests of the lists that clip_grad_norm takes: any iterable, gone through once."""
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


def tensors(n):
    g = torch.Generator(device="cuda").manual_seed(n)
    return [torch.randn(100 + 37 * i, generator=g, device="cuda") for i in range(n)]


KINDS = {"list": list, "tuple": tuple, "generator": lambda v: (t for t in v), "map": lambda v: map(lambda t: t, v),
         "iterator": iter, "dict": lambda v: dict(enumerate(v)).values()}


@pytest.mark.parametrize("n", [1, 5, 200])
@pytest.mark.parametrize("kind", KINDS)
def test_out_of_any_iterable(ops, kind, n):
    say("clip into", kind, n)
    xs, make = tensors(n), KINDS[kind]
    want = [torch.empty_like(x) for x in xs]
    norm = ops.clip_grad_norm(xs, 0.5, out=want)
    outs = [torch.empty_like(x, dtype=torch.bfloat16 if i % 2 else torch.float32) for i, x in enumerate(xs)]
    before = [t._version for t in outs]
    assert torch.equal(ops.clip_grad_norm(make(xs), 0.5, out=make(outs)), norm)
    for o, w, v in zip(outs, want, before):
        assert torch.equal(o, w if o.dtype == torch.float32 else w.to(o.dtype)) and o._version > v
    assert torch.equal(ops.grad_norm(make(xs)), norm)
    versions = [x._version for x in xs]
    assert torch.equal(ops.clip_grad_norm(make(xs), 0.5), norm)     # in place
    assert all(torch.equal(x, w) and x._version > v for x, w, v in zip(xs, want, versions))


def test_out_made_by_its_iterator(ops):
    """Tensors that nothing but the iterator's own list, or nothing at all, refers to."""
    say("clip into new tensors")
    xs = tensors(20)
    want = [torch.empty_like(x) for x in xs]
    norm = ops.clip_grad_norm(xs, 0.5, out=want)
    kept = []

    def fresh():
        for x in xs:
            kept.append(torch.empty_like(x))
            yield kept[-1]
    assert torch.equal(ops.clip_grad_norm(xs, 0.5, out=fresh()), norm)
    assert all(torch.equal(a, b) for a, b in zip(kept, want))
    for _ in range(3):      # written and dropped: the norm has memory of its own
        assert torch.equal(ops.clip_grad_norm((x.clone() for x in xs), 0.5, out=(torch.empty_like(x) for x in xs)), norm)


def test_lists_that_change(ops):
    """What is read is what the lists held when the call began."""
    say("clip of changing lists")
    xs = tensors(6)
    norm = ops.grad_norm(xs)
    grads = list(xs)

    class Most:
        def __float__(self):
            grads.clear()
            return 0.5

    outs = [torch.empty_like(x) for x in xs]
    assert torch.equal(ops.clip_grad_norm(grads, Most(), out=outs), norm) and not grads

    def clearing():
        grads.clear()
        yield from outs
    grads = list(xs)
    assert torch.equal(ops.clip_grad_norm(grads, 0.5, out=clearing()), norm) and not grads


def test_iterator_refusals(ops):
    say("clip list refusals")
    xs = tensors(3)
    fails, before = (1 / 0 for _ in xs), [x._version for x in xs]
    for error, call in [
        (ValueError, lambda: ops.clip_grad_norm(xs, 1.0, out=(t for t in xs[:2]))),
        (ValueError, lambda: ops.clip_grad_norm((t for t in xs[:2]), 1.0, out=xs)),
        (ValueError, lambda: ops.clip_grad_norm(iter([]), 1.0)),
        (TypeError, lambda: ops.clip_grad_norm(xs, 1.0, out=7)),
        (TypeError, lambda: ops.clip_grad_norm(xs, 1.0, out=(None for _ in xs))),
        (ZeroDivisionError, lambda: ops.clip_grad_norm(xs, 1.0, out=fails)),
    ]:
        with pytest.raises(error):
            call()
    assert [x._version for x in xs] == before
