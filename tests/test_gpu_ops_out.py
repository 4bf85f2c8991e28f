"""GPU tests of `out` arguments and of what autograd sees: a tensor that a call
writes is marked as changed, and one that requires a gradient is refused while
gradients are recorded."""
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
