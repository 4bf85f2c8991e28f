"""GPU tests of clip_grad_norm with thousands of tensors: their partial sums come from
many launches.  Tolerances: the norm is summed in 64 bits and rounded once to fp32, the
factor and the scaled value are rounded once each; u is half a step of the output's
type."""
import math
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


def views(n, size, dtype, fill=None):
    buf = torch.empty(n * size, dtype=dtype, device="cuda")
    if fill is None:
        buf.normal_(generator=torch.Generator(device="cuda").manual_seed(n))
    else:
        buf.fill_(fill)
    return buf, list(buf.detach().view(n, size).unbind(0))


# launches of 160 tensors with a partial sum to each chunk, up to 1024 of them: below, at and
# beyond the 2048 sums that are added up by every block, and uneven last launches
@pytest.mark.parametrize("n, size", [(321, 5000), (2048, 7), (2049, 7), (2100, 1), (321, 30000), (5003, 300), (700, 40001)])
@pytest.mark.parametrize("name", ["bf16", "f32"])
def test_many_tensors(ops, n, size, name):
    say("clip of many tensors", n, size, name)
    dtype = torch.bfloat16 if name == "bf16" else torch.float32
    x, xs = views(n, size, dtype)
    ref = x.double()
    norm = ref.norm().item()
    got = ops.grad_norm(xs)
    assert abs(got.item() - norm) <= 2 * E32 * norm
    most = 0.5 * norm
    f = most / (norm + 1e-6)
    for out in (torch.float32, torch.bfloat16, None):
        u = 2.0 ** -8 if (out or dtype) == torch.bfloat16 else E32
        if out is None:
            assert torch.equal(ops.clip_grad_norm(xs, most), got)
            y = x
        else:
            y, ys = views(n, size, out, fill=7.0)
            assert torch.equal(ops.clip_grad_norm(xs, most, out=ys), got)
        assert bool(((y.double() - ref * f).abs() <= (1.01 * u + 6 * E32) * (ref * f).abs() + 2.0 ** -133).all()), out


def test_graph_of_many_tensors(ops):
    say("graph of many tensors")
    x, xs = views(3000, 50, torch.float32)
    y, ys = views(3000, 50, torch.float32, fill=0.0)
    norm = ops.clip_grad_norm(xs, 1.0, out=ys)
    want = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = ops.clip_grad_norm(xs, 1.0, out=ys)
    for _ in range(3):
        y.zero_()
        held.zero_()
        ops.clip_grad_norm([x + 1.0], 1.0)      # eager work between the replays
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, norm) and torch.equal(y, want)


def test_time_of_many_tensors(ops):
    """Scaling moves twice the bytes that the norm reads, so both take about three times it,
    more where launches are short, also of very many tensors: 128000 partial sums added up
    by each of 128000 blocks would be several times that."""
    say("time of many tensors")
    _, xs = views(64000, 16400, torch.bfloat16)
    _, ys = views(64000, 16400, torch.bfloat16, fill=0.0)

    def least(f):
        best = math.inf
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            f()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best
    norm, both = least(lambda: ops.grad_norm(xs)), least(lambda: ops.clip_grad_norm(xs, 1.0, out=ys))
    say(f"norm {norm:.3f} ms, with scaling {both:.3f} ms")
    assert both < 5.5 * norm, (norm, both)
