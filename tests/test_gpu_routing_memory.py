"""GPU tests of the memory behind what route returns: it can be saved, copied and kept
piece by piece."""
import copy
import gc
import io
import pickle
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
SIZES = [(16, 8, 2), (64, 128, 32), (0, 5, 1), (100, 20, 3), (5000, 130, 8)]


@pytest.fixture(scope="module")
def ops():
    from tile_dependency_pipelined_amd import ops as o
    assert torch.cuda.is_available()
    return o


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def routing(ops, T, E, k):
    g = torch.Generator(device="cuda").manual_seed(T)
    return ops.route(torch.randn(T, E, generator=g, device="cuda"), k, normalize=True)


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_saved_and_copied(ops, size):
    say("routing saved", size)
    r = routing(ops, *size)
    f = io.BytesIO()
    torch.save(r._asdict(), f)
    f.seek(0)
    loaded = torch.load(f, weights_only=True)
    deep, pickled = copy.deepcopy(r), pickle.loads(pickle.dumps(tuple(r)))
    for i, (name, v) in enumerate(r._asdict().items()):
        for w in (loaded[name], deep[i], pickled[i]):
            assert w.dtype == v.dtype and w.is_contiguous() and torch.equal(w, v), name


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_each_can_be_kept(ops, size):
    """A loss kept for a log holds nothing else; the others hold outputs of their type, and no scratch memory."""
    say("routing kept", size)
    T, E, k = size
    r = routing(ops, T, E, k)
    assert r.loss.untyped_storage().nbytes() <= 512
    f = io.BytesIO()
    torch.save(r.loss, f)
    assert f.getbuffer().nbytes < 4096
    for v, n in ((r.experts, 2 * T * k + 2 * E + 1), (r.gates, T * k + E)):
        assert v.untyped_storage().nbytes() <= 4 * n + 4 * 256
    del v
    kept = r.loss
    torch.cuda.synchronize()
    gc.collect()
    before = torch.cuda.memory_allocated()
    del r
    assert before - torch.cuda.memory_allocated() >= 4 * (3 * T * k + 3 * E + 1)
    assert kept.item() >= 0.0
