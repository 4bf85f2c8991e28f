"""GPU test of the routed block of examples/feed_forward.py as the example runs it: a few
steps with the router, clipping, then a token with packed weights."""
import importlib.util
import math
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ff():
    spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


# 64 normal weights of deviation d span about 4.8 d, in 15 steps of 0.32 d; rounding to
# them is off by 0.29 of a step, 0.09 d.  Each layer's output is then off by that share of
# itself, the first layer's passes through the activation, whose slope and value are about
# as large: 0.14 for both together.  Twice that, for one token has few columns.  A decode
# step with wrong weights, experts or gates would be off by about 1.
@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_trained_and_packed(ff, name):
    print("routed example, steps and decode", name, file=sys.stderr, flush=True)
    dtype = torch.bfloat16 if name == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(300, 128, generator=g, device="cuda").to(dtype)
    target = x.float() + torch.tanh(torch.roll(x.float(), 1, 1))
    block = ff.Routed(128, 256, 4, dtype)
    losses, off = ff.train_routed(block, x, target, 12, 0.02)
    assert len(losses) == 12 and all(math.isfinite(v) for v in losses) and math.isfinite(block.norm.item())
    assert all(v.isfinite().all() for v in block.params.values())
    assert 0.0 < off < 0.28, off
