"""GPU tests of arguments that a conversion could turn into others."""
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


def test_activation_codes_beyond_32_bits(ops):
    say("activation codes")
    x, w = torch.zeros(4, 8, device="cuda"), torch.zeros(8, 8, device="cuda")
    for act in (1 << 32, (1 << 32) + 1, -(1 << 32)):
        with pytest.raises((RuntimeError, ValueError, OverflowError)):
            ops.linear(x, w, act=act)
