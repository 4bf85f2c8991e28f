"""GPU test of an output of dispatch beside, and on top of, the offsets it still reads."""
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_out_and_offsets_in_one_buffer():
    from tile_dependency_pipelined_amd import ops
    print("dispatch out and offsets", file=sys.stderr, flush=True)
    x = torch.randn(4, 8, device="cuda")
    rows = torch.arange(8, dtype=torch.int32, device="cuda").flip(0).view(4, 2)
    want = ops.dispatch(x, rows, torch.tensor([0, 8], dtype=torch.int32, device="cuda"))
    buf = torch.zeros(80, device="cuda")
    out, words = buf[:64].view(8, 8), buf.view(torch.int32)
    for at in (0, 30, 62):
        words[at:at + 2] = torch.tensor([0, 8], dtype=torch.int32)
        with pytest.raises(RuntimeError):
            ops.dispatch(x, rows, words[at:at + 2], out=out)
    words[63:65] = torch.tensor([0, 8], dtype=torch.int32)     # the last offset alone is read
    assert torch.equal(ops.dispatch(x, rows, words[63:65], out=out), want) and words[64].item() == 8
