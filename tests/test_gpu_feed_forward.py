"""GPU test of the operators used together: the example's blocks against torch's
autograd in 64 bits, and their training."""
import importlib.util
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


def reference(block, x, dy):
    """y and the gradients, on the host in 64 bits."""
    p = {k: v.double().cpu().requires_grad_(True) for k, v in block.weights().items()}
    x = x.double().cpu().requires_grad_(True)
    n = torch.nn.functional.layer_norm(x, x.shape[1:], p["g"], p["b"])
    if hasattr(block, "experts"):
        expert = (x.detach().float() @ block.router.cpu()).argmax(1)
        y = torch.stack([x[i] + torch.nn.functional.gelu(n[i] @ p["w1"][e] + p["b1"][e], approximate="tanh") @ p["w2"][e]
                         + p["b2"][e] for i, e in enumerate(expert.tolist())])
    else:
        y = x + torch.nn.functional.gelu(n @ p["w1"] + p["b1"], approximate="tanh") @ p["w2"] + p["b2"]
    y.backward(dy.double().cpu())
    return y.detach(), {k: v.grad for k, v in p.items()}, x.grad


# Relative 2-norms.  fp32: sums of at most 200 products, each operator within a few
# hundred roundings of 2^-24, five in a row: below 1e-4.  bf16: each of the five
# operators rounds its output (2^-8 at most, about a third of that on
# average) and the gradients pass through up to eight roundings: below 2e-2.
@pytest.mark.parametrize("name, tol", [("f32", 1e-4), ("bf16", 2e-2)])
@pytest.mark.parametrize("kind", ["dense", "experts"])
def test_block_against_autograd(ff, kind, name, tol):
    print("feed-forward block", kind, name, file=sys.stderr, flush=True)
    dtype = torch.bfloat16 if name == "bf16" else torch.float32
    block = ff.Dense(72, 200, dtype) if kind == "dense" else ff.Experts(72, 200, 5, dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    for k in ("g", "b", "b1", "b2"):
        block.params[k] += 0.2 * torch.randn(block.params[k].shape, generator=g, device="cuda")
    x, dy = (torch.randn(150, 72, generator=g, device="cuda").to(dtype) for _ in range(2))
    y = block.forward(x)
    grads, dx = block.backward(dy)
    wy, wg, wx = reference(block, x, dy)
    for what, got, want in [("y", y, wy), ("dx", dx, wx)] + [(k, grads[k], wg[k]) for k in wg]:
        err = ((got.double().cpu() - want).norm() / want.norm()).item()
        assert err < tol, (what, err)


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_training_and_decode(ff, name):
    print("feed-forward training", name, file=sys.stderr, flush=True)
    out = ff.main(["--tokens", "300", "--width", "128", "--hidden", "256", "--experts", "4", "--steps", "12", "--lr", "0.02",
                   "--dtype", name])
    for kind, (losses, off) in out.items():
        assert losses[-1] < 0.7 * losses[0], (kind, losses)
        # the same token through the kernels of few rows and of many: roundings of a few units of 2^-8 (2^-24)
        assert off < (0.1 if name == "bf16" else 1e-4), (kind, off)
