"""GPU test of the routed block of examples/feed_forward.py: its passes against
torch's autograd in 64 bits, its decode step against the quantised weights in 64
bits, and the example as it is run."""
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


def make(ff, dtype):
    block = ff.Routed(72, 200, 5, dtype, k=2)
    g = torch.Generator(device="cuda").manual_seed(1)
    for k in ("g", "b", "b1", "b2"):
        block.params[k] += 0.2 * torch.randn(block.params[k].shape, generator=g, device="cuda")
    x, dy = (torch.randn(150, 72, generator=g, device="cuda").to(dtype) for _ in range(2))
    return block, x, dy


def reference(p, x, experts, balance, group=None):
    """y and the objective's share of the balance loss, on the host in 64 bits, the experts given."""
    n = torch.nn.functional.layer_norm(x, x.shape[1:], p["g"], p["b"])
    prob = torch.softmax(n @ p["wr"], 1)
    gates = torch.gather(prob, 1, experts)
    gates = gates / gates.sum(1, keepdim=True)
    rows = []
    for i in range(x.shape[0]):
        out = 0
        for j, e in enumerate(experts[i].tolist()):
            h = torch.nn.functional.gelu(n[i] @ p["w1"][e] + p["b1"][e], approximate="tanh")
            out = out + gates[i, j] * (h @ p["w2"][e] + p["b2"][e])
        rows.append(x[i] + out)
    counts = torch.bincount(experts.reshape(-1), minlength=prob.shape[1]).double()
    loss = prob.shape[1] * (counts / experts.numel() * prob.mean(0)).sum()
    return torch.stack(rows), balance * loss


# Relative 2-norms.  fp32: sums of at most 200 products, nine operators in a row each
# within a few hundred roundings of 2^-24: below 1e-4.  bf16: each operator
# rounds its output (2^-8 at most, about a third of that on average); gradients pass
# through up to eleven of them, and the router's come from differences
# of products that nearly cancel (a gate's gradient less its mean): 3e-2, the router's 6e-2.
@pytest.mark.parametrize("name, tol, router", [("f32", 1e-4, 1e-4), ("bf16", 3e-2, 6e-2)])
def test_block_against_autograd(ff, name, tol, router):
    print("routed block", name, file=sys.stderr, flush=True)
    block, x, dy = make(ff, torch.bfloat16 if name == "bf16" else torch.float32)
    y = block.forward(x)
    grads, dx = block.backward(dy)
    p = {k: v.double().cpu().requires_grad_(True) for k, v in block.weights().items()}
    xr = x.double().cpu().requires_grad_(True)
    wy, loss = reference(p, xr, block.saved[6].experts.cpu().long(), block.balance)
    ((wy * dy.double().cpu()).sum() + loss).backward()
    for what, got, want in [("y", y, wy.detach()), ("dx", dx, xr.grad)] + [(k, grads[k], p[k].grad) for k in p]:
        err = ((got.double().cpu() - want).norm() / want.norm()).item()
        assert err < (router if what == "wr" else tol), (what, err)
    norm = torch.sqrt(sum((v.double() ** 2).sum() for v in grads.values())).item()
    before = {k: v.clone() for k, v in block.params.items()}
    block.step(grads, 0.5)
    assert abs(block.norm.item() - norm) < 1e-6 * norm
    f = min(1.0, block.max_norm / norm)
    for k, v in block.params.items():
        want = before[k].double() - 0.5 * f * grads[k].double()
        assert bool(((v.double() - want).abs() <= 1e-6 * (want.abs() + before[k].double().abs() + 1e-3)).all()), k


@pytest.mark.parametrize("name, tol", [("f32", 1e-4), ("bf16", 2e-2)])
def test_decode(ff, name, tol):
    """With the quantised weights in the 64-bit form: roundings as above."""
    print("routed decode", name, file=sys.stderr, flush=True)
    block, x, _ = make(ff, torch.bfloat16 if name == "bf16" else torch.float32)
    block.pack(group_size=32)
    p = {k: v.double().cpu() for k, v in block.weights().items()}
    for k in ("w1", "w2"):
        q, s, z = ff.ops.quantize_int4(block.weights()[k], 32)
        g = torch.arange(q.shape[1]) // 32
        p[k] = s.double().cpu()[:, g] * (q.double().cpu() - z.double().cpu()[:, g])
    for rows in (1, 7, 150):
        y = block.decode(x[:rows])
        block.forward(x[:rows], keep=False)
        want, _ = reference(p, x[:rows].double().cpu(), block.saved[6].experts.cpu().long(), 0.0)
        err = ((y.double().cpu() - want).norm() / want.norm()).item()
        assert err < tol, (rows, err)


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_example_runs(ff, name, capsys):
    print("routed example", name, file=sys.stderr, flush=True)
    ff.main(["--tokens", "200", "--width", "96", "--hidden", "160", "--experts", "4", "--steps", "3", "--dtype", name])
    assert "routed:" in capsys.readouterr().out
