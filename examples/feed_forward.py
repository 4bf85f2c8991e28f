"""Feed-forward blocks of a transformer, dense and by expert, from the operators
of tile_dependency_pipelined_amd.ops: a few training steps on synthetic data and a
decode step.

    python examples/feed_forward.py [--tokens 2048] [--width 512] [--hidden 2048]
                                    [--experts 8] [--steps 20] [--dtype bf16|f32]

The dense block is y = x + W2 gelu(W1 norm(x) + b1) + b2, the expert block the same
with each token's weights chosen by a fixed router.  Both blocks learn to
reproduce a target: the printed loss has to fall.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from tile_dependency_pipelined_amd import ops  # noqa: E402


class Dense:
    """norm -> linear with GeLU -> linear with the residual in its epilogue."""

    def __init__(self, width, hidden, dtype, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(*shape, generator=g, device="cuda") * std
        self.dtype = dtype
        # 32-bit master weights; the operators work on copies of their type
        self.params = {"g": torch.ones(width, device="cuda"), "b": torch.zeros(width, device="cuda"),
                       "w1": normal(width, hidden, std=width ** -0.5), "b1": torch.zeros(hidden, device="cuda"),
                       "w2": normal(hidden, width, std=hidden ** -0.5), "b2": torch.zeros(width, device="cuda")}

    def weights(self):
        return {k: v.to(self.dtype) for k, v in self.params.items()}

    def forward(self, x, keep=True):
        p = self.weights()
        n, mean, rstd = ops.layer_norm(x, p["g"], p["b"])
        h = ops.linear(n, p["w1"], p["b1"], act=ops.ACT_GELU_TANH, need_pre=keep)
        h, z = h if keep else (h, None)
        y = ops.linear(h, p["w2"], p["b2"], residual=x)
        self.saved = (p, x, n, mean, rstd, h, z)
        return y

    def backward(self, dy):
        """Gradients of the parameters by name, and of x."""
        p, x, n, mean, rstd, h, z = self.saved
        dh, dw2, db2 = ops.linear_backward(dy, h, p["w2"])
        dn, dw1, db1 = ops.linear_backward(dh, n, p["w1"], pre=z, act=ops.ACT_GELU_TANH)
        dx, dg, db = ops.layer_norm_backward(dn, x, mean, rstd, p["g"])
        return {"g": dg, "b": db, "w1": dw1, "b1": db1, "w2": dw2, "b2": db2}, dx + dy

    def step(self, grads, lr):
        for k, v in self.params.items():
            v -= lr * grads[k].float()


class Experts(Dense):
    """The same with one pair of layers per expert; rows are sorted by expert once."""

    def __init__(self, width, hidden, experts, dtype, seed=0):
        super().__init__(width, hidden, dtype, seed)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        E = experts
        self.experts = E
        self.params["w1"] = torch.randn(E, width, hidden, generator=g, device="cuda") * width ** -0.5
        self.params["w2"] = torch.randn(E, hidden, width, generator=g, device="cuda") * hidden ** -0.5
        self.params["b1"], self.params["b2"] = torch.zeros(E, hidden, device="cuda"), torch.zeros(E, width, device="cuda")
        self.router = torch.randn(width, E, generator=g, device="cuda")

    def route(self, x):
        expert = (x.float() @ self.router).argmax(1)
        order = torch.argsort(expert, stable=True)
        counts = (expert[:, None] == torch.arange(self.experts, device=x.device)).sum(0)
        offsets = torch.zeros(self.experts + 1, dtype=torch.int32, device=x.device)
        offsets[1:] = counts.cumsum(0)
        return order, offsets

    def forward(self, x, keep=True):
        p = self.weights()
        order, offsets = self.route(x)
        n, mean, rstd = ops.layer_norm(x, p["g"], p["b"])
        rows = n[order]
        h = ops.grouped_linear(rows, p["w1"], offsets, p["b1"], act=ops.ACT_GELU_TANH, need_pre=keep)
        h, z = h if keep else (h, None)
        out = ops.grouped_linear(h, p["w2"], offsets, p["b2"])
        y = x.clone()
        y[order] += out
        self.saved = (p, x, order, offsets, rows, mean, rstd, h, z)
        return y

    def backward(self, dy):
        p, x, order, offsets, rows, mean, rstd, h, z = self.saved
        dout = dy[order]
        dh, dw2, db2 = ops.grouped_linear_backward(dout, h, p["w2"], offsets)
        drows, dw1, db1 = ops.grouped_linear_backward(dh, rows, p["w1"], offsets, pre=z, act=ops.ACT_GELU_TANH)
        dn = torch.empty_like(drows)
        dn[order] = drows
        dx, dg, db = ops.layer_norm_backward(dn, x, mean, rstd, p["g"])
        return {"g": dg, "b": db, "w1": dw1, "b1": db1, "w2": dw2, "b2": db2}, dx + dy


def train(block, x, target, steps, lr):
    """Mean squared error before each step."""
    losses = []
    for _ in range(steps):
        y = block.forward(x)
        diff = y.float() - target
        losses.append(diff.square().mean().item())
        grads, _ = block.backward((diff * (2.0 / x.shape[0])).to(x.dtype))
        block.step(grads, lr)
    return losses


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=0.01)
    ap.add_argument("--dtype", choices=["bf16", "f32"], default="bf16")
    a = ap.parse_args(argv)
    dtype = torch.bfloat16 if a.dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(a.tokens, a.width, generator=g, device="cuda").to(dtype)
    target = x.float() + torch.tanh(torch.roll(x.float(), 1, 1))
    result = {}
    for name, block in (("dense", Dense(a.width, a.hidden, dtype)),
                        ("experts", Experts(a.width, a.hidden, a.experts, dtype))):
        losses = train(block, x, target, a.steps, a.lr)
        token = block.forward(x[:1], keep=False)
        batch = block.forward(x, keep=False)[:1]
        off = (token.float() - batch.float()).abs().max().item()
        print(f"{name}: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps; "
              f"one token alone is {off:.4f} from the same token in the batch", flush=True)
        result[name] = (losses, off)
    return result


if __name__ == "__main__":
    main()
