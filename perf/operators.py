"""Measured cases of the feed-forward operators: linear layers with a fused
epilogue, linear layers grouped by expert, and layer normalisation, each with
its backward pass.

    y = act(x w + b) + r          x [M][K], w [K][N] (or stored [N][K]), b [N], r [M][N]
    y_t = act(x_t w_e + b_e)      rows sorted by expert, expert e has rows offsets[e] .. offsets[e+1]-1
    y = (x - mean) rstd w + b     per row, rstd = 1 / sqrt(var + eps)

A case runs either the plain form (elementary torch operations in 32 bits,
rounded once at the end) or the library's entry points (`own`).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5

# Widths are those of this repository's workloads (512, 4096, 8192, 28672) or
# powers of two; the odd sizes are generic.
LISTED = [
    # one token through a 4096-wide projection with bias and tanh-GeLU: the decode step, where latency counts
    dict(name="linear_token", op="linear", dtype="bf16", m=1, k=4096, n=4096, act="gelu_tanh", bias=True),
    # thirteen sequences decoded together through the up projection of the 8192 / 28672 MLP: weight streaming
    dict(name="linear_decode_batch", op="linear", dtype="bf16", m=13, k=8192, n=28672, act="silu", bias=True),
    # a prompt of 2048 tokens through an 8192-square layer, all of the epilogue on: the largest product
    dict(name="linear_prefill", op="linear", dtype="bf16", m=2048, k=8192, n=8192, act="gelu_tanh", bias=True, res=True),
    # odd sizes, so that no row but the first is aligned: pruned or concatenated layers
    dict(name="linear_odd", op="linear", dtype="bf16", m=777, k=1003, n=2049, act="relu", bias=True, res=True),
    # a 32-bit layer with its weight stored [N][K], batch not a multiple of anything
    dict(name="linear_f32", op="linear", dtype="f32", m=515, k=1024, n=2048, act="gelu_tanh", bias=True, wt=True),
    # gradients of a 4096-square layer over 2048 tokens
    dict(name="linear_bwd", op="linear_bwd", dtype="bf16", m=2048, k=4096, n=4096, act="gelu_tanh", bias=True),
    # sixteen rows over eight experts: the decode step of a mixture of experts
    dict(name="grouped_decode", op="grouped", dtype="bf16", m=16, k=4096, n=4096, experts=8, act="silu", bias=True),
    # a training batch sorted by expert, skewed, one expert idle; keeps the pre-activation for the backward pass
    dict(name="grouped_train", op="grouped", dtype="bf16", m=8192, k=2048, n=4096, experts=16, act="gelu_tanh", bias=True,
         pre=True),
    # its gradients at an odd number of rows
    dict(name="grouped_bwd", op="grouped_bwd", dtype="bf16", m=4099, k=2048, n=4096, experts=8, act="gelu_tanh", bias=True),
    # one row of the widest layer: the norm of a decode step
    dict(name="norm_token", op="norm", dtype="bf16", m=1, n=8192),
    # 32-bit rows of odd width
    dict(name="norm_f32_odd", op="norm", dtype="f32", m=4093, n=4099),
    # the gradients of a long batch, weight and bias reductions with them
    dict(name="norm_bwd", op="norm_bwd", dtype="bf16", m=16384, n=8192),
]
DEFAULTS = dict(act="none", bias=False, res=False, pre=False, wt=False, experts=0, k=0)


def listed():
    return [{**DEFAULTS, **c} for c in LISTED]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: half of them multiples of 64, as in most models, half as they fall."""
    w = _log(rng, lo, hi)
    return max(64, w // 64 * 64) if w >= 64 and rng.random() < 0.5 else w


def draw(rng):
    while True:
        c = dict(DEFAULTS)
        c["op"] = rng.choice(["linear", "linear", "linear_bwd", "grouped", "grouped_bwd", "norm", "norm_bwd"])
        c["dtype"] = rng.choice(["bf16", "bf16", "bf16", "f32"])
        if c["op"].startswith("norm"):
            c["m"], c["n"] = _log(rng, 1, 16384), _width(rng, 8, 16384)
        else:
            c["k"], c["n"] = _width(rng, 16, 8192), _width(rng, 16, 8192)
            c["m"] = _log(rng, 1, 2048)
            c["act"] = rng.choice(["none", "gelu_tanh", "relu", "silu"])
            c["bias"] = rng.random() < 0.7
            c["wt"] = rng.random() < 0.3
            if c["op"].startswith("grouped"):
                c["m"], c["experts"] = _log(rng, 1, 8192), _log(rng, 1, 32)
                if c["experts"] * c["k"] * c["n"] > 1 << 28:
                    continue
            if c["op"] == "linear":
                c["res"] = rng.random() < 0.5
            if c["op"] in ("linear", "grouped"):
                c["pre"] = rng.random() < 0.3
        w = work(c)
        if w["flops"] <= (2.7e11 if c["dtype"] == "bf16" else 6e10) and w["bytes"] <= 8e8:
            return c


def work(case):
    """What one pass reads, writes and computes at the least."""
    es = 2 if case["dtype"] == "bf16" else 4
    m, k, n, e = case["m"], case["k"], case["n"], case["experts"]
    if case["op"] == "norm":
        return {"bytes": es * (2 * m * n + 2 * n) + 8 * m, "flops": 8 * m * n}
    if case["op"] == "norm_bwd":
        return {"bytes": es * (3 * m * n + 3 * n) + 8 * m, "flops": 14 * m * n}
    used = sum(c > 0 for c in _counts(case)) if e else 1  # experts whose weights have to be read
    b = es * n if case["bias"] else 0
    if case["op"] in ("linear", "grouped"):
        outs = 1 + (1 if case["pre"] else 0) + (1 if case["res"] else 0)
        return {"bytes": es * (m * k + used * k * n + outs * m * n) + used * b, "flops": 2 * m * k * n}
    acts = 2 if case["act"] != "none" else 1          # dy and the pre-activation
    return {"bytes": es * (2 * m * k + acts * m * n + (used + max(e, 1)) * k * n) + max(e, 1) * b, "flops": 4 * m * k * n}


def _counts(case, seed=0):
    """Rows of each expert: a skewed router, one expert idle where there are
    several.  The seed says which expert gets which count."""
    rng = np.random.default_rng(case["m"])
    p = np.exp(0.7 * rng.standard_normal(case["experts"]))
    if case["experts"] >= 4:
        p[0] = 0.0
    counts = rng.multinomial(case["m"], p / p.sum())
    return [int(c) for c in np.random.default_rng(seed).permutation(counts)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    m, k, n, e = case["m"], case["k"], case["n"], case["experts"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    s = {"case": case}
    if case["op"].startswith("norm"):
        # a residual stream: rows off zero, a few channels far larger than the rest
        x = torch.randn(m, n, generator=g, device="cuda") + torch.randn(m, 1, generator=g, device="cuda")
        x[:, ::257] *= 12.0
        s["x"] = x.to(dt)
        s["w"], s["b"] = (1 + 0.2 * torch.randn(n, generator=g, device="cuda")).to(dt), normal(n, std=0.1)
        if case["op"] == "norm_bwd":
            s["dy"] = normal(m, n, std=0.05)
            xf = s["x"].float()
            s["mean"] = xf.mean(1)
            s["rstd"] = torch.rsqrt(((xf - s["mean"][:, None]) ** 2).mean(1) + EPS)
        return s
    s["x"] = normal(m, k)
    lead = (e,) if e else ()
    shape = lead + ((n, k) if case["wt"] else (k, n))
    w = torch.empty(shape, dtype=dt, device="cuda")
    for i in range(max(e, 1)):
        (w[i] if e else w).copy_(torch.randn(shape[-2:], generator=g, device="cuda") * k ** -0.5)
    s["w"] = w.transpose(-1, -2) if case["wt"] else w
    if case["bias"]:
        s["b"] = normal(*lead, n, std=0.1)
    if case["res"]:
        s["r"] = normal(m, n)
    if e:
        s["counts"] = _counts(case, seed)
        s["offsets"] = torch.tensor([0] + list(np.cumsum(s["counts"])), dtype=torch.int32, device="cuda")
    if case["op"].endswith("bwd"):
        s["dy"] = normal(m, n, std=0.05)
        if case["act"] != "none":
            s["pre"] = normal(m, n)
    return s


# ---- the plain form -------------------------------------------------------

C0 = math.sqrt(2.0 / math.pi)


def _act(z, act):
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(C0 * (z + 0.044715 * z * z * z)))
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "gelu_tanh":
        t = torch.tanh(C0 * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * C0 * (1.0 + 3 * 0.044715 * z * z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-z))
        return sg * (1.0 + z * (1.0 - sg))
    return torch.ones_like(z)


def _plain_linear(s, dt):
    c = s["case"]
    z = s["x"].float() @ s["w"].float()
    if c["bias"]:
        z = z + s["b"].float()
    y = _act(z, c["act"])
    if c["res"]:
        y = y + s["r"].float()
    out = {"y": y.to(dt)}
    if c["pre"]:
        out["pre"] = z.to(dt)
    return out


def _plain_linear_bwd(s, dt):
    c = s["case"]
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _act_grad(s["pre"].float(), c["act"])
    out = {"dx": (dz @ s["w"].float().t()).to(dt), "dw": (s["x"].float().t() @ dz).to(dt)}
    if c["bias"]:
        out["db"] = dz.sum(0).to(dt)
    return out


def _plain_grouped(s, dt):
    c = s["case"]
    z = torch.empty(c["m"], c["n"], device="cuda")
    r0 = 0
    for e, rows in enumerate(s["counts"]):
        if rows:
            z[r0:r0 + rows] = s["x"][r0:r0 + rows].float() @ s["w"][e].float()
            if c["bias"]:
                z[r0:r0 + rows] += s["b"][e].float()
            r0 += rows
    out = {"y": _act(z, c["act"]).to(dt)}
    if c["pre"]:
        out["pre"] = z.to(dt)
    return out


def _plain_grouped_bwd(s, dt):
    c = s["case"]
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _act_grad(s["pre"].float(), c["act"])
    dx = torch.empty(c["m"], c["k"], dtype=dt, device="cuda")
    dw = torch.zeros(c["experts"], c["k"], c["n"], dtype=dt, device="cuda")
    db = torch.zeros(c["experts"], c["n"], dtype=dt, device="cuda")
    r0 = 0
    for e, rows in enumerate(s["counts"]):
        if rows:
            d = dz[r0:r0 + rows]
            dx[r0:r0 + rows] = (d @ s["w"][e].float().t()).to(dt)
            dw[e] = (s["x"][r0:r0 + rows].float().t() @ d).to(dt)
            db[e] = d.sum(0).to(dt)
            r0 += rows
    out = {"dx": dx, "dw": dw}
    if c["bias"]:
        out["db"] = db
    return out


def _plain_norm(s, dt):
    x = s["x"].float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = torch.rsqrt((d * d).mean(1) + EPS)
    y = d * rstd[:, None] * s["w"].float() + s["b"].float()
    return {"y": y.to(dt), "mean": mean, "rstd": rstd}


def _plain_norm_bwd(s, dt):
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["w"].float()
    dx = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
    return {"dx": dx.to(dt), "dw": (dy * xh).sum(0).to(dt), "db": dy.sum(0).to(dt)}


PLAIN = {"linear": _plain_linear, "linear_bwd": _plain_linear_bwd, "grouped": _plain_grouped,
         "grouped_bwd": _plain_grouped_bwd, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}


# ---- the library's entry points -------------------------------------------

def _own(s):
    from tile_dependency_pipelined_amd import ops
    c = s["case"]
    act = ops.ACTS[c["act"]]
    if c["op"] == "norm":
        y, mean, rstd = ops.layer_norm(s["x"], s["w"], s["b"], eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if c["op"] == "norm_bwd":
        dx, dw, db = ops.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"], need_bias=True)
        return {"dx": dx, "dw": dw, "db": db}
    if c["op"] in ("linear", "grouped"):
        if c["op"] == "linear":
            out = ops.linear(s["x"], s["w"], s.get("b"), residual=s.get("r"), act=act, need_pre=c["pre"])
        else:
            out = ops.grouped_linear(s["x"], s["w"], s["offsets"], s.get("b"), act=act, need_pre=c["pre"])
        return {"y": out[0], "pre": out[1]} if c["pre"] else {"y": out}
    if c["op"] == "linear_bwd":
        dx, dw, db = ops.linear_backward(s["dy"], s["x"], s["w"], pre=s.get("pre"), act=act, need_bias=c["bias"])
    else:
        dx, dw, db = ops.grouped_linear_backward(s["dy"], s["x"], s["w"], s["offsets"], pre=s.get("pre"), act=act,
                                                 need_bias=c["bias"])
    return {"dx": dx, "dw": dw, "db": db} if c["bias"] else {"dx": dx, "dw": dw}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state, DTYPES[state["case"]["dtype"]])


# ---- 64 bits ---------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    d = {key: v.double() for key, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    op, act = case["op"], case["act"]
    if op == "norm":
        mu = d["x"].sum(1, keepdim=True) / case["n"]
        rs = 1.0 / torch.sqrt(((d["x"] - mu) ** 2).sum(1, keepdim=True) / case["n"] + EPS)
        return {"y": (d["x"] - mu) * rs * d["w"] + d["b"], "mean": mu[:, 0], "rstd": rs[:, 0]}
    if op == "norm_bwd":
        mu, rs = d["mean"][:, None], d["rstd"][:, None]
        xh = (d["x"] - mu) * rs
        gw = d["dy"] * d["w"]
        dx = rs * (gw - gw.sum(1, keepdim=True) / case["n"] - xh * ((gw * xh).sum(1, keepdim=True) / case["n"]))
        return {"dx": dx, "dw": (d["dy"] * xh).sum(0), "db": d["dy"].sum(0)}

    def phi(z):                     # activation and derivative
        if act == "none":
            return z, torch.ones_like(z)
        if act == "relu":
            return z.clamp(min=0.0), (z > 0).double()
        if act == "silu":
            p = torch.sigmoid(z)
            return z * p, p + z * p * (1 - p)
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        p = torch.sigmoid(2 * u)    # (1 + tanh u) / 2
        return z * p, p + z * 2 * p * (1 - p) * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2)

    spans, r0 = [], 0
    for rows in s.get("counts", [case["m"]]):
        spans.append((r0, r0 + rows))
        r0 += rows
    ws = d["w"] if case["experts"] else d["w"][None]
    if op in ("linear", "grouped"):
        z = torch.cat([d["x"][a:b].matmul(ws[i]) for i, (a, b) in enumerate(spans)])
        if case["bias"]:
            bs = d["b"] if case["experts"] else d["b"][None]
            z = z + torch.cat([bs[i][None].expand(b - a, -1) for i, (a, b) in enumerate(spans)])
        out = {"y": phi(z)[0] + (d["r"] if case["res"] else 0.0)}
        if case["pre"]:
            out["pre"] = z
        return out
    dz = d["dy"] if act == "none" else d["dy"] * phi(d["pre"])[1]
    dx = torch.cat([dz[a:b].matmul(ws[i].t()) for i, (a, b) in enumerate(spans)])
    dw = torch.stack([d["x"][a:b].t().matmul(dz[a:b]) for a, b in spans])
    db = torch.stack([dz[a:b].sum(0) for a, b in spans])
    if not case["experts"]:
        dw, db = dw[0], db[0]
    return {"dx": dx, "dw": dw, "db": db} if case["bias"] else {"dx": dx, "dw": dw}
