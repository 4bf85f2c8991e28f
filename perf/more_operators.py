"""Measured cases of the operators around a feed-forward block's products: the
router of an expert layer with its balance loss, the rows' way to the experts
and back, linear layers with 4-bit weights, and the clipping of gradients by
their global norm.

    route      p = softmax(logits), the k largest per token, g their probabilities (or these over their sum);
               counts and offsets per expert, each slot's row in expert order, L = E sum_e f_e P_e with
               f_e = counts_e / (n k) and P_e = sum_t p_te / n over the n tokens that have an expert
    dispatch   out[rows_tj] = x_t                  combine   out_t = sum_j g_tj y[rows_tj] + r_t
    int4       y = act(x w + b) + r,  w_kn = s_gn (q_kn - z_gn),  g = k / group, q and z of 4 bits
    clip       N = sqrt(sum over all tensors of x^2), x min(1, c / (N + 1e-6))

A case runs either the plain form (elementary torch operations in 32 bits,
rounded once at the end) or the library's entry points (`own`).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# Widths are those of this repository's workloads (512, 2048, 4096, 8192, 28672)
# or powers of two; the odd sizes are generic.
LISTED = [
    # the router of a decode step: sixteen sequences, eight experts, where latency counts
    dict(name="route_decode", op="route", dtype="bf16", t=16, e=8, k=2, norm=True),
    # a training batch of padded sequences over many experts, 32-bit logits
    dict(name="route_train", op="route", dtype="f32", t=16384, e=128, k=8, norm=True, pad=True),
    # the router's gradient, an odd number of tokens and experts, some experts closed to some tokens
    dict(name="route_bwd", op="route_bwd", dtype="f32", t=8191, e=60, k=6, off=True),
    # a training batch's rows to their experts
    dict(name="dispatch_train", op="dispatch", dtype="bf16", t=8192, k=2, e=16, d=4096),
    # and back, weighted, onto the residual stream; sequences padded
    dict(name="combine_train", op="combine", dtype="bf16", t=8192, k=2, e=16, d=4096, res=True, pad=True),
    # the gradient of that at an odd number of tokens, four experts each
    dict(name="combine_bwd", op="combine_bwd", dtype="bf16", t=4099, k=4, e=60, d=2048),
    # one token through a 4096-square layer of 4-bit weights: the decode step, where latency counts
    dict(name="int4_token", op="int4", dtype="bf16", m=1, kk=4096, n=4096, group=128, zeros=True, act="silu", bias=True),
    # thirteen sequences decoded together through the up projection of the 8192 / 28672 MLP: weight streaming
    dict(name="int4_decode_batch", op="int4", dtype="bf16", m=13, kk=8192, n=28672, group=128, act="gelu_tanh"),
    # a short prompt through an odd number of columns, the residual in the epilogue
    dict(name="int4_prompt", op="int4", dtype="bf16", m=300, kk=8192, n=8191, group=64, zeros=True, res=True),
    # sixteen tokens' rows over eight experts of 4-bit weights: the decode step of an expert layer
    dict(name="int4_experts", op="int4", dtype="bf16", m=32, kk=4096, n=4096, group=128, zeros=True, e=8, act="silu"),
    # 32-bit gradients of a 512-wide block, biases and norms among them
    dict(name="clip_block", op="clip", dtype="f32", out="f32", sizes="block", width=512, hidden=2048),
    # bf16 gradients of the 8192 / 28672 MLP, clipped into the 32 bits that the optimizer works in
    dict(name="clip_mlp", op="clip", dtype="bf16", out="f32", sizes="block", width=8192, hidden=28672),
]
DEFAULTS = dict(t=0, e=0, k=0, d=0, m=0, kk=0, n=0, group=0, norm=False, pad=False, off=False, res=False, gates=True,
                zeros=False, act="none", bias=False, out="f32", sizes="", width=0, hidden=0, tensors=0)


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
        c["op"] = rng.choice(["route", "route", "route_bwd", "dispatch", "combine", "combine_bwd", "int4", "int4", "int4",
                              "int4_experts", "clip", "clip"])
        c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
        if c["op"].startswith("route"):
            c["t"], c["e"] = _log(rng, 1, 32768), _log(rng, 2, 512)
            c["k"] = min(c["e"], rng.choice([1, 2, 2, 4, 6, 8]))
            c["norm"], c["pad"], c["off"] = rng.random() < 0.5, rng.random() < 0.3, rng.random() < 0.2
        elif c["op"] in ("dispatch", "combine", "combine_bwd"):
            c["t"], c["e"], c["d"] = _log(rng, 1, 16384), _log(rng, 2, 128), _width(rng, 16, 8192)
            c["k"] = min(c["e"], rng.choice([1, 2, 2, 4, 6, 8]))
            c["pad"] = rng.random() < 0.3
            if c["op"] == "combine":
                c["res"], c["gates"] = rng.random() < 0.5, rng.random() < 0.7
        elif c["op"].startswith("int4"):
            c["m"], c["kk"], c["n"] = _log(rng, 1, 512), _width(rng, 32, 16384), _width(rng, 16, 16384)
            c["dtype"] = rng.choice(["bf16", "bf16", "bf16", "f32"])
            c["group"], c["zeros"] = rng.choice([32, 64, 128, 128]), rng.random() < 0.6
            c["act"], c["bias"] = rng.choice(["none", "gelu_tanh", "relu", "silu"]), rng.random() < 0.4
            if c["op"] == "int4":
                c["res"] = rng.random() < 0.4
            else:
                c["e"] = _log(rng, 1, 32)
            c["op"] = "int4"
        else:
            c["sizes"], c["tensors"] = str(rng.randrange(1 << 30)), _log(rng, 1, 300)
            c["out"] = rng.choice(["f32", c["dtype"]])
        w = work(c)
        if c["op"] == "int4" and max(c["e"], 1) * c["kk"] * c["n"] > 1 << 28:
            continue
        if w["flops"] <= (4e10 if c["dtype"] == "bf16" else 1e10) and w["bytes"] <= 1e9:
            return c


def _numels(case):
    """Elements of each gradient."""
    if case["sizes"] == "block":  # norm weight and bias, two layers with their biases
        w, h = case["width"], case["hidden"]
        return [w, w, w * h, h, h * w, w]
    rng = np.random.default_rng(int(case["sizes"]))
    n = np.exp(rng.uniform(0.0, math.log(2 ** 24), case["tensors"])).astype(int)
    return [int(v) for v in n]


def work(case):
    """What one pass reads, writes and computes at the least."""
    es = 2 if case["dtype"] == "bf16" else 4
    op, t, e, k, d = case["op"], case["t"], case["e"], case["k"], case["d"]
    if op == "route":
        return {"bytes": t * e * es + 12 * t * k + (t if case["pad"] else 0) + 12 * e + 8, "flops": 6 * t * e}
    if op == "route_bwd":
        return {"bytes": 2 * t * e * es + 8 * t * k + 4 * e, "flops": 8 * t * e}
    if op == "dispatch":
        return {"bytes": es * d * t * (1 + k) + 4 * t * k, "flops": 0}
    if op == "combine":
        return {"bytes": es * d * t * (1 + k + (1 if case["res"] else 0)) + (8 if case["gates"] else 4) * t * k,
                "flops": 2 * t * k * d}
    if op == "combine_bwd":
        return {"bytes": es * d * t * (1 + 2 * k) + 12 * t * k, "flops": 3 * t * k * d}
    if op == "clip":
        n = sum(_numels(case))
        return {"bytes": n * (es + (2 if case["out"] == "bf16" else 4)) + 4, "flops": 3 * n}
    m, kk, n = case["m"], case["kk"], case["n"]
    used = sum(c > 0 for c in _counts(case)) if e else 1
    groups = -(-kk // case["group"])
    weight = kk * n / 2 + groups * n * (es + (0.5 if case["zeros"] else 0))
    outs = 2 if case["res"] else 1
    return {"bytes": int(used * (weight + (es * n if case["bias"] else 0)) + es * m * (kk + outs * n)), "flops": 2 * m * kk * n}


def _counts(case, seed=0):
    """Rows of each expert: a skewed router, one expert idle where there are
    several.  The seed says which expert gets which count."""
    rng = np.random.default_rng(case["m"])
    p = np.exp(0.7 * rng.standard_normal(case["e"]))
    if case["e"] >= 4:
        p[0] = 0.0
    counts = rng.multinomial(case["m"], p / p.sum())
    return [int(c) for c in np.random.default_rng(seed).permutation(counts)]


def _logits(case, g):
    """A router's logits: some experts liked more than others, in all tokens."""
    t, e = case["t"], case["e"]
    x = torch.randn(t, e, generator=g, device="cuda") + 0.7 * torch.randn(e, generator=g, device="cuda")
    if case["off"]:     # a quarter of the experts closed, another quarter for each token
        x[torch.rand(t, e, generator=g, device="cuda") < 0.25] = float("-inf")
    return x.to(DTYPES[case["dtype"]])


def _valid(case, g):
    """Sequences of up to 256 tokens, padded behind their ends."""
    t = case["t"]
    ends = torch.randint(128, 257, ((t + 255) // 256,), generator=g, device="cuda")
    i = torch.arange(t, device="cuda")
    return (i % 256) < ends[i // 256]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op, t, e, k, d = case["op"], case["t"], case["e"], case["k"], case["d"]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = {"case": case}
    if op in ("route", "route_bwd", "dispatch", "combine", "combine_bwd"):
        s["logits"] = _logits({**case, "off": case["off"] and op.startswith("route")}, g)
        s["valid"] = _valid(case, g) if case["pad"] else None
        if op == "route":
            return s
        r = _plain_route(s, dt)
        if op == "route_bwd":
            s["experts"], s["slopes"] = r["experts"], r["slopes"]
            s["dgates"], s["dloss"] = normal(t, k, std=0.05, dtype=torch.float32), torch.full((), 0.01, device="cuda")
            return s
        del s["logits"]
        s["rows"], s["offsets"] = r["rows"], r["offsets"]
        if op == "dispatch":
            s["x"] = normal(t, d)
            return s
        s["y"] = normal(t * k, d)
        s["gates"] = r["gates"] if case["gates"] else None
        s["res"] = normal(t, d) if case["res"] else None
        if op == "combine_bwd":
            s["dout"] = normal(t, d, std=0.05)
        return s
    if op == "clip":
        # gradients of very different sizes from one tensor to the next
        s["grads"] = [normal(n, std=math.exp(1.5 * math.sin(7.0 * i)) * 1e-3) for i, n in enumerate(_numels(case))]
        s["out"] = [torch.empty(x.shape, dtype=DTYPES[case["out"]], device="cuda") for x in s["grads"]]
        s["max_norm"] = 1e-2 if seed % 2 else 1e-3
        return s
    m, kk, n, group = case["m"], case["kk"], case["n"], case["group"]
    lead = (e,) if e else ()
    groups = -(-kk // group)
    s["x"] = normal(m, kk)
    s["q"] = torch.randint(0, 16, (*lead, kk, n), generator=g, device="cuda", dtype=torch.uint8)
    s["scales"] = ((0.5 + torch.rand(*lead, groups, n, generator=g, device="cuda")) * 0.2 * kk ** -0.5).to(dt)
    s["zeros"] = torch.randint(5, 11, (*lead, groups, n), generator=g, device="cuda", dtype=torch.uint8) if case["zeros"] else None
    s["bias"] = normal(*lead, n, std=0.1) if case["bias"] else None
    s["res"] = normal(m, n) if case["res"] else None
    if e:
        s["counts"] = _counts(case, seed)
        s["offsets"] = torch.tensor([0] + list(np.cumsum(s["counts"])), dtype=torch.int32, device="cuda")
    if own:     # a program keeps its weights laid out
        from tile_dependency_pipelined_amd import ops
        s["w"] = ops.pack_int4(s["q"], s["scales"], s["zeros"], group_size=group)
        del s["q"]
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


def _softmax(x):
    """Over rows; zeros where nothing is allowed."""
    top = x.amax(1, keepdim=True)
    p = torch.exp(x - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    z = p.sum(1, keepdim=True)
    return p / torch.where(z == 0, torch.ones_like(z), z)


def _plain_route(s, dt):
    c = s["case"]
    t, e, k = c["t"], c["e"], c["k"]
    x = s["logits"].float()
    if s["valid"] is not None:
        x = torch.where(s["valid"][:, None], x, torch.full_like(x, float("-inf")))
    p = _softmax(x)
    v, order = torch.sort(x, dim=1, descending=True, stable=True)
    v, order = v[:, :k], order[:, :k]
    used = v != float("-inf")
    gates = torch.where(used, torch.gather(p, 1, order), torch.zeros_like(v))
    if c["norm"]:
        total = gates.sum(1, keepdim=True)
        gates = gates / torch.where(total == 0, torch.ones_like(total), total)
    experts = torch.where(used, order, torch.full_like(order, -1)).to(torch.int32)
    # expert order: slots sorted by expert, those without one last
    flat = torch.where(used, order, torch.full_like(order, e)).reshape(-1)
    by = torch.argsort(flat, stable=True)
    rows = torch.empty(t * k, dtype=torch.int32, device=x.device)
    rows[by] = torch.arange(t * k, dtype=torch.int32, device=x.device)
    rows = torch.where(used.reshape(-1), rows, torch.full_like(rows, -1)).view(t, k)
    counts = torch.zeros(e + 1, dtype=torch.int32, device=x.device)
    counts.index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))
    counts = counts[:e]
    offsets = torch.zeros(e + 1, dtype=torch.int32, device=x.device)
    offsets[1:] = torch.cumsum(counts, 0)
    n = used[:, 0].sum().to(torch.float32).clamp(min=1.0)
    slopes = counts.float() * (e / (k * n)) / n
    loss = (slopes * p.sum(0)).sum()
    return {"experts": experts, "gates": gates, "rows": rows, "counts": counts, "offsets": offsets, "loss": loss,
            "slopes": slopes}


def _plain_route_bwd(s, dt):
    c = s["case"]
    x = s["logits"].float()
    p = _softmax(x)
    has = s["experts"] >= 0
    idx = s["experts"].clamp(min=0).long()
    dg = torch.where(has, s["dgates"], torch.zeros_like(s["dgates"]))
    grow = s["slopes"][None, :] * s["dloss"]
    dp = grow.expand_as(p)
    if c["norm"]:
        g = torch.where(has, torch.gather(p, 1, idx), torch.zeros_like(dg))
        g = g / g.sum(1, keepdim=True)
        chosen = g * (dg - (g * dg).sum(1, keepdim=True))
    else:
        g = torch.where(has, torch.gather(p, 1, idx), torch.zeros_like(dg))
        dp = dp - (g * dg).sum(1, keepdim=True)      # the softmax's own sum, over the chosen
        chosen = g * dg
    dx = p * (dp - (p * grow).sum(1, keepdim=True))
    dx = dx.scatter_add(1, idx, torch.where(has, chosen, torch.zeros_like(chosen)))
    return {"dlogits": torch.where(has[:, :1], dx, torch.zeros_like(dx)).to(dt)}


def _slots(rows, n):
    """Row of each slot, `n` for those without one."""
    r = rows.reshape(-1).long()
    return torch.where(r < 0, torch.full_like(r, n), r)


def _plain_dispatch(s, dt):
    c = s["case"]
    t, k, d = c["t"], c["k"], c["d"]
    out = torch.zeros(t * k + 1, d, dtype=dt, device="cuda")
    out[_slots(s["rows"], t * k)] = s["x"].repeat_interleave(k, 0)
    return {"rows": out[:t * k]}


def _plain_combine(s, dt):
    c = s["case"]
    t, k = c["t"], c["k"]
    acc = torch.zeros(t, c["d"], device="cuda")
    for j in range(k):
        r = s["rows"][:, j].long()
        v = s["y"][r.clamp(min=0)].float()
        if c["gates"]:
            v = v * s["gates"][:, j, None]
        acc = acc + torch.where((r >= 0)[:, None], v, torch.zeros_like(v))
    if c["res"]:
        acc = acc + s["res"].float()
    return {"out": acc.to(dt)}


def _plain_combine_bwd(s, dt):
    c = s["case"]
    t, k, d = c["t"], c["k"], c["d"]
    g = s["dout"].float()
    dy = torch.zeros(t * k + 1, d, dtype=dt, device="cuda")
    dy[_slots(s["rows"], t * k)] = (g[:, None, :] * s["gates"][:, :, None]).to(dt).view(t * k, d)
    dgates = torch.empty(t, k, device="cuda")
    for j in range(k):
        r = s["rows"][:, j].long()
        dot = (g * s["y"][r.clamp(min=0)].float()).sum(1)
        dgates[:, j] = torch.where(r >= 0, dot, torch.zeros_like(dot))
    return {"dy": dy[:t * k], "dgates": dgates}


def _plain_int4(s, dt):
    c = s["case"]
    group = c["group"]

    def weight(q, scales, zeros):
        z = zeros.float() if zeros is not None else torch.full_like(scales, 8.0, dtype=torch.float32)
        g = torch.arange(c["kk"], device="cuda") // group
        return (q.float() - z[g]) * scales.float()[g]

    if not c["e"]:
        z = s["x"].float() @ weight(s["q"], s["scales"], s["zeros"])
        if c["bias"]:
            z = z + s["bias"].float()
    else:
        z = torch.empty(c["m"], c["n"], device="cuda")
        r0 = 0
        for e, rows in enumerate(s["counts"]):
            if rows:
                w = weight(s["q"][e], s["scales"][e], s["zeros"][e] if c["zeros"] else None)
                z[r0:r0 + rows] = s["x"][r0:r0 + rows].float() @ w
                if c["bias"]:
                    z[r0:r0 + rows] += s["bias"][e].float()
                r0 += rows
    y = _act(z, c["act"])
    if c["res"]:
        y = y + s["res"].float()
    return {"y": y.to(dt)}


def _plain_clip(s, dt):
    sums = [(x.float() * x.float()).sum(dtype=torch.float64) for x in s["grads"]]
    norm = torch.sqrt(torch.stack(sums).sum()).float()
    scale = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    out = [(x.float() * scale).to(o.dtype) for x, o in zip(s["grads"], s["out"])]
    return {"norm": norm, "grads": out}


PLAIN = {"route": _plain_route, "route_bwd": _plain_route_bwd, "dispatch": _plain_dispatch, "combine": _plain_combine,
         "combine_bwd": _plain_combine_bwd, "int4": _plain_int4, "clip": _plain_clip}


# ---- the library's entry points -------------------------------------------

def _own(s):
    from tile_dependency_pipelined_amd import ops
    c = s["case"]
    op = c["op"]
    if op == "route":
        r = ops.route(s["logits"], c["k"], normalize=c["norm"], valid=s["valid"])
        return {"experts": r.experts, "gates": r.gates, "rows": r.rows, "counts": r.counts, "offsets": r.offsets,
                "loss": r.loss, "slopes": r.slopes}
    if op == "route_bwd":
        return {"dlogits": ops.route_backward(s["dgates"], s["dloss"], s["logits"], s["experts"], s["slopes"],
                                              normalize=c["norm"])}
    if op == "dispatch":
        return {"rows": ops.dispatch(s["x"], s["rows"], s["offsets"])}
    if op == "combine":
        return {"out": ops.combine(s["y"], s["rows"], s["gates"], residual=s["res"])}
    if op == "combine_bwd":
        dy, dgates = ops.combine_backward(s["dout"], s["y"], s["rows"], s["offsets"], s["gates"])
        return {"dy": dy, "dgates": dgates}
    if op == "clip":
        norm = ops.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"])
        return {"norm": norm, "grads": s["out"]}
    act = ops.ACTS[c["act"]]
    if c["e"]:
        return {"y": ops.grouped_linear_int4(s["x"], s["w"], s["offsets"], s["bias"], act=act)}
    return {"y": ops.linear_int4(s["x"], s["w"], s["bias"], residual=s["res"], act=act)}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state, DTYPES[state["case"]["dtype"]])


# ---- 64 bits ---------------------------------------------------------------

def _exact_route(case, logits, valid):
    """Expert by expert: the largest logit left, the lowest index among equals."""
    t, e, k = case["t"], case["e"], case["k"]
    x = logits.double()
    if valid is not None:
        x = x.masked_fill(~valid[:, None], -math.inf)
    live = (x > -math.inf).any(1)
    p = torch.where(live[:, None], torch.softmax(x.masked_fill(~live[:, None], 0.0), 1), torch.zeros_like(x))
    left, cols = x.clone(), torch.arange(e, device=x.device)
    experts = torch.full((t, k), -1, dtype=torch.int64, device=x.device)
    taken = torch.zeros(t, e, dtype=torch.int64, device=x.device)
    for j in range(k):
        best = left.max(1, keepdim=True).values
        ok = best[:, 0] > -math.inf
        i = torch.where(left == best, cols[None, :], e).min(1).values
        experts[:, j] = torch.where(ok, i, -1)
        hit = (cols[None, :] == i[:, None]) & ok[:, None]
        taken += hit
        left.masked_fill_(hit, -math.inf)
    gates = torch.gather(p, 1, experts.clamp(min=0)) * (experts >= 0)
    if case["norm"]:
        gates = gates / gates.sum(1, keepdim=True).masked_fill(~live[:, None], 1.0)
    counts = taken.sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    before = taken.cumsum(0) - taken            # earlier tokens with the same expert
    rows = torch.gather(before, 1, experts.clamp(min=0)) + offsets[experts.clamp(min=0)]
    rows = torch.where(experts >= 0, rows, -1)
    n = max(int(live.sum()), 1)
    slopes = counts.double() * e / (float(n) * n * k)
    return dict(experts=experts.int(), gates=gates, rows=rows.int(), counts=counts.int(), offsets=offsets.int(),
                loss=slopes.dot(p.sum(0)), slopes=slopes, p=p)


def exact(case, seed):
    s = prepare(case, seed)
    op, t, k, d = case["op"], case["t"], case["k"], case["d"]
    if op == "route":
        r = _exact_route(case, s["logits"], s["valid"])
        del r["p"]
        return r
    if op == "route_bwd":
        # by autograd through the gates and the loss
        x = s["logits"].double().requires_grad_(True)
        has = s["experts"] >= 0
        live = has.any(1)
        p = torch.softmax(torch.where(live[:, None], x, torch.zeros_like(x)), 1)
        gates = torch.gather(p, 1, s["experts"].clamp(min=0).long()) * has
        if case["norm"]:
            gates = gates / (gates.sum(1, keepdim=True) + (~live[:, None]).double())
        total = (gates * s["dgates"].double()).sum()
        total = total + s["dloss"].double() * (p * live[:, None] * s["slopes"].double()).sum()
        total.backward()
        return {"dlogits": x.grad}
    if op in ("dispatch", "combine", "combine_bwd"):
        rows = s["rows"].long()
        token, slot = torch.nonzero(rows >= 0, as_tuple=True)
        at = rows[token, slot]
        if op == "dispatch":
            out = torch.zeros(t * k, d, dtype=torch.float64, device="cuda")
            out[at] = s["x"].double()[token]
            return {"rows": out}
        y = s["y"].double()
        w = s["gates"].double()[token, slot][:, None] if s["gates"] is not None else 1.0
        if op == "combine":
            out = s["res"].double() if s["res"] is not None else torch.zeros(t, d, dtype=torch.float64, device="cuda")
            return {"out": out.index_add(0, token, y[at] * w)}
        g = s["dout"].double()[token]
        dy = torch.zeros_like(y)
        dy[at] = g * w
        dgates = torch.zeros(t, k, dtype=torch.float64, device="cuda")
        dgates[token, slot] = torch.linalg.vecdot(g, y[at])
        return {"dy": dy, "dgates": dgates}
    if op == "clip":
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(x.double())) ** 2 for x in s["grads"]))
        f = min(1.0, s["max_norm"] / (norm + 1e-6))
        return {"norm": torch.tensor(norm, dtype=torch.float64, device="cuda"), "grads": [x.double() * f for x in s["grads"]]}

    if own:     # (the codes, which the packed weight replaced)
        s = _codes(case, seed)
    group, act = case["group"], case["act"]

    def product(x, i):
        pick = (lambda v: None if v is None else v[i]) if case["e"] else (lambda v: v)
        q, sc, zp, b = pick(s["q"]), pick(s["scales"]), pick(s["zeros"]), pick(s["bias"])
        z = torch.zeros(x.shape[0], case["n"], dtype=torch.float64, device="cuda")
        for g, k0 in enumerate(range(0, case["kk"], group)):
            part = x[:, k0:k0 + group].double()
            zero = zp[g].double() if zp is not None else 8.0
            z += sc[g].double() * (part.matmul(q[k0:k0 + group].double()) - part.sum(1, keepdim=True) * zero)
        return z if b is None else z + b.double()

    if case["e"]:
        spans, r0 = [], 0
        for i, rows in enumerate(s["counts"]):
            spans.append(product(s["x"][r0:r0 + rows], i))
            r0 += rows
        z = torch.cat(spans)
    else:
        z = product(s["x"], 0)
    if act == "relu":
        z = z.clamp(min=0.0)
    elif act == "silu":
        z = z * torch.sigmoid(z)
    elif act == "gelu_tanh":
        z = z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    return {"y": z if s["res"] is None else z + s["res"].double()}


def _codes(case, seed):
    """The inputs with the weight's codes, whichever side runs."""
    global own
    kept, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = kept
