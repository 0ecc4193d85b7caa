"""Cases and plain forms of the operators around a mixture-of-experts layer.

They are what stands between that layer and the rest of a model: the norms
before and after a block with the residual join between them (gate, residual
scale, dropout), dropout of activations by a counter-based generator whose mask
is never stored, and the loss that keeps the router's experts balanced, with
their counts.  Where `own` is false `run` computes them with elementary torch
operations in 32 bits; where it is true it calls the package.
"""
import math

import numpy as np
import torch

own = False

INF = float("inf")
EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one token of a serving step: the block's output joins the residual, and the next block's input is normed
        dict(name="norm_token", op="norm", gates=0, span=1, hidden=4096, dtype="bf16", residual="bf16", weight="bf16",
             post=False, joined=True, normed=True, scale=1.0, p=0.0, grad=False),
        # a small serving batch with a norm after the block too
        dict(name="norm_step", op="norm", gates=0, span=33, hidden=2048, dtype="bf16", residual="bf16", weight="f32",
             post=True, joined=True, normed=True, scale=1.0, p=0.0, grad=False),
        # a training step's rows of the all-to-all workload: both norms, a learned scale per channel, dropout
        dict(name="norm_train", op="norm", gates=1, span=16384, hidden=2048, dtype="bf16", residual="bf16", weight="f32",
             post=True, joined=True, normed=True, scale=0.5, p=0.1, grad=False),
        # its gradients
        dict(name="norm_train_grad", op="norm", gates=1, span=16384, hidden=2048, dtype="bf16", residual="bf16",
             weight="f32", post=True, joined=True, normed=True, scale=0.5, p=0.1, grad=True),
        # gradients of a batch of odd rows whose residual is held in 32 bits, each sequence with a gate of its own
        dict(name="norm_odd_grad", op="norm", gates=13, span=631, hidden=1001, dtype="bf16", residual="f32", weight="f32",
             post=True, joined=True, normed=True, scale=1.0, p=0.0, grad=True),
        # gradients of the wide rows of the all-gather workload, with the join alone after the block
        dict(name="norm_wide_grad", op="norm", gates=0, span=4096, hidden=14336, dtype="bf16", residual="bf16", weight="bf16",
             post=False, joined=True, normed=True, scale=1.0, p=0.0, grad=True),
        # the activations of one expert's few rows
        dict(name="dropout_step", op="dropout", rows=33, cols=1024, dtype="bf16", p=0.1),
        # the activations of the all-to-all workload's rows, as long as a training step has them
        dict(name="dropout_train", op="dropout", rows=131072, cols=1024, dtype="bf16", p=0.1),
        # rows of an odd size in 32 bits
        dict(name="dropout_odd", op="dropout", rows=8191, cols=2047, dtype="f32", p=0.5),
        # a small batch's router: loss, counts and gradient
        dict(name="balance_step", op="balance", tokens=512, experts=64, top_k=8, sequences=1, tail=0, score="softmax",
             dtype="f32", pad=0.0),
        # the router of the all-to-all workload's training step
        dict(name="balance_train", op="balance", tokens=16384, experts=64, top_k=8, sequences=1, tail=0, score="softmax",
             dtype="bf16", pad=0.0),
        # many experts with sigmoid scores, balanced within each of sixteen ragged sequences, with padded tokens
        dict(name="balance_sequences", op="balance", tokens=65521, experts=256, top_k=8, sequences=16, tail=100,
             score="sigmoid", dtype="f32", pad=0.03),
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm", "dropout", "balance"])
    if op == "norm":
        hidden = rng.choice([_log(rng, 5, 16384), 8 * _log(rng, 2, 2048)])
        rows = _log(rng, 1, min(16384, (1 << 25) // hidden))
        # no gate, one for all rows, one for each of a few sequences, one for each row
        gates = rng.choice([0, 0, 1, rng.randint(2, 9), rows])
        joined = rng.random() < 0.85
        return dict(op=op, gates=gates if joined else 0, span=max(1, rows // max(1, gates)), hidden=hidden,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), residual=rng.choice(["bf16", "f32"]),
                    weight=rng.choice(["f32", "bf16", "none"]), post=joined and rng.random() < 0.5, joined=joined,
                    normed=not joined or rng.random() < 0.85, scale=rng.choice([1.0, 0.25]),
                    p=rng.choice([0.0, 0.0, 0.1, 0.3]) if joined else 0.0, grad=rng.random() < 0.5)
    if op == "dropout":
        cols = rng.choice([_log(rng, 3, 16384), 8 * _log(rng, 2, 2048)])
        return dict(op=op, rows=_log(rng, 1, min(131072, (1 << 25) // cols)), cols=cols, dtype=rng.choice(["bf16", "f32"]),
                    p=rng.choice([0.05, 0.1, 0.2, 0.5]))
    experts = _log(rng, 4, 512)
    return dict(op=op, tokens=_log(rng, 1, 32768), experts=experts, top_k=rng.randint(1, min(12, experts // 2)),
                sequences=rng.choice([1, 1, _log(rng, 2, 64)]), tail=rng.choice([0, 0, 19]),
                score=rng.choice(["softmax", "sigmoid"]), dtype=rng.choice(["f32", "bf16"]), pad=rng.choice([0.0, 0.05]))


# ---- inputs -----------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _logits(g, tokens, experts):
    """log p + Gumbel noise with the all-to-all workload's expert probabilities: Zipf with exponent 1.2."""
    p = torch.arange(1, experts + 1, device="cuda", dtype=torch.float64) ** -1.2
    logp = torch.log(p / p.sum()).float()[torch.randperm(experts, generator=g, device="cuda")]
    u = torch.rand(tokens, experts, generator=g, device="cuda").clamp(1e-6, 1 - 1e-6)
    return logp - torch.log(-torch.log(u))


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"c": c, "seed": 0x9E3779B97F4A7C15 * (seed + 1) % 2 ** 63, "offset": 1000 * seed + 17}
    if own:
        import lossless_bf16_exponent_split_gb300 as z
    if c["op"] == "norm":
        t, h = max(1, c["gates"]) * c["span"], c["hidden"]
        block, residual, weight = TYPES[c["dtype"]], TYPES[c["residual"]], TYPES.get(c["weight"])

        def weights(there):
            return (1.0 + 0.2 * _randn(g, h)).to(weight) if there and weight is not None else None

        # rows of differing size, as a residual stream has them
        s["x"] = (_randn(g, t, h) * torch.exp(_randn(g, t, 1))).to(residual)
        s["y"] = (_randn(g, t, h) * torch.exp(0.5 * _randn(g, t, 1))).to(block) if c["joined"] else None
        s["weight"], s["post_weight"] = weights(c["normed"]), weights(c["post"])
        s["gate"] = (0.5 + 0.3 * _randn(g, c["gates"], h)).to(block) if c["gates"] else None
        if c["grad"]:
            s["grad_r"] = (1e-3 * _randn(g, t, h)).to(residual) if c["joined"] else None
            s["grad_h"] = (1e-3 * _randn(g, t, h) * torch.exp(_randn(g, t, 1))).to(block) if c["normed"] else None
        if own:
            s["norm"] = z.ResidualNorm(h, post=c["post"], eps=EPS, scale=c["scale"], dropout=c["p"], seed=s["seed"])
    if c["op"] == "dropout":
        s["x"] = _randn(g, c["rows"], c["cols"]).to(TYPES[c["dtype"]])
        if own:
            s["dropout"] = z.Dropout(c["p"], seed=s["seed"])
    if c["op"] == "balance":
        t, e, q = c["tokens"], c["experts"], c["sequences"]
        x = _logits(g, t + c["tail"], e)
        # padded tokens choose nothing
        pad = torch.rand(t + c["tail"], 1, generator=g, device="cuda") < c["pad"]
        idx = torch.sort(x, dim=1, descending=True, stable=True).indices[:, : c["top_k"]]
        s["idx"] = torch.where(pad, -1, idx).to(torch.int32).contiguous()
        s["logits"] = x.to(TYPES[c["dtype"]])
        cuts = torch.sort(torch.randint(0, t + 1, (q - 1,), generator=g, device="cuda")).values
        ends = torch.tensor([0, t], device="cuda")
        # one sequence without a tail needs no table
        s["sequences"] = None if q == 1 and not c["tail"] else torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)
        if own:
            s["moe"] = z.Moe(e, c["top_k"], score=c["score"])
    return s


# ---- plain forms ------------------------------------------------------------
LOW = 0xFFFFFFFF


def _product(a, m):
    """The high and low 32 bits of a * m, for whole numbers below 2^32 in 64-bit signed ones."""
    lo, hi = (a & 0xFFFF) * m, (a >> 16) * m
    mid = hi + (lo >> 16)
    return mid >> 16, ((mid & 0xFFFF) << 16) | (lo & 0xFFFF)


def _kept(s, rows, cols, p):
    """Which elements stay: Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011) with the seed as its key on the counter
    (column / 8, row, offset); each of its four words holds the 16 bits of two neighbouring elements."""
    c1 = torch.arange(rows, device="cuda")[:, None]
    c0 = torch.arange(-(-cols // 8), device="cuda")[None, :]
    c2, c3 = torch.full_like(c0, s["offset"] & LOW), torch.full_like(c0, s["offset"] >> 32)
    k0, k1 = s["seed"] & LOW, s["seed"] >> 32
    for _ in range(10):
        (h0, l0), (h1, l1) = _product(c0, 0xD2511F53), _product(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    words = torch.stack(torch.broadcast_tensors(c0, c1, c2, c3), 2)
    bits = torch.stack([words & 0xFFFF, words >> 16], 3).reshape(rows, -1)[:, :cols]
    return bits >= _dropped_of(p)


def _dropped_of(p):
    """How many of the 2^16 values of an element's bits drop it."""
    return int(math.floor(p * 65536 + 0.5))


def _gain(p):
    return 1.0 / (1.0 - _dropped_of(p) / 65536)


def _unit(v):
    """v over its root mean square, and that factor."""
    f = 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * f, f


def _times(v, w):
    return v if w is None else v * w.float()


def _keep(s):
    """Which elements of the block's output stay, or None for all."""
    c = s["c"]
    return _kept(s, *s["y"].shape, c["p"]) if c["p"] > 0 else None


def _drop(v, keep, p):
    return v if keep is None else torch.where(keep, v * _gain(p), 0.0)


def _factor(s, keep):
    """What the block's output is multiplied by: scale, gate and dropout."""
    c = s["c"]
    f = torch.full((1, 1), c["scale"], device="cuda")
    if s["gate"] is not None:
        f = f * s["gate"].float().repeat_interleave(c["span"], 0)
    return _drop(f, keep, c["p"])


def _norm(s):
    c, w, w2 = s["c"], s["weight"], s["post_weight"]
    block = TYPES[c["dtype"]]
    if not c["grad"]:
        out = {}
        r = s["x"]
        if c["joined"]:
            b = s["y"].float()
            if c["post"]:
                b = _times(_unit(b)[0], w2)
            r = out["r"] = (r.float() + _factor(s, _keep(s)) * b).to(r.dtype)
        if c["normed"]:
            out["h"] = _times(_unit(r.float())[0], w).to(block)  # of r as it is held
        return out
    out = {}
    up = None if s["grad_r"] is None else s["grad_r"].float()
    if c["normed"]:
        dh = s["grad_h"].float()
        unit, f = _unit(s["x"].float())
        if w is not None:
            out["grad_weight"] = (dh * unit).sum(0).to(w.dtype)
        dh = _times(dh, w)
        part = f * (dh - unit * (dh * unit).mean(1, keepdim=True))
        up = part if up is None else up + part
    out["grad_x"] = up.to(s["x"].dtype)
    if not c["joined"]:
        return out
    b = s["y"].float()
    keep = _keep(s)
    factor = _factor(s, keep)
    unit, f = _unit(b) if c["post"] else (b, None)
    if s["gate"] is not None:
        each = _drop(up * _times(unit, w2) * c["scale"], keep, c["p"])
        out["grad_gate"] = each.reshape(c["gates"], c["span"], -1).sum(1).to(s["gate"].dtype)
    up = up * factor
    if c["post"]:
        if w2 is not None:
            out["grad_post_weight"] = (up * unit).sum(0).to(w2.dtype)
        up = _times(up, w2)
        up = f * (up - unit * (up * unit).mean(1, keepdim=True))
    out["grad_y"] = up.to(block)
    return out


def _dropout(s):
    c, x = s["c"], s["x"]
    return {"out": torch.where(_kept(s, *x.shape, c["p"]), x.float() * _gain(c["p"]), 0.0).to(x.dtype)}


def _balance(s):
    c, l, idx = s["c"], s["logits"].float(), s["idx"].long()
    n, q, e = l.shape[0], c["sequences"], c["experts"]
    live = (idx >= 0).any(1)
    if c["score"] == "softmax":
        p = torch.exp(l - l.amax(1, keepdim=True))
        slope = 1.0
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
        slope = 1.0 / (1.0 + torch.exp(l))
    p = torch.where(live[:, None], p / p.sum(1, keepdim=True), 0.0)
    at = torch.zeros(n, dtype=torch.long, device="cuda")
    if s["sequences"] is not None:  # the sequence of each token; q: behind the last one
        at = (s["sequences"][None, 1:] <= torch.arange(n, device="cuda")[:, None]).sum(1)
    flat = torch.where(idx < 0, q * e, torch.where(at[:, None] == q, q * e, at[:, None] * e + idx)).reshape(-1)
    counts = torch.zeros(q * e + 1, dtype=torch.int32, device="cuda").scatter_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))
    counts = counts[: q * e].reshape(q, e)
    member = (at[None, :] == torch.arange(q, device="cuda")[:, None]) & live
    tokens = member.sum(1)
    mean = member.double() @ p.double() / tokens.clamp(min=1)[:, None]
    share = counts.double() * (e / counts.sum(1).clamp(min=1)[:, None].double())
    alive = (tokens > 0).sum()
    loss = (share * mean).sum() / alive.clamp(min=1)
    share = (share / (tokens.clamp(min=1) * alive.clamp(min=1))[:, None]).float()
    f = torch.cat([share, share.new_zeros(1, e)])[at]
    grad = p * slope * (f - (f * p).sum(1, keepdim=True))
    return {"loss": loss.float().reshape(1), "counts": counts, "tokens": torch.cat([tokens, alive[None]]).to(torch.int32),
            "grad": grad.to(s["logits"].dtype)}


def run(state):
    s = state
    c = s["c"]
    if not own:
        return {"norm": _norm, "dropout": _dropout, "balance": _balance}[c["op"]](s)
    if c["op"] == "dropout":
        return {"out": s["dropout"].apply(s["x"], offset=s["offset"])}
    if c["op"] == "balance":
        b = s["moe"].balance(s["logits"], s["idx"], sequences=s["sequences"])
        grad = s["moe"].balance_backward(s["logits"], s["idx"], b, sequences=s["sequences"])
        return {"loss": b.loss, "counts": b.counts, "tokens": b.tokens, "grad": grad}
    n, w = s["norm"], s["weight"]
    if not c["joined"]:
        if not c["grad"]:
            return {"h": n.norm(s["x"], w, dtype=TYPES[c["dtype"]])}
        gx, gw = n.norm_backward(s["grad_h"], s["x"], w)
        return {"grad_x": gx} if gw is None else {"grad_weight": gw, "grad_x": gx}
    more = dict(post_weight=s["post_weight"], gate=s["gate"], offset=s["offset"])
    if not c["grad"]:
        r, h = n.add(s["x"], s["y"], w, normed=c["normed"], **more)
        return {"r": r, "h": h} if c["normed"] else {"r": r}
    g = n.add_backward(s["grad_r"], s["grad_h"], s["x"] if c["normed"] else None, s["y"], w, **more)
    names = [("grad_weight", g.weight), ("grad_x", g.x), ("grad_gate", g.gate), ("grad_post_weight", g.post_weight), ("grad_y", g.y)]
    return {k: v for k, v in names if v is not None}


# ---- what a pass cannot do without ------------------------------------------
def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "none": 0}
    if c["op"] == "dropout":
        n = c["rows"] * c["cols"]
        return {"bytes": 2 * n * size[c["dtype"]], "flops": 2 * n}
    if c["op"] == "balance":
        n, e = c["tokens"] + c["tail"], c["experts"]
        # logits and indices once, the gradient and the counts out
        return {"bytes": 2 * n * e * size[c["dtype"]] + 4 * n * c["top_k"] + 4 * c["sequences"] * e, "flops": 10 * n * e}
    t, h = max(1, c["gates"]) * c["span"], c["hidden"]
    n, block, residual, weight = t * h, size[c["dtype"]], size[c["residual"]], size[c["weight"]]
    each = (c["normed"] + c["post"]) * h * weight + c["gates"] * h * block
    if not c["grad"]:
        # x, and y and r with a join, and h
        return {"bytes": n * (residual + c["joined"] * (block + residual) + c["normed"] * block) + each, "flops": 10 * n}
    # x's gradient; of a join r's and y's too, and y (which the join alone without a gate does without); h's gradient and r
    reads_y = c["joined"] and (c["post"] or c["gates"] > 0)
    moved = residual + c["joined"] * (residual + block) + reads_y * block + c["normed"] * (block + residual)
    return {"bytes": n * moved + 2 * each, "flops": 24 * n}


# ---- the definitions in 64 bits ---------------------------------------------
def _exact_kept(s, rows, cols, p):
    """The generator's bits with unsigned 64-bit numbers on the host, a slab of rows at a time."""
    blocks = -(-cols // 8)
    out = np.empty((rows, cols), dtype=np.bool_)
    u = np.uint64
    mask, half = u(0xFFFFFFFF), u(32)
    step = max(1, (1 << 16) // blocks)
    for lo in range(0, rows, step):
        m = min(step, rows - lo)
        x = [np.tile(np.arange(blocks, dtype=u), m), np.repeat(np.arange(lo, lo + m, dtype=u), blocks),
             np.full(m * blocks, s["offset"] % 2 ** 32, u), np.full(m * blocks, s["offset"] // 2 ** 32, u)]
        key = [s["seed"] % 2 ** 32, s["seed"] // 2 ** 32]
        for _ in range(10):
            a, b = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
            x = [(b >> half) ^ x[1] ^ u(key[0]), b & mask, (a >> half) ^ x[3] ^ u(key[1]), a & mask]
            key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
        words = np.stack(x, 1).astype("<u4")  # little-endian: the low half of a word comes first
        out[lo:lo + m] = words.view("<u2").reshape(m, blocks * 8)[:, :cols] >= round(p * 65536)
    return torch.from_numpy(out).cuda()


def _exact_norm(s):
    c = s["c"]

    def unit(v, w):
        v = v * (v.square().mean(1, keepdim=True) + EPS).rsqrt()
        return v if w is None else v * w

    def leaf(v):
        return None if v is None else v.double().requires_grad_(c["grad"])

    w, w2, gate, y = leaf(s["weight"]), leaf(s["post_weight"]), leaf(s["gate"]), leaf(s["y"])
    x = leaf(s["x"])
    keep = _exact_kept(s, *x.shape, c["p"]) if c["p"] > 0 else None

    def joined():
        b = unit(y, w2) if c["post"] else y
        if keep is not None:
            b = (b / (1 - round(c["p"] * 65536) / 65536)).masked_fill(~keep, 0.0)
        if gate is not None:
            b = (b.unflatten(0, (c["gates"], c["span"])) * gate[:, None, :]).flatten(0, 1)
        return b * c["scale"]

    if not c["grad"]:
        out, r = {}, x
        if c["joined"]:
            r = out["r"] = x + joined()
            r = r.to(s["x"].dtype).double()
        if c["normed"]:
            out["h"] = unit(r, w)
        return out
    out = {}
    with torch.enable_grad():
        up = 0.0 if s["grad_r"] is None else s["grad_r"].double()
        if c["normed"]:
            parts = [x] if w is None else [x, w]
            got = torch.autograd.grad(unit(x, w), parts, s["grad_h"].double())
            up = up + got[0]
            if w is not None:
                out["grad_weight"] = got[1]
        out["grad_x"] = up
        if c["joined"]:
            parts = [("grad_gate", gate), ("grad_post_weight", w2), ("grad_y", y)]
            parts = [(k, v) for k, v in parts if v is not None]
            for (k, _), v in zip(parts, torch.autograd.grad(joined(), [v for _, v in parts], up)):
                out[k] = v
    return out


def _exact_balance(s):
    c = s["c"]
    e, idx = c["experts"], s["idx"].long()
    bounds = [0, idx.shape[0]] if s["sequences"] is None else s["sequences"].tolist()
    terms = []
    with torch.enable_grad():
        l = s["logits"].double().requires_grad_()
        for lo, hi in zip(bounds[:-1], bounds[1:]):
            rows = torch.nonzero(idx[lo:hi, 0] >= 0)[:, 0] + lo  # a token of these cases chooses all or nothing
            if rows.numel() == 0:
                continue
            q = torch.softmax(l[rows], 1) if c["score"] == "softmax" else torch.sigmoid(l[rows])
            q = q / q.sum(1, keepdim=True)
            f = torch.bincount(idx[rows].flatten(), minlength=e).double()
            terms.append(e * (f / f.sum() * q.mean(0)).sum())
        loss = sum(terms) / max(1, len(terms)) + 0.0 * l.sum()
        (grad,) = torch.autograd.grad(loss, l)
    return {"loss": loss.detach().reshape(1), "counts": None, "tokens": None, "grad": grad}


def exact(case, seed):
    global own
    was, own = own, False  # the inputs alone: no handle of the package
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "balance":
        return _exact_balance(s)
    gain = 1 - round(case["p"] * 65536) / 65536
    return {"out": (s["x"].double() / gain).masked_fill(~_exact_kept(s, *s["x"].shape, case["p"]), 0.0)}
