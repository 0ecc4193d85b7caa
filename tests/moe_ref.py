"""The router, dispatch and combine in numpy, in 64 bits, row by row."""
import numpy as np


def scores(l, kind):
    """Scores of one row of logits; an unavailable expert (-inf) has 0."""
    l = np.asarray(l, np.float64)
    if kind == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    if not (l > -np.inf).any():
        return np.zeros_like(l)
    e = np.exp(l - l.max())
    return e / e.sum()


def choose(l, bias, kind, k, groups, top_groups):
    """(chosen experts in order, margin): the margin is the smallest gap that the
    choice and its order rest on, in units of the largest value."""
    v = scores(l, kind) + (0.0 if bias is None else np.asarray(bias, np.float64))
    v = np.where(np.isneginf(l), -np.inf, v)
    gaps = [np.inf]

    def ranked(values, count):
        order = np.argsort(-values, kind="stable")
        top = values[order]
        for a, b in zip(top[:count], top[1:]):
            if np.isfinite(a) and np.isfinite(b) and a != b:
                gaps.append(abs(a - b))
        return order[:count]

    if groups > 1:
        by = v.reshape(groups, -1)
        two = -np.sort(-by, axis=1)[:, :2]
        value = np.where(np.isneginf(two[:, 0]), -np.inf, np.where(np.isneginf(two), 0.0, two).sum(1))
        kept = ranked(value, top_groups)
        mask = np.zeros(groups, bool)
        mask[kept] = True
        v = np.where(np.repeat(mask, by.shape[1]), v, -np.inf)
    idx = [e for e in ranked(v, k) if v[e] > -np.inf]
    return idx, min(gaps)


def weights(l, idx, kind, renorm, scale):
    """Weights of the chosen experts; renormalised ones over a common factor that does not underflow."""
    l = np.asarray(l, np.float64)
    if not idx:
        return np.zeros(0)
    x = l[idx]
    if not renorm:
        return scale * scores(l, kind)[idx]
    if kind == "softmax":
        u = np.exp(x - x.max())
    else:
        logs = -np.logaddexp(0.0, -x)
        u = np.exp(logs - logs.max())
    return scale * u / u.sum()


def route(logits, bias, kind, k, groups=1, top_groups=1, renorm=True, scale=1.0):
    t = logits.shape[0]
    idx, w, margin = np.full((t, k), -1, np.int32), np.zeros((t, k)), np.full(t, np.inf)
    for r in range(t):
        chosen, margin[r] = choose(logits[r], bias, kind, k, groups, top_groups)
        idx[r, : len(chosen)] = chosen
        w[r, : len(chosen)] = weights(logits[r], chosen, kind, renorm, scale)
    return idx, w, margin


def route_grad(logits, idx, gw, kind, renorm, scale):
    """Gradient of sum(gw * weights) by the formulas, the choice held fixed."""
    out = np.zeros(logits.shape)
    for r, l in enumerate(np.asarray(logits, np.float64)):
        on = idx[r] >= 0
        e, up = idx[r][on], scale * gw[r][on].astype(np.float64)
        if not e.size:
            continue
        p = scores(l, kind)
        if renorm:
            w = weights(l, list(e), kind, True, 1.0)
            d = w * (up - (w * up).sum())
            out[r, e] = d if kind == "softmax" else d * (1.0 - p[e])
        elif kind == "softmax":
            g = np.zeros_like(l)
            g[e] = up
            out[r] = p * (g - (p * g).sum())
        else:
            out[r, e] = up * p[e] * (1.0 - p[e])
    return out


def places(idx, experts):
    """(pos, counts, offsets, order) of the stable order by expert; slots without one last."""
    flat = idx.reshape(-1)
    key = np.where((flat < 0) | (flat >= experts), experts, flat)
    order = np.argsort(key, kind="stable")
    pos = np.empty(flat.size, np.int64)
    pos[order] = np.arange(flat.size)
    pos[key == experts] = -1
    counts = np.bincount(key, minlength=experts + 1)[:experts]
    return pos.reshape(idx.shape), counts, np.concatenate([[0], np.cumsum(counts)]), order
