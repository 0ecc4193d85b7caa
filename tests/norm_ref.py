"""Plain 64-bit forms of the join, the norms, the dropout and the balance loss, with
the sums of their terms' magnitudes that bound what rounding can do."""
import numpy as np
import torch

MUL = (0xD2511F53, 0xCD9E8D57)
ADD = (0x9E3779B9, 0xBB67AE85)


def philox(counter, key, rounds=10):
    """The four words of Philox4x32 (Salmon, Moraes, Dror and Shaw, 2011) for arrays of counters."""
    c = [np.asarray(v, np.uint64) for v in counter]
    k = list(key)
    low = np.uint64(0xFFFFFFFF)
    for _ in range(rounds):
        a, b = c[0] * np.uint64(MUL[0]), c[2] * np.uint64(MUL[1])
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(v + d) & 0xFFFFFFFF for v, d in zip(k, ADD)]
    return c


def dropped_of(p):
    return int(np.floor(float(np.float32(p)) * 65536 + 0.5))


def kept(rows, cols, p, seed, offset):
    """bool [rows, cols]: which elements stay."""
    blocks = -(-cols // 8)
    b, r = np.meshgrid(np.arange(blocks, dtype=np.uint64), np.arange(rows, dtype=np.uint64))
    offset %= 1 << 64
    words = philox((b, r, np.full_like(b, offset & 0xFFFFFFFF), np.full_like(b, offset >> 32)),
                   (seed & 0xFFFFFFFF, seed >> 32))
    halves = np.stack([np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1) for w in words], -2)
    return torch.from_numpy(halves.reshape(rows, blocks * 8)[:, :cols] >= dropped_of(p))


def gain(p):
    m = dropped_of(p)
    return 0.0 if m == 65536 else 1.0 / (1.0 - m / 65536)


def d(t):
    return None if t is None else t.detach().double().cpu()


def inverse_rms(v, eps):
    return 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + float(np.float32(eps)))


class Ref:
    """One call's arguments in 64 bits."""

    def __init__(self, *, x=None, y=None, weight=None, post_weight=None, gate=None, post=False, eps=1e-6, scale=1.0,
                 dropout=0.0, seed=0, offset=0):
        self.x, self.y, self.post, self.eps = d(x), d(y), post, eps
        some = self.x if self.x is not None else self.y
        rows, hidden = some.shape
        ones = torch.ones(hidden, dtype=torch.float64)
        self.w = ones if weight is None else d(weight)
        self.p = ones if post_weight is None else d(post_weight)
        k = torch.full((rows, hidden), float(np.float32(scale)), dtype=torch.float64)
        self.span = 1
        if dropout > 0:
            self.keep = kept(rows, hidden, dropout, seed, offset)
            k = torch.where(self.keep, k * gain(dropout), 0.0)
        self.k_no_gate = k
        if gate is not None and rows:
            self.span = rows // gate.shape[0]
            k = k * d(gate).repeat_interleave(self.span, 0)
        self.k = k

    def branch(self):
        return self.y * inverse_rms(self.y, self.eps) * self.p if self.post else self.y

    def r(self):
        """(r, magnitude)"""
        t = torch.where(self.k == 0, 0.0, self.k * torch.where(self.k == 0, 0.0, self.branch()))
        return self.x + t, self.x.abs() + t.abs()

    def h(self, r):
        return d(r) * inverse_rms(d(r), self.eps) * self.w

    def backward(self, grad_r, grad_h, r):
        """{name: (gradient, magnitude)}"""
        out = {}
        up = mag = torch.zeros(self.k.shape, dtype=torch.float64)
        if grad_r is not None:
            up, mag = d(grad_r), d(grad_r).abs()
        if grad_h is not None:
            r, dh = d(r), d(grad_h)
            rho = inverse_rms(r, self.eps)
            out["weight"] = ((dh * r * rho).sum(0), (dh * r * rho).abs().sum(0))
            hw = dh * self.w
            up = up + rho * (hw - r * rho * rho * (hw * r).mean(1, keepdim=True))
            mag = mag + rho * (hw.abs() + r.abs() * rho * rho * (hw * r).abs().mean(1, keepdim=True))
        out["x"] = (up, mag)
        if self.y is None:
            return out
        unit = self.y * inverse_rms(self.y, self.eps) if self.post else self.y
        each, each_mag = up * self.k_no_gate * unit * self.p, mag * (self.k_no_gate * unit * self.p).abs()
        out["gate"] = tuple(t.unflatten(0, (-1, self.span)).sum(1) for t in (each, each_mag))
        u, um = self.k * up, self.k.abs() * mag
        out["post_weight"] = ((u * unit).sum(0), (um * unit.abs()).sum(0))
        if self.post:
            eta = inverse_rms(self.y, self.eps)
            u, um = u * self.p, um * self.p.abs()
            u, um = (eta * (u - unit * (u * unit).mean(1, keepdim=True)),
                     eta * (um + unit.abs() * (um * unit.abs()).mean(1, keepdim=True)))
        out["y"] = (u, um)
        return out


def balance(logits, idx, bounds, score, coefficient=1.0):
    """(loss, counts, tokens, gradient, its magnitude), a sequence at a time."""
    l, idx = d(logits), idx.cpu().long()
    e = l.shape[1]
    q = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    q = torch.nan_to_num(q / q.sum(1, keepdim=True), nan=0.0)
    slope = torch.ones_like(q) if score == "softmax" else torch.sigmoid(-l)
    grad, mag = torch.zeros_like(l), torch.zeros_like(l)
    counts, tokens, losses, parts = [], [], [], []
    for lo, hi in zip(bounds[:-1], bounds[1:]):
        i = idx[lo:hi]
        there = (i >= 0) & (i < e)
        c = torch.bincount(i[there], minlength=e).double()
        rows = torch.nonzero(there.any(1))[:, 0] + lo
        m, n = len(rows), float(c.sum())
        counts.append(c)
        tokens.append(m)
        if m:
            f = c * (e / (n * m))
            losses.append(float((f * q[rows].sum(0)).sum()))
            parts.append((rows, f))
    for rows, f in parts:
        f = f * (coefficient / len(parts))
        p = q[rows]
        dot = (p * f).sum(1, keepdim=True)
        grad[rows] = p * slope[rows] * (f - dot)
        mag[rows] = p * slope[rows] * (f + dot).abs()
    loss = coefficient * sum(losses) / max(1, len(losses))
    return loss, torch.stack(counts).to(torch.int32), torch.tensor(tokens + [len(parts)], dtype=torch.int32), grad, mag
