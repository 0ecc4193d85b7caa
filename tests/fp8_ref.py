"""Block-scaled e4m3 layers in numpy, in 64 bits from the quantised values on."""
import numpy as np

BLOCK = 128
F32 = np.float32


def round_e4m3(v):
    """The nearest e4m3 value: 3 fraction bits, exponents down to -6, saturated at 448, ties to even."""
    v = np.asarray(v, np.float64)
    _, ex = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(ex - 1, -6) - 3)
    return np.clip(np.round(v / step) * step, -448.0, 448.0)


def quantize(x, amax):
    """(values of the codes, scales): the scale and its inverse are rounded to fp32, and so is the product that is
    rounded to a code, as the definition says."""
    a = np.maximum(amax, F32(2.0 ** -100)).astype(F32)
    factor = F32(448.0) * (F32(1.0) / a)
    return round_e4m3((x.astype(F32) * factor).astype(F32)), (a / F32(448.0)).astype(np.float64)


def rows(x):
    """x with each block of 128 along the last axis quantised: the values stood for, in 64 bits."""
    x = np.asarray(x, F32)
    out = np.empty(x.shape, np.float64)
    for lo in range(0, x.shape[-1], BLOCK):
        part = x[..., lo:lo + BLOCK]
        q, s = quantize(part, np.abs(part).max(-1, keepdims=True))
        out[..., lo:lo + BLOCK] = q * s
    return out


def tokens(x):
    """Blocks of 128 along the first axis."""
    return rows(np.asarray(x, F32).T).T


def weight(w):
    """w [groups, n, k] in blocks of 128 x 128: (codes' values, scales, values stood for)."""
    w = np.asarray(w, F32)
    g, n, k = w.shape
    q = np.empty(w.shape, np.float64)
    s = np.empty((g, -(-n // BLOCK), -(-k // BLOCK)))
    full = np.empty(w.shape, np.float64)
    for i in range(s.shape[1]):
        for j in range(s.shape[2]):
            at = (slice(None), slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
            q[at], scale = quantize(w[at], np.abs(w[at]).max((1, 2), keepdims=True))
            s[:, i, j] = scale[:, 0, 0]
            full[at] = q[at] * scale
    return q, s, full


def linear(x, w, offsets):
    """(y, sum of the terms' magnitudes): w the values stood for, [groups, n, k]."""
    xq = rows(x)
    y = np.zeros((x.shape[0], w.shape[1]))
    size = np.zeros_like(y)
    for g in range(w.shape[0]):
        r = slice(offsets[g], offsets[g + 1])
        y[r] = xq[r] @ w[g].T
        size[r] = np.abs(xq[r]) @ np.abs(w[g]).T
    return y, size


def weight_grad(grad, x, offsets):
    groups = len(offsets) - 1
    dw = np.zeros((groups, grad.shape[1], x.shape[1]))
    size = np.zeros_like(dw)
    for g in range(groups):
        r = slice(offsets[g], offsets[g + 1])
        if offsets[g + 1] > offsets[g]:
            a, b = tokens(grad[r]), tokens(x[r])
            dw[g] = a.T @ b
            size[g] = np.abs(a).T @ np.abs(b)
    return dw, size
