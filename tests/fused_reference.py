"""Plain references of the fused A8W8 products, their gradients and the int8 form:
numpy, in 64 bits, or in single fp32 steps where the definition asks for them.
Nothing of the library is used."""
import math

import numpy as np

BLOCK = 32
_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(kind, z):
    """The activation in 64 bits."""
    if kind in (None, "none"):
        return z
    if kind == "relu":
        return np.where(z < 0, 0, z)
    with np.errstate(over="ignore"):
        if kind == "silu":
            return z / (1 + np.exp(-z))
        if kind == "gelu":
            return z * (1 + _erf(z / math.sqrt(2))) / 2
        return z / (1 + np.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def slope(kind, z):
    """Its derivative."""
    if kind in (None, "none"):
        return np.ones_like(z)
    if kind == "relu":
        return np.where(z > 0, 1.0, 0.0)
    with np.errstate(over="ignore"):
        if kind == "silu":
            s = 1 / (1 + np.exp(-z))
            return s * (1 + z * (1 - s))
        if kind == "gelu":
            return (1 + _erf(z / math.sqrt(2))) / 2 + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        k = 2 * math.sqrt(2 / math.pi)
        s = 1 / (1 + np.exp(-k * (z + 0.044715 * z ** 3)))
        return s + z * s * (1 - s) * k * (1 + 3 * 0.044715 * z * z)


def act_error(kind, z):
    """Bound of the fp32 activation's error at z: |f| (|y| + 8) 2^-22 for those by a
    sigmoid of y (the exponential's argument is rounded four times, the reciprocal and
    the sum once each), |z| 2^-22 for the one by erf (erf within 2 units of 1, two
    products and a sum)."""
    z = np.abs(z)
    if kind in (None, "none", "relu"):
        return 0 * z
    if kind == "gelu":
        return z * 2.0 ** -22
    y = z if kind == "silu" else 1.6 * np.minimum(z, 32) * (1 + 0.045 * np.minimum(z, 32) ** 2)
    # both signs of z: f is at most |z| min(1, exp(-y) for negative z); bounded by the larger one's own
    return z * (y + 8) * 2.0 ** -22 * np.where(y > 40, np.exp(-np.minimum(y, 700)) + 2.0 ** -10, 1)


def accumulate(a, w, b_trans):
    """int64 sums of int8 products."""
    w = w.astype(np.int64)
    return a.astype(np.int64) @ (w.T if b_trans else w)


def z32(acc, act_scale, weight_scale, bias=None):
    """The definition's fp32 steps."""
    with np.errstate(over="ignore", invalid="ignore"):
        z = (acc.astype(np.float32) * np.asarray(act_scale, np.float32).reshape(-1, 1)) * \
            np.asarray(weight_scale, np.float32).reshape(1, -1)
        return z if bias is None else z + np.asarray(bias, np.float32)


def int8_form(x, block=None):
    """fp32 [M, n] -> (codes, scale [M] or [M, blocks]), by the definition's steps."""
    x = np.asarray(x, np.float32)
    m, n = x.shape
    width = n if block is None else block
    b = -(-n // width)
    v = np.zeros((m, b * width), np.float32)
    v[:, :n] = x
    v = v.reshape(m, b, width)
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], np.float32(0), v)
    top = np.abs(v).max(-1)
    up = np.where(top < np.float32(2.0 ** -100), np.float32(2.0 ** 60), np.float32(1))
    with np.errstate(divide="ignore"):
        inv = np.where(top > 0, np.float32(127) / (top * up), np.float32(0)).astype(np.float32)
    codes = np.rint((v * up[..., None]) * inv[..., None]).astype(np.int8).reshape(m, -1)[:, :n]
    scale = np.where(bad, np.float32(np.nan), np.where(top > 0, top / np.float32(127), np.float32(1))).astype(np.float32)
    return codes, scale[:, 0] if block is None else scale


def values(codes, scale):
    """What codes with a scale per block stand for, in 64 bits."""
    return codes.astype(np.float64) * np.repeat(scale.astype(np.float64), BLOCK, 1)[:, :codes.shape[1]]


def weight_rows(w, b_trans):
    """[N, K] in 64 bits."""
    return (w if b_trans else w.T).astype(np.float64)


def grad(pairs, scales, weights, b_trans):
    """(dx, bound of its error before dx is rounded): pairs of factors before the weights'
    scales.  A factor, with its scale, is rounded to a / 32639 for the row's largest a (half
    a step, and the step itself and the quotient twice in fp32), and is itself the end of
    at most 12 roundings and an activation in fp32 (2^-20 of it, and 2^-19 absolute of its
    dy scale where a difference cancels, which the caller adds)."""
    f = [p * np.asarray(s, np.float64).reshape(1, -1) for p, s in zip(pairs, scales)]
    top = np.max([np.abs(x).max(1) for x in f], 0)[:, None]
    rows = [weight_rows(w, b_trans) for w in weights]
    dx = sum(x @ w for x, w in zip(f, rows))
    off = sum((np.abs(x) * 2.0 ** -20 + top * (0.5 / 32639 + 2.0 ** -21)) @ np.abs(w) for x, w in zip(f, rows))
    return dx, off
