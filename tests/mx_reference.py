"""Plain references, in 64 bits, of the RMS norm, its gradient, the MX formats
and the MX product.  numpy only; nothing of the library is used."""
import numpy as np

BLOCK = 32
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([np.ldexp(c & 7, -9) if c < 8 else np.ldexp(8 + (c & 7), (c >> 3) - 10) for c in range(127)])
EMAX = {"mxfp4": 2, "mxfp8": 8}
GRID = {"mxfp4": E2M1, "mxfp8": E4M3}


def nearest(grid, v):
    """Index of the grid value nearest to v >= 0, ties to the even index (the
    index is the code, so its last bit is the mantissa's)."""
    hi = np.clip(np.searchsorted(grid, v), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    below, above = v - grid[lo], grid[hi] - v
    return np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)


def mx_quantize(x, fmt):
    """[M, n] -> (codes uint8 [M, 32 B], one element each, scale uint8 [M, B])."""
    x = np.asarray(x, np.float64)
    m, n = x.shape
    b = -(-n // BLOCK)
    v = np.zeros((m, b * BLOCK))
    v[:, :n] = x
    v = v.reshape(m, b, BLOCK)
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], 0, v)
    top = np.abs(v).max(-1)
    e = np.frexp(top)[1] - 1 - EMAX[fmt]
    e = np.where(top > 0, np.clip(e, -127, 127), -127)
    u = np.ldexp(v, -e[..., None])
    code = nearest(GRID[fmt], np.abs(u)) | np.where(np.signbit(v), 8 if fmt == "mxfp4" else 128, 0)
    return code.reshape(m, b * BLOCK).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def mx_values(codes, scale, fmt):
    """Elements (one a byte) and scale bytes -> the values, in 64 bits."""
    half = 8 if fmt == "mxfp4" else 128
    c = codes.astype(np.int64)
    v = np.where(c % half < len(GRID[fmt]), GRID[fmt][np.minimum(c % half, len(GRID[fmt]) - 1)], np.nan)
    v = np.where(c >= half, -v, v)
    f = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    return v * np.repeat(f, BLOCK, 1)


def pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def unpack(packed):
    return np.stack((packed & 15, packed >> 4), -1).reshape(len(packed), 2 * packed.shape[1])


def rstd(h, eps):
    h = np.asarray(h, np.float64)
    return 1 / np.sqrt((h * h).sum(-1) / h.shape[-1] + eps)


def int8_codes(h, w):
    """The int8 codes, by the fp32 steps that define them, and the row maxima."""
    t = np.asarray(h, np.float32) * np.asarray(w, np.float32)
    a = np.abs(t).max(-1)
    q = np.zeros(t.shape, np.int8)
    for i in range(len(t)):
        if np.isfinite(a[i]) and a[i] > 0:
            up = np.float32(2.0 ** 60 if a[i] < 2.0 ** -100 else 1)
            inv = np.float32(127) / (a[i] * up)
            q[i] = np.rint((t[i] * up) * inv).astype(np.int8)
    return q, a


def grad(dy, h, w, r, dh=None):
    dy, h, w, r = (np.asarray(v, np.float64) for v in (dy, h, w, r))
    g = dy * w
    dot = (g * h).sum(1, keepdims=True)
    dx = r[:, None] * g - h * r[:, None] ** 3 / h.shape[1] * dot
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * h * r[:, None]).sum(0)
