"""Plain CPU oracle of the 4-bit experts and of the input norm (include/moe.h), in numpy
float64. It shares no code with the GPU path.

Quantised arrays are held as values: `q` the e2m1 values as float64, `b` the scale bytes as
integers (255: the block is not finite, its q are 0 here).
"""
from __future__ import annotations

import numpy as np

BLOCK, GROUP = 32, 256
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_codes(y):
    """Code of the nearest e2m1 value of |y| <= 6 (ties to the even code), sign in bit 3.
    Found by comparing distances to all eight."""
    y = np.asarray(y, np.float64)
    d = np.abs(np.abs(y)[..., None] - GRID)
    near = d == d.min(-1, keepdims=True)
    first = near.argmax(-1)
    second = len(GRID) - 1 - near[..., ::-1].argmax(-1)
    code = np.where(first % 2 == 0, first, second)
    return code + 8 * np.signbit(y)


def of_codes(c):
    return np.where(c & 8, -1.0, 1.0) * GRID[c & 7]


def scale_byte(amax):
    """Smallest b in 0..254 with amax <= 6 * 2^(b - 127); 255 if amax is not finite."""
    amax = np.asarray(amax, np.float64)
    b = np.zeros(amax.shape, np.int64)
    for cand in range(254, -1, -1):
        b = np.where(amax <= np.ldexp(6.0, cand - 127), cand, b)
    return np.where(np.isfinite(amax), b, 255)


def quantize(x):
    """[..., C] -> codes [..., C], b [..., C / 32]."""
    x = np.asarray(x, np.float64)
    y = x.reshape(*x.shape[:-1], -1, BLOCK)
    fin = np.isfinite(y).all(-1)
    y = np.where(fin[..., None], y, 0.0)
    b = np.where(fin, scale_byte(np.abs(y).max(-1)), 255)
    c = e2m1_codes(np.ldexp(y, (127 - np.minimum(b, 254))[..., None]))
    return c.reshape(x.shape), b


def scale(b):
    return np.where(b == 255, np.nan, np.ldexp(1.0, np.asarray(b, np.int64) - 127))


def values(c, b):
    """What codes [..., C] with scale bytes [..., C / 32] stand for."""
    return of_codes(c) * np.repeat(scale(b), BLOCK, axis=-1)


def pack(c):
    c = np.asarray(c).astype(np.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def unpack(q):
    q = np.asarray(q).astype(np.int64)
    return np.stack((q & 15, q >> 4), -1).reshape(*q.shape[:-1], -1)


def groups(b, rows=None):
    """Scale bytes [..., R, nb] -> [..., ceil(nb / 8), rows or R, 8], filled up with 0."""
    *lead, r, nb = b.shape
    rows = r if rows is None else rows
    out = np.zeros((*lead, -(-nb // 8), rows, 8), np.uint8)
    for j in range(nb):
        out[..., j // 8, :r, j % 8] = b[..., j]
    return out


def ungroup(s, rows, nb):
    """The other way."""
    s = np.asarray(s).astype(np.int64)
    return np.stack([s[..., j // 8, :rows, j % 8] for j in range(nb)], -1)


def roundtrip(x):
    return values(*quantize(x))


# ----------------------------------------------------------------------------- stages
def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def swiglu(a):
    g, u = np.split(a, 2, axis=1)
    return g * sigmoid(g) * u


def grouped(rows, off, w):
    """rows of expert e times w[e]^T; rows that no expert has come out 0."""
    out = np.zeros((rows.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            out[lo:hi] = rows[lo:hi] @ w[e].T
    return out


def ffn_forward(x, off, w1, w2, quant=roundtrip):
    """The expert FFN on (already quantised) values; nothing else is rounded."""
    a = grouped(x, off, w1)
    h = swiglu(a)
    return dict(a=a, h=h, o=grouped(quant(h), off, w2))


# ----------------------------------------------------------------------------- input norm
def rms_norm(r, w, eps):
    """y and rstd of the rows r (the sum, as it is held)."""
    rstd = 1.0 / np.sqrt((r * r).sum(1) / r.shape[1] + eps)
    return r * rstd[:, None] * w, rstd


def rms_norm_bwd(dy, r, w, rstd, dr=None):
    """dx and dw, with rstd taken as given (the forward's)."""
    xh = r * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - xh * (g * xh).sum(1, keepdims=True) / r.shape[1])
    return dx if dr is None else dx + dr, (dy * xh).sum(0)
