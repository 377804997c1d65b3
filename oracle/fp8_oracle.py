"""Plain CPU oracle of the layer's 8-bit experts (include/moe.h, "8-bit experts"):
block quantisation to e4m3 with power-of-two scales, and the expert stages on
quantised operands, in numpy float64. It shares no code with the GPU path.

Quantised arrays are held as values: `q` the e4m3 values as float64 (NaN where
the block is not finite), `b` the scale bytes as integers.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128


def identity(x):
    return x


def bf16(x):
    """float64 -> nearest bf16 (ties to even), as float64. Direct, without a
    rounding to float32 on the way."""
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        _, e = np.frexp(x)
        step = np.ldexp(1.0, np.maximum(e - 8, -133))  # 8 significant bits, subnormals 2^-133
        y = np.where(np.isfinite(x), np.round(x / step) * step, x)
        return np.where(np.abs(y) >= 2.0 ** 128, np.copysign(np.inf, x), y)


def e4m3(y):
    """Nearest e4m3 value (ties to even) of |y| <= 448."""
    y = np.asarray(y, np.float64)
    _, e = np.frexp(y)
    step = np.ldexp(1.0, np.maximum(e - 4, -9))  # 4 significant bits, subnormals 2^-9
    return np.round(y / step) * step


def scale_byte(amax):
    """Smallest b in 0..254 with amax <= 448 * 2^(b - 127); 255 if amax is not finite.
    Found by comparing, not by taking a logarithm."""
    amax = np.asarray(amax, np.float64)
    b = np.zeros(amax.shape, np.int64)
    for cand in range(254, -1, -1):
        b = np.where(amax <= np.ldexp(448.0, cand - 127), cand, b)
    return np.where(np.isfinite(amax), b, 255)


def _quantize_block(v):
    if not np.all(np.isfinite(v)):
        return np.full(v.shape, np.nan), 255
    b = int(scale_byte(np.abs(v).max()) if v.size else 0)
    return e4m3(np.ldexp(v, 127 - b)), b


def quantize_rows(x):
    """[N, C] -> q [N, C], b [N, ceil(C / 128)]: blocks of 128 columns."""
    x = np.asarray(x, np.float64)
    n, c = x.shape
    nb = -(-c // BLOCK)
    q, b = np.empty_like(x), np.empty((n, nb), np.int64)
    for j in range(nb):
        v = x[:, j * BLOCK:(j + 1) * BLOCK]
        fin = np.isfinite(v).all(1)
        bj = scale_byte(np.where(fin, np.abs(np.where(np.isfinite(v), v, 0)).max(1), np.inf))
        b[:, j] = bj
        with np.errstate(all="ignore"):
            y = np.ldexp(np.where(fin[:, None], v, 0.0), (127 - np.minimum(bj, 254))[:, None])
        q[:, j * BLOCK:(j + 1) * BLOCK] = np.where(fin[:, None], e4m3(y), np.nan)
    return q, b


def quantize_weights(w):
    """[M, R, C] -> q [M, R, C], b [M, ceil(R / 128), ceil(C / 128)]."""
    w = np.asarray(w, np.float64)
    m, r, c = w.shape
    q = np.empty_like(w)
    b = np.empty((m, -(-r // BLOCK), -(-c // BLOCK)), np.int64)
    for i in range(m):
        for j in range(b.shape[1]):
            for l in range(b.shape[2]):
                rs, cs = slice(j * BLOCK, (j + 1) * BLOCK), slice(l * BLOCK, (l + 1) * BLOCK)
                q[i, rs, cs], b[i, j, l] = _quantize_block(w[i, rs, cs])
    return q, b


def _scale(b):
    return np.where(b == 255, np.nan, np.ldexp(1.0, np.asarray(b, np.int64) - 127))


def values_rows(q, b):
    """The values that quantised rows stand for."""
    return q * np.repeat(_scale(b), BLOCK, axis=1)[:, : q.shape[1]]


def values_weights(q, b):
    s = np.repeat(np.repeat(_scale(b), BLOCK, axis=1), BLOCK, axis=2)
    return q * s[:, : q.shape[1], : q.shape[2]]


def unpack_words(s, nb):
    """Scale bytes [ceil(nb / 4), N, 4] -> [N, nb]."""
    s = np.asarray(s).astype(np.int64)
    return np.moveaxis(s, 0, 1).reshape(s.shape[1], -1)[:, :nb]


def halves(x):
    """[N, 2F] -> [2N, F]: the gate and the up half of a row as two rows."""
    n, c = x.shape
    return x.reshape(2 * n, c // 2)


# ----------------------------------------------------------------------------- stages
def grouped(rows, off, w):
    """rows of expert e times w[e]^T."""
    out = np.zeros((rows.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            out[lo:hi] = rows[lo:hi] @ w[e].T
    return out


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def swiglu(a):
    g, u = np.split(a, 2, axis=1)
    return g * sigmoid(g) * u


def swiglu_grad(dh, a):
    """[da_gate, da_up] of h = silu(a_gate) a_up."""
    g, u = np.split(a, 2, axis=1)
    s = sigmoid(g)
    return np.concatenate([dh * u * s * (1 + g * (1 - s)), dh * g * s], axis=1)


def ffn_forward(x, off, w1, w2, round16=bf16, quant=None):
    """The expert FFN on (already quantised) values x, w1 [E, 2F, H], w2 [E, H, F];
    quant rounds h between the products."""
    a = round16(grouped(x, off, w1))
    h = round16(swiglu(a))
    o = round16(grouped((quant or identity)(h), off, w2))
    return dict(a=a, h=h, o=o)


def ffn_dgrad(d_o, a, off, w1, w2, round16=bf16, quant=None):
    dh = grouped(d_o, off, np.swapaxes(w2, 1, 2))
    da = round16(swiglu_grad(dh, a))
    return dict(da=da, dx_perm=round16(grouped((quant or identity)(da), off,
                                               np.swapaxes(w1, 1, 2))))


def roundtrip_rows(x):
    return values_rows(*quantize_rows(x))


def roundtrip_halves(x):
    return roundtrip_rows(halves(x)).reshape(x.shape)
