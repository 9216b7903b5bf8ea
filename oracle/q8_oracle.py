"""Rows in 8 bits in fp64: which power of two a block takes, and the e4m3 number nearest to each quotient.
Numbers are looked up in the table of all e4m3 magnitudes, so nothing here is shared with the kernels."""

from __future__ import annotations

import numpy as np

BLOCK, TOP, LEAST = 128, 448.0, -110
# the 127 magnitudes in order: the index is the number's code, so its last bit is the mantissa's
TABLE = np.array([(m if e == 0 else 8 + m) * 2.0 ** (max(e, 1) - 10) for e in range(16) for m in range(8)][:127])


def decode(codes):
    """Values of e4m3 codes (uint8)."""
    c = np.asarray(codes)
    mag = np.where((c & 127) == 127, np.nan, TABLE[np.minimum(c & 127, 126)])
    return np.where(c & 128, -mag, mag)


def nearest(x):
    """The e4m3 values nearest to x (|x| <= 448), ties to the even code."""
    a = np.abs(x)
    hi = np.minimum(np.searchsorted(TABLE, a), 126)
    lo = np.maximum(hi - 1, 0)
    up, down = TABLE[hi] - a, a - TABLE[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.copysign(TABLE[code], x)


def exponents(amax):
    """Smallest e >= -110 with amax / 2^e <= 448."""
    amax = np.asarray(amax, np.float64)
    with np.errstate(divide="ignore"):
        e = np.where(amax > 0, np.ceil(np.log2(np.where(amax > 0, amax, 1.0) / TOP)), LEAST)
    e = np.where(amax / 2.0 ** e > TOP, e + 1, e)
    e = np.where(amax / 2.0 ** (e - 1) <= TOP, e - 1, e)
    return np.maximum(e, LEAST).astype(np.int64)


def blocks(x):
    """Rows x [N][H] as [N][blocks][128], zeros past H."""
    n, h = x.shape
    out = np.zeros((n, -(-h // BLOCK) * BLOCK))
    out[:, :h] = x
    return out.reshape(n, -1, BLOCK)


def quantise(x):
    """(values [N][H], exponents [N][blocks]) of rows x."""
    x = np.asarray(x, np.float64)
    v = blocks(x)
    ok = np.isfinite(v)
    e = exponents(np.where(ok, np.abs(v), 0.0).max(2))
    s = 2.0 ** e[:, :, None]
    q = np.where(ok, nearest(np.where(ok, v, 0.0) / s), np.nan) * s
    return q.reshape(len(x), -1)[:, :x.shape[1]], e


def quantise_weights(w):
    """(values [E][K][N], exponents [E][K blocks][N blocks]) of matrices with a scale per 128 x 128."""
    w = np.asarray(w, np.float64)
    E, K, N = w.shape
    kb, nb = -(-K // BLOCK), -(-N // BLOCK)
    v = np.zeros((E, kb * BLOCK, nb * BLOCK))
    v[:, :K, :N] = w
    v = v.reshape(E, kb, BLOCK, nb, BLOCK)
    e = exponents(np.where(np.isfinite(v), np.abs(v), 0.0).max((2, 4)))
    s = 2.0 ** e[:, :, None, :, None]
    q = nearest(v / s) * s
    return q.reshape(E, kb * BLOCK, nb * BLOCK)[:, :K, :N], e


def half_step(x, scale):
    """Half the distance between the e4m3 numbers around x / scale, times the scale."""
    with np.errstate(divide="ignore"):
        b = np.floor(np.log2(np.abs(x) / scale))
    return 2.0 ** (np.maximum(b, -6) - 4) * scale


def swiglu(a, u):
    return a / (1 + np.exp(-a)) * u


def swiglu_backward(a, u, dh):
    g = 1 / (1 + np.exp(-a))
    return dh * u * g * (1 + a * (1 - g)), dh * a * g


def rms(x, gamma, eps):
    """(y, rstd)"""
    r = 1 / np.sqrt((x * x).mean(1) + eps)
    return x * r[:, None] * gamma, r


def rms_backward(x, gamma, dy, r, ds=None):
    """(dx, dgamma)"""
    xh, d = x * r[:, None], dy * gamma
    dx = r[:, None] * (d - xh * (d * xh).mean(1, keepdims=True))
    return (dx if ds is None else dx + ds), (dy * xh).sum(0)
