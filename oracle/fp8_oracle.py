"""The 8-bit path written out in numpy, in 64 bits: e4m3 values with power-of-two
block scales, the products, the norm and its gradient.

Imports nothing from the library.  Arrays of 8-bit values are uint8 bytes, as
are scales (e8m0: 2^(byte - 127)).
"""

from __future__ import annotations

import numpy as np


def _table() -> np.ndarray:
    """The value of each e4m3 byte: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    t = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = np.nan if (b & 0x7F) == 0x7F else (m * 2.0**-9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        t[b] = -v if b & 0x80 else v
    return t


E4M3 = _table()
_POS = E4M3[:127]  # 0 .. 448, ascending


def e4m3_encode(v) -> np.ndarray:
    """The nearest e4m3 value's byte (ties to the even mantissa) of |v| <= 448; NaN and infinities give 0x7f."""
    v = np.asarray(v, dtype=np.float64)
    a = np.where(np.isfinite(v), np.abs(v), 0)
    hi = np.minimum(np.searchsorted(_POS, a), 126)  # _POS[hi - 1] < a <= _POS[hi]
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(np.isfinite(v), pick | np.where(np.signbit(v), 0x80, 0), 0x7F).astype(np.uint8)


def scale_byte(a) -> np.ndarray:
    """e8m0 byte of the smallest power of two p >= 2^-126 with a <= 448 p (a finite, >= 0)."""
    m, e = np.frexp(np.asarray(a, dtype=np.float64) / 448)  # m in [0.5, 1)
    e = np.where(m == 0.5, e - 1, e)
    return np.maximum(np.where(np.asarray(a) == 0, -126, e), -126) + 127


def power(byte) -> np.ndarray:
    return np.exp2(np.asarray(byte, dtype=np.float64) - 127)


def _finite_max(x, axis):
    return np.where(np.isfinite(x), np.abs(x), 0).max(axis)


def _padded_scales(byte) -> np.ndarray:
    g = byte.shape[-1]
    width = [(0, 0)] * (byte.ndim - 1) + [(0, -g % 4)]
    return np.pad(byte, width, constant_values=127).astype(np.uint8)


def quant_rows(x):
    """x [M, K] -> (bytes [M, Kp], scales [M, Gs])."""
    x = np.asarray(x, dtype=np.float64)
    M, K = x.shape
    g = np.pad(x, ((0, 0), (0, -K % 128))).reshape(M, -1, 128)
    byte = scale_byte(_finite_max(g, 2))
    return e4m3_encode(g / power(byte)[..., None]).reshape(M, -1), _padded_scales(byte)


def quant_weight(w):
    """w [N, K] -> (bytes [N, Kp], scales [ceil(N / 128), Gs])."""
    w = np.asarray(w, dtype=np.float64)
    N, K = w.shape
    b = np.pad(w, ((0, -N % 128), (0, -K % 128)))
    b = b.reshape(b.shape[0] // 128, 128, -1, 128)
    byte = scale_byte(_finite_max(b, (1, 3)))
    q = e4m3_encode(b / power(byte)[:, None, :, None])
    return q.reshape(q.shape[0] * 128, -1)[:N], _padded_scales(byte)


def wide_rows(q, s):
    """The values [M, Kp] that rows of bytes with their scales stand for."""
    g = q.shape[1] // 128
    return E4M3[q] * np.repeat(power(s[:, :g]), 128, axis=1)


def wide_weight(q, s):
    g = q.shape[1] // 128
    return E4M3[q] * np.repeat(np.repeat(power(s[:, :g]), 128, axis=1), 128, axis=0)[: q.shape[0]]


def linear(x, w, bias=None):
    """(y, |x| |w|^T) for wide rows x [M, Kp] and a wide weight [N, Kp]."""
    y = x @ w.T
    return (y if bias is None else y + bias), np.abs(x) @ np.abs(w).T


def experts(x, rows, offsets, weights, bias=None):
    """linear() for rows grouped by expert; rows past offsets[-1] are not part of the result."""
    ys, bs = [], []
    for e in range(len(offsets) - 1):
        r = np.arange(offsets[e], offsets[e + 1])
        y, b = linear(x[r if rows is None else rows[r]], weights[e], None if bias is None else bias[e])
        ys.append(y)
        bs.append(b)
    return np.concatenate(ys), np.concatenate(bs)


def rms_norm(h, weight, eps):
    """(y, r) of h [M, K]."""
    h = np.asarray(h, dtype=np.float64)
    r = 1 / np.sqrt((h * h).mean(1) + eps)
    return h * r[:, None] * (1 if weight is None else weight), r


def rms_norm_bwd(dy, h, weight, r, dresidual=None):
    """(dx, dweight) for dy [M, K]."""
    dy, h = np.asarray(dy, dtype=np.float64), np.asarray(h, dtype=np.float64)
    r = np.asarray(r, dtype=np.float64)[:, None]
    g = dy if weight is None else dy * weight
    dx = r * (g - h * (r * r * (g * h).mean(1, keepdims=True)))
    return (dx if dresidual is None else dx + dresidual), (dy * h * r).sum(0)
