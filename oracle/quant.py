"""fp64 reference of quantised pages and of the norms of queries and keys. Test
infrastructure; shares no code with the CUDA path."""
import math

import numpy as np


def e4m3_values():
    """The 256 values: sign, four bits of exponent (bias 7), three of mantissa;
    the largest pattern of either sign is NaN."""
    out = np.empty(256)
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        x = math.nan if b & 127 == 127 else \
            (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        out[b] = -x if b & 128 else x
    return out


VALUES = e4m3_values()
_UP = VALUES[:127]  # 0 .. 448


def exponent(a):
    """Least e with a <= 448 2^e, kept within [-64, 63]."""
    e = -64
    while e < 63 and a > 448 * 2.0 ** e:
        e += 1
    return e


def quantise(x):
    """x [..., D] -> codes (uint8) and e + 127 (uint8) of each head."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x)
    mag = np.abs(np.where(fine, x, 0.0))
    border = 448 * 2.0 ** np.arange(-64, 63)  # e is the number of borders passed, less 64
    e = np.searchsorted(border, mag.max(-1), side="left") - 64
    y = np.minimum(mag * 2.0 ** -e.astype(np.float64)[..., None], 448.0)
    hi = np.clip(np.searchsorted(_UP, y), 0, 126)  # nearest of two neighbours, ties to even
    lo = np.maximum(hi - 1, 0)
    up, down = _UP[hi] - y, y - _UP[lo]
    c = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    c = np.where(np.signbit(x), c | 128, c)
    return np.where(fine, c, 127).astype(np.uint8), (e + 127).astype(np.uint8)


def value(codes, scale):
    """What codes [..., D] with their bytes [...] stand for."""
    return VALUES[codes] * 2.0 ** (scale.astype(np.float64) - 127)[..., None]


def norm(x, w, eps):
    """x [..., D] by the root of its mean square, times w (None: x itself)."""
    if w is None:
        return np.asarray(x, np.float64)
    return x * w / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
