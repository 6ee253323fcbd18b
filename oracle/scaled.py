"""RMS norm and 8-bit values with scales in float64 NumPy, straight from the formulas."""

import numpy as np

BLOCK = 128
# the 256 e4m3 values by their code
E4M3 = np.array([(-1.0) ** (c >> 7) * (np.nan if c & 127 == 127 else
                                       (c & 7) / 8 * 2.0 ** -6 if c >> 3 & 15 == 0 else
                                       (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7)) for c in range(256)])
POSITIVE = E4M3[:127]  # ascending, from 0 to 448


def rms_norm(t, w=None, eps=1e-6):
    """(y, rstd) over the last axis of t [rows, cols]."""
    t = np.asarray(t, np.float64)
    rstd = 1.0 / np.sqrt((t * t).mean(axis=1) + eps)
    return t * rstd[:, None] * (1.0 if w is None else w), rstd


def rms_norm_backward(dy, t, w, rstd, dtotal=None):
    """(dx, dw), with the rstd given."""
    th = t * rstd[:, None]
    g = dy * (1.0 if w is None else w)
    dx = rstd[:, None] * (g - th * (g * th).mean(axis=1, keepdims=True))
    return dx + (0.0 if dtotal is None else dtotal), (dy * th).sum(axis=0)


def scale_of(values):
    """The scale's byte for a block's values."""
    a = np.abs(values[np.isfinite(values)])
    top = a.max() if a.size else 0.0
    k = -126
    while top > 448 * 2.0 ** k:
        k += 1
    return k + 127


def codes(values):
    """The codes of the nearest e4m3 values, ties to the even code; |values| <= 448, or not finite (NaN)."""
    v = np.asarray(values, np.float64)
    a = np.where(np.isfinite(v), np.abs(v), 0.0)
    hi = np.minimum(np.searchsorted(POSITIVE, a), 126)
    lo = np.maximum(hi - 1, 0)
    up = np.where(POSITIVE[hi] - a == a - POSITIVE[lo], hi % 2 == 0, POSITIVE[hi] - a < a - POSITIVE[lo])
    c = np.where(up, hi, lo) | np.where(np.signbit(v), 128, 0)
    return np.where(np.isfinite(v), c, 127).astype(np.uint8)  # (a NaN's sign is of no matter)


def quantize(x, height=1):
    """(codes, scales) of x [rows, cols], a scale for each `height` x 128 values."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    q = np.empty((rows, cols), np.uint8)
    s = np.empty((-(-rows // height), -(-cols // BLOCK)), np.uint8)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = np.s_[i * height:(i + 1) * height, j * BLOCK:(j + 1) * BLOCK]
            s[i, j] = scale_of(x[at])
            q[at] = codes(x[at] / 2.0 ** (int(s[i, j]) - 127))
    return q, s


def values(q, scales, height=1):
    """What codes q [rows, cols] and their scales stand for."""
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    s = np.repeat(np.repeat(s, height, axis=0)[:q.shape[0]], BLOCK, axis=1)[:, :q.shape[1]]
    return E4M3[q] * s
