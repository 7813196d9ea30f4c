"""float64 reference of the RMS norm (residual added, FP8 output) and its gradient.

NumPy only; written apart from the kernels, from the formulas of the header."""

import numpy as np

TINY = 2.0 ** -100


def rmsnorm(h, w, eps):
    """h (T, H), w (H,) -> normalised rows v and 1/rms, both float64."""
    h, w = h.astype(np.float64), w.astype(np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * w, rstd


def block_scales(v):
    """FP8 scales of float64 rows: max(amax, 2^-100) / 448 per 128 columns."""
    T, H = v.shape
    p = np.zeros((T, -(-H // 128) * 128))
    p[:, :H] = np.abs(v)
    return np.maximum(p.reshape(T, -1, 128).max(2), TINY) / 448


def rmsnorm_bwd(dy, h, w, rstd, dh=None):
    """-> dx, dw and the magnitudes that rounding errors are counted against."""
    dy, h, w, rstd = (a.astype(np.float64) for a in (dy, h, w, rstd))
    n, g = h * rstd[:, None], dy * w
    dx = rstd[:, None] * (g - n * (g * n).mean(1, keepdims=True))
    mag = rstd[:, None] * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(1, keepdims=True))
    if dh is not None:
        dx, mag = dx + dh, mag + np.abs(dh)
    return dx, (dy * n).sum(0), mag, np.abs(dy * n).sum(0)
