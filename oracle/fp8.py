"""FP8 with a scale for each block of 128, and the gradients around the experts.

Formulas (b runs over blocks of 128 columns; the last may be shorter):
  quantise     m = max(amax of the block, 2^-100); scale = m / 448, r = 448 / m,
               code = E4M3(x * r); fp32 operations, round to nearest even; a NaN
               does not count in amax
  SwiGLU       h = gate / (1 + exp(-gate)) * up
  product      c[d][n] = sum_b sa[s][b] sw[n/128][b] sum_{k in b} a[s][k] w[n][k]
  dispatch     rows[inv[t*k+j]] = x[t] for inv < n, else 0
  gradients    dx[t] = sum_j drows[inv[t*k+j]];  dy[inv] = w * dout;
               dw = <dout, y[inv]>;  dlogits[ids_j] += w_j (dw_j - sum_i w_i dw_i)
Sums are in float64 on exactly decoded operands.
"""

import numpy as np

from . import formats as F

BLOCK = 128
FLOOR = np.float32(2.0 ** -100)
_TABLE = F.e4m3_decode(np.arange(0x7F))          # 0 .. 448, ascending


def e4m3_encode(v):
    """E4M3 byte nearest to each v (|v| <= 464: more would round past 448),
    ties to the even code, sign bit taken from v; 0x7F or 0xFF for a NaN."""
    v = np.asarray(v)
    nan = np.isnan(v)
    mag = np.where(nan, 0.0, np.minimum(np.abs(v.astype(np.float64)), 448.0))
    code = np.where(nan, 0x7F, F._nearest_ties_even(_TABLE, mag)).astype(np.uint8)
    return code | (np.signbit(v).astype(np.uint8) << 7)


def _amax_blocks(x, br):
    R, C = x.shape
    p = np.zeros((-(-R // br) * br, -(-C // BLOCK) * BLOCK), np.float32)
    p[:R, :C] = np.fmax(np.abs(x), 0)
    return p.reshape(p.shape[0] // br, br, p.shape[1] // BLOCK, BLOCK).max(axis=(1, 3))


def quantize(x, block_rows=1):
    """x (R, C) float32 -> (codes uint8 (R, C), scales float32) with one scale
    per block_rows x 128 block (1: activations, 128: weights)."""
    x = np.asarray(x, np.float32)
    R, C = x.shape
    m = np.maximum(_amax_blocks(x, block_rows), FLOOR)
    r = np.float32(448.0) / m
    rr = np.repeat(np.repeat(r, block_rows, 0)[:R], BLOCK, 1)[:, :C]
    with np.errstate(invalid="ignore"):                  # infinity times r = 0
        return e4m3_encode(x * rr), m / np.float32(448.0)


def decode(q, sf, block_rows=1):
    """The float64 values that codes and scales stand for."""
    R, C = q.shape
    s = np.repeat(np.repeat(np.asarray(sf, np.float64), block_rows, 0)[:R], BLOCK, 1)[:, :C]
    return F.e4m3_decode(q) * s


def swiglu(x):
    """[gate | up] -> silu(gate) * up in float64."""
    x = np.asarray(x, np.float64)
    I = x.shape[1] // 2
    with np.errstate(over="ignore"):
        return x[:, :I] / (1.0 + np.exp(-x[:, :I])) * x[:, I:]


def _peaks(x):
    """Largest magnitude of every eight consecutive columns."""
    R, C = x.shape
    p = np.zeros((R, -(-C // 8) * 8))
    p[:, :C] = np.abs(x)
    return p.reshape(R, -1, 8).max(2)


def grouped_product(a, w_list, offsets, rows):
    """a (R, K) float64, w_list[e] (N, K) float64, rows[d] = A row of d (-1: a
    row of zeros) -> (c (M, N) with rows from offsets[-1] on zero, the sum of
    the terms' magnitudes (M, N), and a bound of the sum, over every eight
    consecutive terms, of the largest of them (M, N))."""
    M, N = len(rows), w_list[0].shape[0]
    c, mag, peak = np.zeros((M, N)), np.zeros((M, N)), np.zeros((M, N))
    az = np.vstack([a, np.zeros((1, a.shape[1]))])
    for e, w in enumerate(w_list):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            x = az[rows[lo:hi]]
            c[lo:hi] = x @ w.T
            mag[lo:hi] = np.abs(x) @ np.abs(w).T
            peak[lo:hi] = _peaks(x) @ _peaks(w).T
    return c, mag, peak


def dispatch(x, inv, n, k):
    T, H = x.shape
    rows = np.zeros((T * k, H), x.dtype)
    for f in range(T * k):
        if inv[f] < n:
            rows[inv[f]] = x[f // k]
    return rows


def dispatch_bwd(drows, inv, n, k):
    """-> (dx float64 (T, H), sum of magnitudes)."""
    T = len(inv) // k
    dx, mag = np.zeros((T, drows.shape[1])), np.zeros((T, drows.shape[1]))
    for f in range(T * k):
        if inv[f] < n:
            dx[f // k] += drows[inv[f]]
            mag[f // k] += np.abs(drows[inv[f]])
    return dx, mag


def combine_bwd(dout, y, inv, w, n):
    """-> (dy float32 products (T*k, H), dw float64 (T, k), dw's sum of magnitudes)."""
    T, k = w.shape
    dy = np.zeros((T * k, dout.shape[1]), np.float32)
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            d = inv[t * k + j]
            if d < n:
                dy[d] = np.float32(w[t, j]) * dout[t].astype(np.float32)
                p = dout[t].astype(np.float64) * y[d].astype(np.float64)
                dw[t, j], mag[t, j] = p.sum(), np.abs(p).sum()
    return dy, dw, mag


def router_bwd(ids, w, dw, E):
    """-> (dlogits float64 (T, E), bound of the terms' magnitudes)."""
    ids = np.asarray(ids)
    w, dw = np.asarray(w, np.float64), np.asarray(dw, np.float64)
    T, k = ids.shape
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    mean, mm = (w * dw).sum(1), np.abs(w * dw).sum(1)
    for t in range(T):
        for j in range(k):
            if 0 <= ids[t, j] < E:
                out[t, ids[t, j]] += w[t, j] * (dw[t, j] - mean[t])
                mag[t, ids[t, j]] += abs(w[t, j]) * (abs(dw[t, j]) + mm[t])
    return out, mag
