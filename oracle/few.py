"""float64 reference of the expert layer whose activations are not quantised,
with the bound on what fp32 sums and the rounding of h may change.

NumPy only.  Weights come as float64 values: w1[e] (2I, H) with rows
[gate | up], w2[e] (H, I)."""

import numpy as np


def silu(g):
    return g / (1.0 + np.exp(-g))


def forward(x, ids, topk_w, w1, w2, h_bits=16, h_floor=0.0):
    """x (T, H), ids and topk_w (T, k); w1, w2: functions of an expert id ->
    (out (T, H), err (T, H)): err bounds the difference of a kernel whose
    products are exact, whose sums may lose 2^-23 of the magnitude that has gone
    in at every addition (32 in a matrix instruction, at most 8 of these in a row
    over 128 columns, then one addition for every 1024 columns,
    and 24 for scales, join and division), and whose h keeps h_bits bits, or is off
    by h_floor of the largest of its 128, plus half a BF16 step of out."""
    T, H = x.shape
    E_live = sorted({int(e) for e in ids.ravel() if e >= 0})
    out, err = np.zeros((T, H)), np.zeros((T, H))
    x = x.astype(np.float64)
    u23 = 2.0 ** -23
    for e in E_live:
        a, b = w1(e), w2(e)
        I = b.shape[1]
        c1 = (152 + H / 1024) * u23
        c2 = (280 + len(E_live) * (I / 1024 + 1)) * u23
        for t in range(T):
            js = np.nonzero(ids[t] == e)[0]
            if not len(js):
                continue
            c = topk_w[t, js].astype(np.float64).sum()
            cm = np.abs(topk_w[t, js].astype(np.float64)).sum()
            y, m = a @ x[t], np.abs(a) @ np.abs(x[t])
            g, u, eg, eu = y[:I], y[I:], c1 * m[:I], c1 * m[I:]
            h = silu(g) * u
            # silu's slope is below 1.1 in size
            eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(silu(g)) * eu + (2.0 ** -h_bits + 16 * u23) * np.abs(h)
            if h_floor:
                eh += h_floor * np.repeat(np.maximum.reduceat(np.abs(h) + eh, np.arange(0, I, 128)), 128)[:I]
            out[t] += c * (b @ h)
            err[t] += cm * (np.abs(b) @ (eh + c2 * np.abs(h)))
    return out, err + 2.0 ** -8 * (np.abs(out) + err) + 1e-37
