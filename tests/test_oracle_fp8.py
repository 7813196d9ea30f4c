"""Pins of the FP8 block oracle and of the gradient formulas (CPU): the codec
against the format's table, hand-worked blocks, triple loops, and gradients
against central differences of the formulas they belong to."""

import numpy as np
import pytest

from oracle import formats as F
from oracle import fp8 as P


def test_encode_is_nearest_even_and_keeps_the_sign():
    vals = F.e4m3_decode(np.arange(0x7F))
    assert np.array_equal(P.e4m3_encode(vals), np.arange(0x7F))
    assert np.array_equal(P.e4m3_encode(-vals), np.arange(0x7F) | 0x80)
    mid = (vals[:-1] + vals[1:]) / 2
    even = np.where(np.arange(126) % 2 == 0, np.arange(126), np.arange(1, 127))
    assert np.array_equal(P.e4m3_encode(mid), even)
    assert np.array_equal(P.e4m3_encode(np.nextafter(mid, 0)), np.arange(126))
    assert np.array_equal(P.e4m3_encode(np.nextafter(mid, 500)), np.arange(1, 127))


def test_hand_worked_blocks():
    # amax 224: scale 0.5, r = 2; 1 -> 2 (0x40), -0.9375 -> -1.875 (0xBF), 224 -> 448 (0x7E)
    x = np.zeros((1, 144), np.float32)
    x[0, :3] = [1.0, -0.9375, 224.0]
    x[0, 128] = -448.0                       # its own (16-wide) block: scale 1
    q, sf = P.quantize(x)
    assert list(q[0, :3]) == [0x40, 0xBF, 0x7E] and q[0, 128] == 0xFE
    assert sf.shape == (1, 2) and list(sf[0]) == [0.5, 1.0]
    # a block of zeros: codes 0, scale 2^-100 / 448 (positive and finite)
    q, sf = P.quantize(np.zeros((1, 16), np.float32))
    assert not q.any() and sf[0, 0] == np.float32(2.0 ** -100) / np.float32(448)


def test_weight_blocks_are_128_square():
    x = np.zeros((130, 256), np.float32)
    x[0, 0], x[129, 0], x[127, 255] = 448.0, 1.0, 224.0
    _, sf = P.quantize(x, 128)
    one = np.float32(1) / np.float32(448)
    floor = np.float32(2.0 ** -100) / np.float32(448)
    assert np.array_equal(sf, np.array([[1.0, 0.5], [one, floor]], np.float32))


@pytest.mark.parametrize("br", [1, 128])
def test_round_trip_error_is_half_a_step(br):
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((133, 272)) * np.exp(rng.standard_normal((133, 1)))).astype(np.float32)
    q, sf = P.quantize(x, br)
    s = np.repeat(np.repeat(sf.astype(np.float64), br, 0)[:133], 128, 1)[:, :272]
    v = np.abs(x / s)
    step = np.exp2(np.floor(np.log2(np.maximum(v, 2.0 ** -6))) - 3)
    # half a code step, and the roundings of scale, r and the product (2^-24 each) of a value <= 448
    assert np.all(np.abs(P.decode(q, sf, br) - x) <= s * (step / 2 + 448 * 3 * 2.0 ** -24))
    assert np.abs(F.e4m3_decode(q)).max() == 448.0


def test_product_is_the_triple_loop():
    rng = np.random.default_rng(4)
    a = rng.standard_normal((5, 20))
    w = [rng.standard_normal((3, 20)) for _ in range(3)]
    off, rows = [0, 2, 2, 5], np.array([4, -1, 0, 4, 2, 1])
    c, mag, peak = P.grouped_product(a, w, off, rows)
    for d in range(6):
        e = 0 if d < 2 else 2
        for n in range(3):
            t = [a[rows[d], k] * w[e][n, k] for k in range(20)] if d < 5 and rows[d] >= 0 else [0.0]
            assert abs(c[d, n] - sum(t)) < 1e-12 and abs(mag[d, n] - sum(map(abs, t))) < 1e-12
            assert peak[d, n] >= sum(max(map(abs, t[g:g + 8])) for g in range(0, len(t), 8)) - 1e-12


def _route(T, k, n_valid, rng):
    perm = rng.permutation(T * k)
    return perm, n_valid


def test_gradients_are_differences_of_the_forward():
    rng = np.random.default_rng(5)
    T, k, H, E = 4, 3, 5, 7
    inv, n = _route(T, k, 10, rng)
    x = rng.standard_normal((T, H))
    y = rng.standard_normal((T * k, H))
    lg = rng.standard_normal((T, E))
    ids = np.argsort(-lg, 1)[:, :k]
    dout = rng.standard_normal((T, H))
    drows = rng.standard_normal((T * k, H))
    eps = 1e-6

    def weights(lg):
        v = np.take_along_axis(lg, ids, 1)
        e = np.exp(v - v.max(1, keepdims=True))
        return e / e.sum(1, keepdims=True)

    def combine(y, w):
        out = np.zeros((T, H))
        for f in range(T * k):
            if inv[f] < n:
                out[f // k] += w[f // k, f % k] * y[inv[f]]
        return out

    def diff(f, v):
        g = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            p, m = v.copy(), v.copy()
            p[i] += eps
            m[i] -= eps
            g[i] = (f(p) - f(m)) / (2 * eps)
        return g

    w = weights(lg)
    dx, _ = P.dispatch_bwd(drows, inv, n, k)
    np.testing.assert_allclose(dx, diff(lambda v: (P.dispatch(v, inv, n, k) * drows).sum(), x), atol=1e-8)
    dy, dw, _ = P.combine_bwd(dout, y, inv, w, n)
    np.testing.assert_allclose(dy, diff(lambda v: (combine(v, w) * dout).sum(), y), atol=1e-6)
    np.testing.assert_allclose(dw, diff(lambda v: (combine(y, v) * dout).sum(), w), atol=1e-8)
    dl, _ = P.router_bwd(ids, w, dw, E)
    np.testing.assert_allclose(dl, diff(lambda v: (combine(y, weights(v)) * dout).sum(), lg), atol=1e-8)


def test_dispatch_places_rows_and_zeroes_the_rest():
    inv = np.array([2, 0, 3, 1])
    x = np.array([[1.0, 2.0], [3.0, 4.0]])
    rows = P.dispatch(x, inv, 3, 2)
    assert np.array_equal(rows, [[1, 2], [0, 0] if inv[3] >= 3 else [3, 4], [1, 2], [0, 0]])


def test_swiglu_closed_forms():
    x = np.array([[0.0, 100.0, -100.0, 2.0, 3.0, 5.0]])
    h = P.swiglu(x)
    assert h[0, 0] == 0 and abs(h[0, 1] - 300) < 1e-9 and abs(h[0, 2]) < 1e-30


def test_nan_keeps_to_itself_and_infinity_takes_its_block():
    x = np.zeros((2, 256), np.float32)
    x[0, :3] = [np.nan, 448.0, -1.0]
    x[0, 128:131] = [-np.nan, np.nan, 0.0]               # no finite magnitude: the floor
    x[1, :3] = [-np.inf, 5.0, np.nan]
    x[1, 128] = 224.0
    q, sf = P.quantize(x)
    assert list(q[0, :3]) == [0x7F, 0x7E, 0xB8] and sf[0, 0] == 1.0
    assert q[0, 128] & 0x7F == 0x7F and q[0, 129] == 0x7F and sf[0, 1] == np.float32(2.0 ** -100) / np.float32(448)
    assert q[1, 0] & 0x7F == 0x7F and q[1, 1] == 0 and q[1, 2] == 0x7F and sf[1, 0] == np.inf
    assert q[1, 128] == 0x7E and sf[1, 1] == 0.5
