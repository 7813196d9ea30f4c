"""The float64 references of the RMS norm and of the few-token expert layer:
hand-worked values, gradients against central differences, a triple loop."""

import numpy as np
import pytest

from oracle import few, norm


def test_rmsnorm_hand_worked():
    v, rstd = norm.rmsnorm(np.array([[3.0, 4.0, 0.0, 0.0]]), np.array([1.0, 2.0, 3.0, 4.0]), 0.0)
    assert np.allclose(rstd, 0.4) and np.allclose(v, [[1.2, 3.2, 0, 0]])      # mean square 25/4
    assert np.allclose(norm.block_scales(np.array([[448.0] * 128 + [-4.48] * 16])), [[1.0, 0.01]])
    assert norm.block_scales(np.zeros((1, 16)))[0, 0] == 2.0 ** -100 / 448


@pytest.mark.parametrize("T,H,extra", [(1, 8, False), (3, 24, True)])
def test_rmsnorm_gradient_against_differences(T, H, extra):
    rng = np.random.default_rng(H)
    h, w, dy, dh = rng.standard_normal((T, H)), rng.standard_normal(H), rng.standard_normal((T, H)), rng.standard_normal((T, H))
    _, rstd = norm.rmsnorm(h, w, 1e-3)
    dx, dw, _, _ = norm.rmsnorm_bwd(dy, h, w, rstd, dh if extra else None)
    loss = lambda h, w: (dy * norm.rmsnorm(h, w, 1e-3)[0]).sum() + ((dh * h).sum() if extra else 0.0)
    s = 1e-6
    for i in np.ndindex(T, H):
        d = np.zeros((T, H))
        d[i] = s
        assert abs((loss(h + d, w) - loss(h - d, w)) / (2 * s) - dx[i]) < 1e-7
    for i in range(H):
        d = np.zeros(H)
        d[i] = s
        assert abs((loss(h, w + d) - loss(h, w - d)) / (2 * s) - dw[i]) < 1e-7


def test_few_against_a_triple_loop():
    rng = np.random.default_rng(5)
    T, H, I, E, k = 3, 4, 2, 3, 3
    w1, w2 = rng.standard_normal((E, 2 * I, H)), rng.standard_normal((E, H, I))
    x, w = rng.standard_normal((T, H)), rng.standard_normal((T, k))
    ids = np.array([[0, 1, 1], [2, -1, 0], [-1, -1, -1]])
    out, err = few.forward(x, ids, w, lambda e: w1[e], lambda e: w2[e])
    for t in range(T):
        for n in range(H):
            s = 0.0
            for j in range(k):
                if ids[t, j] < 0:
                    continue
                for i in range(I):
                    g = sum(w1[ids[t, j], i, c] * x[t, c] for c in range(H))
                    u = sum(w1[ids[t, j], I + i, c] * x[t, c] for c in range(H))
                    s += w[t, j] * w2[ids[t, j], n, i] * (g / (1 + np.exp(-g)) * u)
            assert abs(out[t, n] - s) < 1e-12
    assert np.all(err[:2] > 0) and np.all(out[2] == 0)
