"""The expert layer for a few tokens with weights and tokens of sizes far from one
whose products are ordinary numbers: what the scales carry must not overflow or
vanish on the way."""

import numpy as np
import pytest
import torch

import test_gpu_few as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("sx,s1,s2", [(1e20, 1e-20, 1e10), (1e-20, 1e20, 1e-10), (1e28, 1e-28, 1.0), (1e-28, 1e28, 1.0),
                                      (1.0, 1.0, 1e-27), (1.0, 1.0, 1e28), (1e-12, 1.0, 1e24), (1e9, 1.0, 1e-25),
                                      (1e33, 1e-29, 1.0), (1.0, 2e16, 1e-28)])   # next to 2^112, FP8's limit of x and h
def test_few_scales(monkeypatch, fmt, sx, s1, s2):
    rng = np.random.default_rng(17)
    T, H, I, E, k = 6, 384, 256, 4, 2
    sizes = iter([s1, s2])
    plain = B._bf
    monkeypatch.setattr(B, "_bf", lambda rng, *shape, scale=1.0: plain(rng, *shape, scale=scale * next(sizes)))
    make, call = B.MAKE[fmt]
    args, w1, w2 = make(rng, E, H, I)
    x = plain(rng, T, H, scale=sx)
    ids, w = B._routing(rng, T, E, k)
    out = call(x.to(B.DEV), torch.from_numpy(ids).to(B.DEV), torch.from_numpy(w).to(B.DEV), *args)
    assert torch.isfinite(out.float()).all() and (out != 0).any()
    B._check(out, x, ids, w, w1, w2)
