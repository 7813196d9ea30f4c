"""Gradient of the RMS norm of rows that are spaced apart: without a residual
rmsnorm returns x itself as h, and rmsnorm_bwd takes it as it is."""

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_04_amd as nv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _bf(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("T,H", [(1, 64), (70, 128), (33, 1000), (9, 1040), (600, 2048), (5, 4104), (300, 7168), (3, 16392)])
def test_gradient_of_a_slice(T, H):
    """Equal bits to those of a contiguous h; what lies between the rows is not read."""
    print(f"[case] T={T} H={H}", flush=True)
    rng = np.random.default_rng(T + H)
    wide = _bf(rng, T, 2 * H + 24)
    wide[:, :8] = wide[:, 8 + H:] = float("nan")
    x, dy, dh, w = wide[:, 8:8 + H], _bf(rng, T, H), _bf(rng, T, H), _bf(rng, H)
    y, h, rstd = nv.rmsnorm(x, w, need_rstd=True)
    assert h is x
    for extra in (dh, None):
        want = nv.rmsnorm_bwd(dy, x.contiguous(), w, rstd, dh=extra)
        got = nv.rmsnorm_bwd(dy, h, w, rstd, dh=extra)
        assert torch.isfinite(got[0].float()).all() and torch.isfinite(got[1]).all()
        for a, b in zip(want, got):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    place = dy.clone()
    assert torch.equal(nv.rmsnorm_bwd(place, h, w, rstd, out=(place, None))[0].view(torch.int16), want[0].view(torch.int16))


def test_gradient_of_a_slice_refuses():
    rng = np.random.default_rng(0)
    wide, dy, w = _bf(rng, 4, 200), _bf(rng, 4, 64), _bf(rng, 64)
    rstd = torch.ones(4, device=DEV)
    for h in (wide[:, 4:68], wide[:, 8:136:2], wide[:3, 8:72], wide[:, 8:80], wide[:, 8:72].float(), wide[:1, 8:72].expand(4, 64)):
        with pytest.raises((ValueError, TypeError, nv.Nvfp4Error)):
            nv.rmsnorm_bwd(dy, h, w, rstd)
    odd = _bf(rng, 4, 68)[:, :64]                         # rows 68 elements apart
    with pytest.raises(nv.Nvfp4Error):
        nv.rmsnorm_bwd(dy, odd, w, rstd)
    with pytest.raises(nv.Nvfp4Error):                    # dx between the rows of h
        at = torch.empty(4 * 128, dtype=torch.bfloat16, device=DEV)
        nv.rmsnorm_bwd(dy, at.view(4, 128)[:, :64], w, rstd, out=(at[64:320].view(4, 64), None))
