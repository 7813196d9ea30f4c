"""RMS norm and its gradient where a tensor passes 2^25 elements (rows then go past
the caches), every width's kernel, and with one tensor in several places.

Bounds as for small calls: 40 roundings of 2^-24 in 1/rms and the rows before
their rounding, 80 in dx against its terms' magnitudes, and in dw a workgroup's
rows in order (a 256th of them, or a sixteenth of that where sixteen share one)
and 70 more."""

import pytest
import torch

import nvfp4_block_scaled_04_amd as nv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("H", [128, 512, 1008, 2048, 4096, 7168, 16384, 32768])
def test_rmsnorm_past_the_caches(H, wide):
    print(f"[case] H={H} wide={wide}", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(H)
    T = (1 << 25) // H + 3
    bf = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=torch.bfloat16)
    x, r, dy, dh = (bf(T, H) for _ in range(4))
    w = 1 + 0.3 * torch.randn((H,), generator=g, device=DEV)
    w = w if wide else w.to(torch.bfloat16)
    q, sf, y, h, rstd = nv.fp8_rmsnorm(x, w, residual=r, eps=1e-5, need_y=True, need_rstd=True)
    assert torch.equal(h.view(torch.int16), (x.float() + r.float()).to(torch.bfloat16).view(torch.int16))
    hd, wd = h.double(), w.double()
    s = 1 / torch.sqrt(hd.square().mean(1) + 1e-5)
    assert ((rstd.double() - s).abs() <= 40 * U * s).all()
    v = hd * s[:, None] * wd
    assert ((y.double() - v).abs() <= (2.0 ** -8 + 41 * U) * v.abs() + 1e-38).all()
    KB = (H + 127) // 128
    b = torch.nn.functional.pad(v.abs(), (0, KB * 128 - H)).view(T, KB, 128).amax(2) / 448
    assert ((sf.double() - b).abs() <= 42 * U * b).all()
    at = lambda t: t.double().repeat_interleave(128, 1)[:, :H]
    assert ((q.double() * at(sf) - v).abs() <= (2.0 ** -4 + 64 * U) * v.abs() + 1.001 * 2.0 ** -10 * at(b)).all()
    del q, sf, y, v, b, x, r
    dx, dw = nv.rmsnorm_bwd(dy, h, w, rstd, dh=dh)
    rs = rstd.double()[:, None]
    n, d = hd * rs, dy.double()
    gw = d * wd
    dot = (gw * n).mean(1, keepdim=True)
    ref = rs * (gw - n * dot) + dh.double()
    mag = rs * (gw.abs() + n.abs() * (gw * n).abs().mean(1, keepdim=True)) + dh.double().abs()
    assert ((dx.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 81 * U * mag).all()
    assert ((dw.double() - (d * n).sum(0)).abs() <= (T / 256 + 70) * U * (d * n).abs().sum(0)).all()


def test_one_tensor_in_several_places():
    """The residual that is x, h over both; the rows' gradient that is h's too, dx over it."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    for T, H in ((5, 136), (33, 1040), (3, 7168), (2, 16392)):
        x = torch.randn((T, H), generator=g, device=DEV, dtype=torch.bfloat16)
        dy, w = torch.randn_like(x), torch.randn((H,), generator=g, device=DEV)
        want = nv.rmsnorm(x, w, residual=x.clone(), need_rstd=True)
        place = x.clone()
        y, h, rstd = nv.rmsnorm(place, w, residual=place, need_rstd=True, out=(None, place, None))
        assert h is place
        for a, b in zip(want, (y, h, rstd)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        want = nv.rmsnorm_bwd(dy, h, w, rstd, dh=dy.clone())
        place = dy.clone()
        got = nv.rmsnorm_bwd(place, h, w, rstd, dh=place, out=(place, None))
        assert got[0] is place
        for a, b in zip(want, got):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
