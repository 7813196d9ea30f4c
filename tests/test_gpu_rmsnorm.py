"""GPU parity of the RMS norm (residual, BF16 and FP8 outputs) and its gradient.

Tolerances.  h and the choice of its rounding are bit-exact.  A lane sums up to
32 squares in order, then 6 exchanges, up to 16 waves and eps: under 64 roundings
of 2^-24 in the mean, half of that in 1/rms, and a few for root, division and
products, so v and 1/rms are within 40 * 2^-24.  BF16 adds half a step (2^-8), an
E4M3 code half a step of itself (2^-4) or of the smallest (2^-10 scales).  dx: 80
roundings against its terms' magnitudes; dw: a workgroup's rows in order (T/256 at
most), then up to 16 groups of rows, 16 workgroups' sums and 32 of those."""

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_04_amd as nv
from oracle import formats as F
from oracle import norm as N
from parity import bf16_values, host

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def _bf(rng, *shape, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(torch.bfloat16)


def _weight(rng, H, wide):
    w = torch.from_numpy((1 + 0.3 * rng.standard_normal(H)).astype(np.float32))
    return w if wide else w.to(torch.bfloat16)


def _check(T, H, x, r, w, eps, got, need_q=True):
    """(q, sf, y, h, rstd) of inputs on the host against float64."""
    q, sf, y, h, rstd = got
    want_h = x if r is None else (x.float() + r.float()).to(torch.bfloat16)
    assert torch.equal(h.cpu().view(torch.int16), want_h.view(torch.int16))
    v, s = N.rmsnorm(want_h.float().numpy(), w.float().numpy(), eps)
    assert np.all(np.abs(host(rstd) - s) <= 40 * U * s)
    assert np.all(np.abs(bf16_values(host(y)) - v) <= (2.0 ** -8 + 41 * U) * np.abs(v) + 1e-38)
    if need_q:
        b = N.block_scales(v)
        got_sf = host(sf).astype(np.float64)
        assert np.all(np.abs(got_sf - b) <= 42 * U * b)
        codes = F.e4m3_decode(host(q.view(torch.uint8))) * np.repeat(got_sf, 128, 1)[:, :H]
        assert np.all(np.abs(codes - v) <= (2.0 ** -4 + 64 * U) * np.abs(v) + 2.0 ** -10 * np.repeat(b, 128, 1)[:, :H] * 1.001)


CASES = [(1, 16), (3, 128), (5, 144), (130, 128), (2, 512), (7, 528), (3, 1024), (65, 1040), (2, 2048), (3, 2064),
         (4, 4096), (3, 4112), (1, 7168), (300, 7168), (2, 8192), (2, 8208), (1, 16384), (2, 32768)]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T,H", CASES)
def test_rmsnorm(T, H, wide):
    print(f"[case] rmsnorm T={T} H={H} wide={wide}", flush=True)
    rng = np.random.default_rng(T * 7 + H)
    x, r, w = _bf(rng, T, H), _bf(rng, T, H, scale=3.0), _weight(rng, H, wide)
    x[0, : H // 2] *= 64
    if T > 1:
        x[1], r[1] = 0, 0                                 # a row of zeros
    for res in (r, None):
        dev = None if res is None else res.to(DEV)
        got = nv.fp8_rmsnorm(x.to(DEV), w.to(DEV), residual=dev, eps=1e-5, need_y=True, need_rstd=True)
        _check(T, H, x, res, w, 1e-5, got)
        y, h, s = nv.rmsnorm(x.to(DEV), w.to(DEV), residual=dev, eps=1e-5, need_rstd=True)
        assert torch.equal(y.view(torch.int16), got[2].view(torch.int16)) and torch.equal(s, got[4])
        only = nv.fp8_rmsnorm(x.to(DEV), w.to(DEV), residual=dev, eps=1e-5)
        assert only[2] is None and only[4] is None
        assert torch.equal(only[0].view(torch.uint8), got[0].view(torch.uint8)) and torch.equal(only[1], got[1])


@pytest.mark.parametrize("T,H", [(3, 8), (2, 24), (9, 136), (4, 1000), (3, 2056), (2, 4104), (2, 8200)])
def test_rmsnorm_of_eights(T, H):
    """BF16 outputs take any multiple of eight columns."""
    rng = np.random.default_rng(H)
    x, r, w = _bf(rng, T, H), _bf(rng, T, H), _weight(rng, H, True)
    y, h, s = nv.rmsnorm(x.to(DEV), w.to(DEV), residual=r.to(DEV), need_rstd=True)
    _check(T, H, x, r, w, 1e-6, (None, None, y, h, s), need_q=False)


@pytest.mark.parametrize("scale", [1e-30, 1e-18, 1e-3, 1e10, 1e18])
def test_rmsnorm_magnitudes(scale):
    rng = np.random.default_rng(11)
    x, w = _bf(rng, 5, 528, scale=scale), _weight(rng, 528, False)
    got = nv.fp8_rmsnorm(x.to(DEV), w.to(DEV), eps=1e-12, need_y=True, need_rstd=True)
    _check(5, 528, x, None, w, 1e-12, got)


def test_rmsnorm_rows_apart_and_in_place():
    rng = np.random.default_rng(3)
    T, H = 9, 1040
    wide = _bf(rng, T, 3 * H + 8).to(DEV)
    x, r = wide[:, :H], wide[:, 2 * H:3 * H]
    w = _weight(rng, H, True).to(DEV)
    want = nv.fp8_rmsnorm(x.contiguous(), w, residual=r.contiguous(), need_y=True, need_rstd=True)
    got = nv.fp8_rmsnorm(x, w, residual=r, need_y=True, need_rstd=True)
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for at in (0, 1):                                     # h over x, over the residual
        pair = [x.contiguous(), r.contiguous()]
        q, sf, y, h, s = nv.fp8_rmsnorm(pair[0], w, residual=pair[1], out=(None, None, None, pair[at], None))
        assert h is pair[at] and torch.equal(h.view(torch.int16), want[3].view(torch.int16))
        assert torch.equal(q.view(torch.uint8), want[0].view(torch.uint8))
    one = nv.rmsnorm(wide[2:3, :H], w)                    # one row of a wider tensor
    assert torch.equal(one[0], nv.rmsnorm(x.contiguous(), w)[0][2:3])
    with pytest.raises(ValueError):
        nv.rmsnorm(x, w, out=(None, x, None))             # no residual: h is x
    with pytest.raises(ValueError):
        nv.rmsnorm(x, w[:-1])
    with pytest.raises(ValueError):
        nv.rmsnorm(x, w, residual=r[:-1])
    with pytest.raises(TypeError):
        nv.rmsnorm(x.float(), w)
    with pytest.raises(nv.Nvfp4Error):
        nv.rmsnorm(x, w, eps=0.0)
    with pytest.raises(nv.Nvfp4Error):
        nv.fp8_rmsnorm(wide[:, :24].contiguous(), w[:24].contiguous())


def test_rmsnorm_non_finite_rows_stay_their_own():
    rng = np.random.default_rng(8)
    x, w = _bf(rng, 6, 272), _weight(rng, 272, True)
    x[1, 3], x[4, 5] = float("nan"), float("inf")
    q, sf, y, h, s = nv.fp8_rmsnorm(x.to(DEV), w.to(DEV), need_y=True, need_rstd=True)
    keep = [0, 2, 3, 5]
    _check(4, 272, x[keep], None, w, 1e-6, (q[keep], sf[keep], y[keep], h[keep], s[keep]))
    assert torch.isnan(s[1]) and torch.isnan(y[1]).all() and s[4] == 0 and torch.isnan(y[4, 5])


def test_outputs_stay_inside_their_buffers():
    rng = np.random.default_rng(4)
    for T, H in [(3, 16), (5, 272), (2, 7168), (1, 8208)]:
        x, r, w = _bf(rng, T, H).to(DEV), _bf(rng, T, H).to(DEV), _weight(rng, H, False).to(DEV)
        kb = (H + 127) // 128
        bufs = [torch.full((T * H + 64,), 7, dtype=torch.uint8, device=DEV), torch.full((T * kb + 64,), 7.0, device=DEV),
                torch.full((T * H + 64,), 7.0, dtype=torch.bfloat16, device=DEV),
                torch.full((T * H + 64,), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((T + 64,), 7.0, device=DEV)]
        n = [T * H, T * kb, T * H, T * H, T]
        shape = [(T, H), (T, kb), (T, H), (T, H), (T,)]
        out = [b[32:32 + m].view(s) for b, m, s in zip(bufs, n, shape)]
        out[0] = out[0].view(torch.float8_e4m3fn)
        nv.fp8_rmsnorm(x, w, residual=r, out=tuple(out))
        dx, dw = bufs[2][32:32 + T * H].view(T, H), torch.full((H + 64,), 7.0, device=DEV)
        nv.rmsnorm_bwd(x, r, w, out[4], out=(dx, dw[32:32 + H]))
        for b in bufs + [dw]:
            assert torch.all(b[:32].float() == 7) and torch.all(b[-32:].float() == 7)


GRADS = [(1, 8), (3, 128), (70, 128), (9000, 128), (5, 136), (7, 1000), (2100, 1024), (33, 1032), (3, 2048), (5, 2056),
         (2, 4104), (600, 4096), (3, 7168), (1100, 7168), (2, 8200), (3, 16384), (520, 8208), (2, 32768)]


@pytest.mark.parametrize("T,H", GRADS)
def test_rmsnorm_gradient(T, H):
    print(f"[case] rmsnorm gradient T={T} H={H}", flush=True)
    rng = np.random.default_rng(T + H)
    wide = bool(T % 2)
    h, dy, dh, w = _bf(rng, T, H), _bf(rng, T, H), _bf(rng, T, H), _weight(rng, H, wide)
    _, s = N.rmsnorm(h.float().numpy(), w.float().numpy(), 1e-6)
    rstd = torch.from_numpy(s.astype(np.float32))
    for extra in (dh, None):
        dev = None if extra is None else extra.to(DEV)
        dx, dw = nv.rmsnorm_bwd(dy.to(DEV), h.to(DEV), w.to(DEV), rstd.to(DEV), dh=dev)
        rx, rw, mx, mw = N.rmsnorm_bwd(dy.float().numpy(), h.float().numpy(), w.float().numpy(), rstd.numpy(),
                                       None if extra is None else extra.float().numpy())
        assert np.all(np.abs(bf16_values(host(dx)) - rx) <= 2.0 ** -8 * np.abs(rx) + 81 * U * mx)
        assert np.all(np.abs(host(dw) - rw) <= (T / 256 + 70) * U * mw)
        only, none = nv.rmsnorm_bwd(dy.to(DEV), h.to(DEV), w.to(DEV), rstd.to(DEV), dh=dev, need_dw=False)
        assert none is None and torch.equal(only.view(torch.int16), dx.view(torch.int16))
        over = dy.to(DEV) if extra is None else dev
        place = nv.rmsnorm_bwd(over if extra is None else dy.to(DEV), h.to(DEV), w.to(DEV), rstd.to(DEV), dh=dev, out=(over, None))
        assert place[0] is over and torch.equal(over.view(torch.int16), dx.view(torch.int16))
        assert torch.equal(place[1], dw)


def test_rmsnorm_gradient_against_differences():
    """Of the whole chain on the device: the directional derivative of sum(dy * y)
    by differences of the float64 formula at the same points."""
    rng = np.random.default_rng(2)
    T, H = 4, 264
    h, dy, w = _bf(rng, T, H), _bf(rng, T, H), _weight(rng, H, True)
    y, _, rstd = nv.rmsnorm(h.to(DEV), w.to(DEV), need_rstd=True)
    dx, dw = nv.rmsnorm_bwd(dy.to(DEV), h.to(DEV), w.to(DEV), rstd)
    hv, wv, dv = h.double().numpy(), w.double().numpy(), dy.double().numpy()
    loss = lambda a, b: (dv * N.rmsnorm(a, b, 1e-6)[0]).sum()
    for seed in range(3):
        d, e = np.random.default_rng(seed).standard_normal((2, T, H))
        num = (loss(hv + 1e-5 * d, wv) - loss(hv - 1e-5 * d, wv)) / 2e-5
        got = bf16_values(host(dx))
        # each dx is off by half a BF16 step at most
        assert abs((got * d).sum() - num) <= 2.0 ** -8 * np.abs(got * d).sum() + 1e-5 * np.abs(got * d).sum()
        num = (loss(hv, wv + 1e-5 * e[0]) - loss(hv, wv - 1e-5 * e[0])) / 2e-5
        assert abs((host(dw) * e[0]).sum() - num) <= 1e-5 * np.abs(host(dw) * e[0]).sum() + 1e-6


def test_rmsnorm_of_nothing():
    e = torch.empty((0, 128), dtype=torch.bfloat16, device=DEV)
    w, s = torch.ones((128,), device=DEV), torch.empty((0,), device=DEV)
    q, sf, y, h, r = nv.fp8_rmsnorm(e, w, residual=e, need_y=True, need_rstd=True)
    assert q.shape == (0, 128) and sf.shape == (0, 1) and y.shape == h.shape == (0, 128) and r.shape == (0,)
    dw = torch.full((128,), 7.0, device=DEV)
    dx, dw = nv.rmsnorm_bwd(e, e, w, s, out=(None, dw))
    assert dx.shape == (0, 128) and torch.all(dw == 0)


def test_rmsnorm_graph_and_streams():
    rng = np.random.default_rng(9)
    T, H = 40, 1040
    w = _weight(rng, H, False).to(DEV)
    xs = [_bf(rng, T, H).to(DEV) for _ in range(3)]
    x, r = xs[0].clone(), xs[1].clone()
    ws = torch.empty(nv.lib().nvfp4_rmsnorm_bwd_workspace_size(T, H), dtype=torch.uint8, device=DEV)
    mk = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device=DEV)
    out = (mk(T, H, t=torch.float8_e4m3fn), mk(T, 9, t=torch.float32), mk(T, H), mk(T, H), mk(T, t=torch.float32))
    grads = (mk(T, H), mk(H, t=torch.float32))

    def both():
        nv.fp8_rmsnorm(x, w, residual=r, out=out)
        nv.rmsnorm_bwd(out[2], out[3], w, out[4], dh=r, out=grads, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        both()
        with torch.cuda.graph(g, stream=side):
            both()
    torch.cuda.synchronize()
    for i in range(4):
        x.copy_(xs[i % 3])
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out + grads]
        both()
        torch.cuda.synchronize()
        for a, b in zip(got, out + grads):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i


def test_more_rows_than_a_row_of_workgroups():
    """2^25 + 3 rows of eight columns: over 2^20 workgroups of sixteen rows."""
    T = (1 << 25) + 3
    x = torch.arange(T * 8, dtype=torch.int32, device=DEV).bitwise_and_(0x3F7F).to(torch.int16).view(torch.bfloat16).view(T, 8)
    w = torch.full((8,), 2.0, device=DEV)
    y, _, s = nv.rmsnorm(x, w, eps=1.0, need_rstd=True)
    at = torch.cat([torch.arange(1000, device=DEV), torch.arange(T - 1000, T, device=DEV), torch.randint(0, T, (5000,), device=DEV)])
    v, r = N.rmsnorm(host(x[at].float()), np.full(8, 2.0), 1.0)
    assert np.all(np.abs(host(s[at]) - r) <= 40 * U * r)
    assert np.all(np.abs(bf16_values(host(y[at])) - v) <= (2.0 ** -8 + 41 * U) * np.abs(v) + 1e-38)
