"""The expert layer for a few tokens at its largest sizes: H or I next to 2^19, an
expert next to 2^31 weights.

The reference is the formula in float64 on the device, from the codes; its bound
counts roundings as `oracle.few.forward` does: 2^-23 of what has gone in at each
addition, h with 16 (FP8) or 12 bits (NVFP4: and 2^-38 of the largest of its 128),
half a BF16 step of out."""

import pytest
import torch

import nvfp4_block_scaled_04_amd as nv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E2M1 = [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]


def _up(a, b):
    return -(-a // b)


def _fp8(E, N, K, g):
    q = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device=DEV)
    for e in range(E):
        for n in range(0, N, step := max(1, (1 << 27) // K)):
            part = q[e, n:n + step]
            part.copy_(torch.randn(part.shape, generator=g, device=DEV, dtype=torch.bfloat16).mul_(100).clamp_(-448, 448).to(q.dtype))
    s = 2.0 ** -12 * (1 + torch.rand((E, _up(N, 128), _up(K, 128)), generator=g, device=DEV))

    def rows(e, a, b):
        col = torch.arange(K, device=DEV) // 128
        return q[e, a:b].double() * s[e][torch.arange(a, b, device=DEV) // 128][:, col].double()
    return (q, s), rows


def _nvfp4(E, N, K, g):
    tiles, S = _up(N, 512), K // 128
    q = torch.randint(0, 256, (E, tiles, S, 512, 64), generator=g, device=DEV, dtype=torch.uint8)
    sf = torch.randint(104, 121, (E, tiles, S, 512, 8), generator=g, device=DEV, dtype=torch.uint8)
    gs = torch.tensor([2e4, 3e4], device=DEV)[:E]

    def rows(e, a, b):
        n = torch.arange(a, b, device=DEV)
        c = q[e, n // 512, :, n % 512].long()              # rows, stages, bytes
        v = torch.tensor(E2M1, dtype=torch.float64, device=DEV)[torch.stack((c & 15, c >> 4), -1)].view(b - a, S, 8, 16)
        return (v * sf[e, n // 512, :, n % 512].view(torch.float8_e4m3fn).double()[..., None]).view(b - a, K) / gs[e].double()
    return (q.flatten(), sf.flatten(), gs), rows


def _product(rows, e, N, K, x):
    """W x and |W| |x| of the columns x (K, T)."""
    out, mag = [], []
    for a in range(0, N, step := max(1, (1 << 25) // K)):
        w = rows(e, a, min(N, a + step))
        out.append(w @ x)
        mag.append(w.abs() @ x.abs())
    return torch.cat(out), torch.cat(mag)


@pytest.mark.parametrize("fmt,H,I", [("fp8", 16, (1 << 19) - 16), ("fp8", (1 << 19) - 16, 16), ("fp8", 32752, 32752),
                                     ("nvfp4", 128, (1 << 19) - 128), ("nvfp4", (1 << 19) - 128, 128), ("nvfp4", 32640, 32640)])
def test_few_largest(fmt, H, I):
    print(f"[case] {fmt} H={H} I={I}", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(H + I)
    E, T = 2, 3
    make = _fp8 if fmt == "fp8" else _nvfp4
    w1, rows1 = make(E, 2 * I, H, g)
    w2, rows2 = make(E, H, I, g)
    x = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    ids = torch.tensor([[0, 1], [1, -1], [1, 0]], dtype=torch.int32, device=DEV)
    tw = torch.tensor([[0.5, 0.25], [1.0, 9.0], [0.75, 0.125]], device=DEV)
    if fmt == "fp8":
        out = nv.moe_expert_forward_few_fp8(x, ids, tw, *w1, *w2)
    else:
        (q1, s1, g1), (q2, s2, g2) = w1, w2
        out = nv.moe_expert_forward_few(x, ids, tw, nv.ExpertWeights(nv.PackedWeight(q1, s1, E, 2 * I, H), g1,
                                                                      nv.PackedWeight(q2, s2, E, H, I), g2))
    u = 2.0 ** -23
    ref, err = (torch.zeros((H, T), dtype=torch.float64, device=DEV) for _ in range(2))
    xt = x.double().t().contiguous()
    for e in range(E):
        y, m = _product(rows1, e, 2 * I, H, xt)
        if fmt == "nvfp4":                                 # gate and up interleaved at 8
            y, m = (a.view(-1, 2, 8, T).transpose(0, 1).reshape(2 * I, T) for a in (y, m))
        c1, c2 = (152 + H / 1024) * u, (280 + 2 * (I / 1024 + 1)) * u
        ga, up, eg, eu = y[:I], y[I:], c1 * m[:I], c1 * m[I:]
        si = ga * torch.sigmoid(ga)
        h = si * up
        eh = 1.1 * eg * (up.abs() + eu) + si.abs() * eu + ((2.0 ** -16 if fmt == "fp8" else 2.0 ** -12) + 16 * u) * h.abs()
        if fmt == "nvfp4":
            eh = eh + 2.0 ** -38 * (h.abs() + eh).view(-1, 128, T).amax(1, keepdim=True).expand(-1, 128, T).reshape(I, T)
        coef = torch.where(ids == e, tw, 0).sum(1).double()
        y, _ = _product(rows2, e, H, I, h)
        _, d = _product(rows2, e, H, I, eh + c2 * h.abs())
        ref += coef * y
        err += coef * d
    err = err + 2.0 ** -8 * (ref.abs() + err) + 1e-37
    worst = float(((out.double().t() - ref).abs() / err).max())
    print(f"[worst share of the bound] {worst:.3f}", flush=True)
    assert worst <= 1.0
