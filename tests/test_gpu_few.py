"""GPU parity of the expert layer for a few tokens, FP8 and NVFP4 weights.

The bound of every output comes from `oracle.few.forward`: roundings counted
against the summed magnitudes, and half a BF16 step."""

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_04_amd as nv
from oracle import few as W
from oracle import formats as F
from oracle import fp8 as P8
from parity import bf16_values, host

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _bf(rng, *shape, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(torch.bfloat16)


def _fp8_weights(rng, E, H, I):
    """(arguments of the call, w1(e), w2(e) in float64)."""
    q, vals = [], []
    for N, K in ((2 * I, H), (H, I)):
        c, s = nv.fp8_quantize_weight(_bf(rng, E, N, K, scale=0.02).to(DEV))
        q += [c, s]
        hc, hs = host(c.view(torch.uint8)), host(s)
        vals.append(lambda e, hc=hc, hs=hs: P8.decode(hc[e], hs[e], 128))
    return tuple(q), vals[0], vals[1]


def _nvfp4_weights(rng, E, H, I):
    w = nv.prepare_expert_weights([_bf(rng, E, H, 2 * I, scale=0.02).to(DEV)], [_bf(rng, E, I, H, scale=0.02).to(DEV)], DEV)
    rm = {k: host(v) for k, v in w.rowmajor.items()}
    g = {"w1": host(w.gs_w1), "w2": host(w.gs_w2)}

    def value(name, e):
        q, sf = rm[name + "_q"][e], rm[name + "_sf"][e]
        codes = np.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)
        return F.e2m1_decode(codes).astype(np.float64) * np.repeat(F.e4m3_decode(sf), 16, 1) / np.float64(g[name][e])

    n = np.arange(2 * I)
    order = np.where(n % 16 < 8, 8 * (n // 16) + n % 8, I + 8 * (n // 16) + n % 8)   # row n holds this of [gate | up]

    def w1(e):
        out = np.empty((2 * I, H))
        out[order] = value("w1", e)
        return out
    return (w,), w1, lambda e: value("w2", e)


MAKE = {"fp8": (_fp8_weights, nv.moe_expert_forward_few_fp8), "nvfp4": (_nvfp4_weights, nv.moe_expert_forward_few)}


def _routing(rng, T, E, k, bad=0.0, few=None):
    ids = rng.integers(0, few or E, (T, k)).astype(np.int32)       # the same id may come twice in a row
    ids[rng.random((T, k)) < bad] = -1
    return ids, rng.random((T, k)).astype(np.float32)


def _check(out, x, ids, w, w1, w2):
    # h: 11 bits at least (half a step is 2^-12 of it)
    ref, err = W.forward(x.float().numpy(), ids, w, w1, w2, h_bits=12)
    got = bf16_values(host(out))
    worst = np.max(np.abs(got - ref) / err)
    print(f"[worst share of the bound] {worst:.3f}", flush=True)
    assert worst <= 1.0


CASES = [("fp8", 1, 16, 16, 1, 1, 0.0, None), ("fp8", 1, 128, 128, 4, 2, 0.0, None), ("fp8", 3, 144, 48, 5, 3, 0.3, None),
         ("fp8", 16, 1040, 528, 40, 3, 0.1, None), ("fp8", 16, 256, 128, 9, 2, 0.0, 2), ("fp8", 13, 2048, 768, 20, 8, 0.0, None),
         ("fp8", 4, 1152, 16, 3, 2, 0.0, None), ("fp8", 16, 64, 32, 300, 64, 0.2, None), ("fp8", 2, 16, 1040, 4, 4, 0.0, None),
         ("fp8", 1, 7168, 2048, 6, 8, 0.0, None), ("fp8", 7, 32, 32, 4096, 5, 0.0, None),
         ("fp8", 3, 4096, 64, 3, 2, 0.0, None), ("fp8", 16, 8256, 48, 5, 2, 0.0, None), ("fp8", 2, 20496, 32, 2, 2, 0.0, None),
         ("fp8", 12, 3088, 80, 2, 2, 0.0, None), ("nvfp4", 3, 4096, 128, 3, 2, 0.0, None), ("nvfp4", 16, 8448, 128, 4, 3, 0.0, None),
         ("nvfp4", 2, 20480, 128, 2, 2, 0.0, None), ("nvfp4", 12, 2816, 256, 2, 2, 0.0, None), ("nvfp4", 4, 256, 640, 40, 16, 0.1, None),
         ("nvfp4", 1, 128, 128, 1, 1, 0.0, None), ("nvfp4", 16, 256, 128, 4, 2, 0.0, None), ("nvfp4", 7, 384, 256, 9, 3, 0.2, None),
         ("nvfp4", 2, 640, 1152, 3, 2, 0.0, None), ("nvfp4", 16, 512, 384, 30, 8, 0.0, 3), ("nvfp4", 1, 7168, 2048, 6, 8, 0.0, None),
         ("nvfp4", 5, 1152, 640, 12, 64, 0.5, None), ("nvfp4", 3, 1024, 896, 17, 4, 0.0, None)]


@pytest.mark.parametrize("fmt,T,H,I,E,k,bad,few", CASES)
def test_few(fmt, T, H, I, E, k, bad, few):
    print(f"[case] {fmt} T={T} H={H} I={I} E={E} k={k} bad={bad} few={few}", flush=True)
    rng = np.random.default_rng(T * 31 + H + I)
    make, call = MAKE[fmt]
    args, w1, w2 = make(rng, E, H, I)
    x = _bf(rng, T, H)
    ids, w = _routing(rng, T, E, k, bad, few)
    out = call(x.to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), *args)
    _check(out, x, ids, w, w1, w2)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_few_without_experts(fmt):
    """Tokens whose ids are all outside [0, E): zeros, and nothing else moves."""
    rng = np.random.default_rng(1)
    make, call = MAKE[fmt]
    args, w1, w2 = make(rng, 4, 256, 128)
    x = _bf(rng, 3, 256)
    for ids in ([[-1, 4], [9, -7], [4, 4]], [[1, 2], [-1, 4], [3, -1]]):
        ids = np.array(ids, np.int32)
        w = rng.random((3, 2)).astype(np.float32)
        out = torch.full((3, 256), 5.0, dtype=torch.bfloat16, device=DEV)
        call(x.to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), *args, out=out)
        _check(out, x, np.where((ids < 0) | (ids > 3), -1, ids), w, w1, w2)
        none = ((ids < 0) | (ids > 3)).all(1)
        assert none.any() and torch.all(out[torch.from_numpy(none).to(DEV)] == 0)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_few_bad_rows_and_experts_stay_their_own(fmt):
    """A token of NaN, and an expert whose scales are no numbers, spoil only the
    tokens that hold or chose them."""
    rng = np.random.default_rng(6)
    make, call = MAKE[fmt]
    T, H, I, E, k = 9, 272 if fmt == "fp8" else 256, 144 if fmt == "fp8" else 128, 6, 2
    args, w1, w2 = make(rng, E, H, I)
    ids = rng.integers(0, E - 1, (T, k)).astype(np.int32)
    ids[4, 1] = E - 1                                     # the bad expert's only token
    w = rng.random((T, k)).astype(np.float32)
    x = _bf(rng, T, H)
    x[7, 3] = float("nan")
    if fmt == "fp8":
        args[1][E - 1, 0, 0] = float("inf")
        args[3][E - 1, 0, 0] = float("inf")
    else:
        args[0].gs_w1[E - 1] = float("nan")
        n = args[0].w2.sf.numel() // E
        args[0].w2.sf[(E - 1) * n:] = 0x7F
    out = call(x.to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), *args)
    keep = [t for t in range(T) if t not in (4, 7)]
    _check(out[keep], x[keep], ids[keep], w[keep], w1, w2)
    assert torch.isnan(out[7].float()).all() and not torch.isfinite(out[4].float()).all()


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_few_magnitudes(fmt):
    """Tokens of sizes far apart in one call: each as exact as alone."""
    rng = np.random.default_rng(14)
    make, call = MAKE[fmt]
    args, w1, w2 = make(rng, 5, 640, 256)
    scale = torch.tensor([1e-15, 1e-9, 1e-4, 1.0, 0.0, 1e4, 1e9, 1e15, 3.0])[:, None]
    x = (_bf(rng, 9, 640).float() * scale).to(torch.bfloat16)
    x[8, ::3] *= 2.0 ** -12                               # and far apart in one token
    ids, w = _routing(rng, 9, 5, 3)
    out = call(x.to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), *args)
    _check(out, x, ids, w, w1, w2)
    assert torch.all(out[4] == 0)


def test_few_infinite_tokens_are_nan():
    rng = np.random.default_rng(15)
    args, w1, w2 = _nvfp4_weights(rng, 4, 256, 128)
    x = _bf(rng, 6, 256)
    x[1, 5], x[4, 250] = float("inf"), float("-inf")
    ids, w = _routing(rng, 6, 4, 2)
    out = nv.moe_expert_forward_few(x.to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), *args)
    keep = [0, 2, 3, 5]
    _check(out[keep], x[keep], ids[keep], w[keep], w1, w2)
    assert torch.isnan(out[[1, 4]].float()).all()


@pytest.mark.parametrize("E,k", [(4096, 8), (3000, 4), (5, 33)])
def test_few_lists_of_many_pairs(E, k):
    """More than 64 pairs: the other way of making the list of experts."""
    rng = np.random.default_rng(E + k)
    args, w1, w2 = _fp8_weights(rng, E, 32, 16)
    x = _bf(rng, 16, 32)
    ids, w = _routing(rng, 16, E, k, 0.1)
    ids[3, 0], ids[3, 1], ids[5, 2] = 0, E - 1, E         # the ends, and one past them
    out = nv.moe_expert_forward_few_fp8(x.to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), *args)
    _check(out, x, np.where(ids >= E, -1, ids), w, w1, w2)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_few_two_graphs_one_workspace(fmt):
    """Two layers captured apart on one workspace, replayed in turn on one stream
    with eager calls between."""
    rng = np.random.default_rng(16)
    make, call = MAKE[fmt]
    layers = [make(rng, 6, 384, 128) for _ in range(2)]
    x = [_bf(rng, T, 384) for T in (4, 11)]
    routes = [_routing(rng, T, 6, 3, 0.1) for T in (4, 11)]
    dev = [(a.to(DEV), torch.from_numpy(i).to(DEV), torch.from_numpy(v).to(DEV)) for a, (i, v) in zip(x, routes)]
    ws = nv.few_workspace(16, 128, 3, DEV)
    outs = [torch.empty(a.shape, dtype=torch.bfloat16, device=DEV) for a in x]
    graphs = []
    for j in range(2):
        call(*dev[j], *layers[j][0], out=outs[j], workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(*dev[j], *layers[j][0], out=outs[j], workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.zero_()
        graphs[0].replay()
        graphs[1].replay()
        call(*dev[0], *layers[1][0], workspace=ws)
        torch.cuda.synchronize()
        for j in range(2):
            _check(outs[j], x[j], *routes[j], layers[j][1], layers[j][2])


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_few_repeats_and_slots(fmt):
    """Equal inputs give equal bits; an id twice in a row counts with both weights;
    a slot of weight 0 changes nothing but the sign of zeros."""
    rng = np.random.default_rng(12)
    make, call = MAKE[fmt]
    args, w1, w2 = make(rng, 7, 512, 256)
    x = _bf(rng, 5, 512).to(DEV)
    ids, w = _routing(rng, 5, 7, 3)
    ids[2] = 3
    i, v = torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV)
    out = call(x, i, v, *args)
    _check(out, x.cpu(), ids, w, w1, w2)
    assert torch.equal(call(x, i, v, *args).view(torch.int16), out.view(torch.int16))
    more = torch.cat([i, torch.full((5, 1), 6, dtype=torch.int32, device=DEV)], 1)
    again = call(x, more, torch.cat([v, torch.zeros((5, 1), device=DEV)], 1), *args)
    _check(again, x.cpu(), ids, w, w1, w2)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_few_graph_streams_and_buffers(fmt):
    """Replays on changed inputs and a filled workspace; two streams at once, each
    with its own; nothing outside out is written."""
    rng = np.random.default_rng(13)
    make, call = MAKE[fmt]
    T, H, I, E, k = 6, 640, 256, 9, 4
    args, w1, w2 = make(rng, E, H, I)
    xs = [_bf(rng, T, H).to(DEV) for _ in range(3)]
    routes = [_routing(rng, T, E, k, 0.2) for _ in range(3)]
    x, ids, w = xs[0].clone(), torch.from_numpy(routes[0][0]).to(DEV), torch.from_numpy(routes[0][1]).to(DEV)
    buf = torch.full((T * H + 256,), 7.0, dtype=torch.bfloat16, device=DEV)
    out, ws = buf[128:-128].view(T, H), nv.few_workspace(T, I, k, DEV)
    guard = torch.full((ws.numel() + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    ws = guard[256:-256]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call(x, ids, w, *args, out=out, workspace=ws)
        with torch.cuda.graph(g, stream=side):
            call(x, ids, w, *args, out=out, workspace=ws)
    torch.cuda.synchronize()
    eager = []
    for i in range(5):
        x.copy_(xs[i % 3])
        ids.copy_(torch.from_numpy(routes[i % 3][0]))
        w.copy_(torch.from_numpy(routes[i % 3][1]))
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        _check(got, xs[i % 3].cpu(), *routes[i % 3], w1, w2)
        eager.append(call(x, ids, w, *args))
        torch.cuda.synchronize()
        assert torch.equal(eager[-1].view(torch.int16), got.view(torch.int16))
        assert torch.all(buf[:128] == 7) and torch.all(buf[-128:] == 7)
        assert torch.all(guard[:256] == 0xA5) and torch.all(guard[-256:] == 0xA5)
    streams = [torch.cuda.Stream() for _ in range(3)]
    ins = [(xs[j], torch.from_numpy(routes[j][0]).to(DEV), torch.from_numpy(routes[j][1]).to(DEV)) for j in range(3)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for j, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs.append((j, call(*ins[j], *args)))
    torch.cuda.synchronize()
    for j, o in outs:
        assert torch.equal(o.view(torch.int16), eager[j].view(torch.int16))


def test_few_refuses():
    rng = np.random.default_rng(0)
    args, _, _ = _fp8_weights(rng, 2, 64, 32)
    x = _bf(rng, 17, 64).to(DEV)
    ids, w = torch.zeros((17, 2), dtype=torch.int32, device=DEV), torch.ones((17, 2), device=DEV)
    f = nv.moe_expert_forward_few_fp8
    with pytest.raises(nv.Nvfp4Error):
        f(x, ids, w, *args)                               # 17 tokens
    x, ids, w = x[:2], ids[:2], w[:2]
    assert f(x[:0], ids[:0], w[:0], *args).shape == (0, 64)
    for bad in ((x.float(), ids, w), (x, ids.long(), w), (x, ids, w.half()), (x, ids, w[:1]), (x[:, :32], ids, w),
                (x.cpu(), ids, w), (x, ids[0], w)):
        with pytest.raises((ValueError, TypeError)):
            f(*bad, *args)
    with pytest.raises(ValueError):
        f(x, ids, w, args[0], args[1], args[2][:1], args[3])
    with pytest.raises(ValueError):
        f(x, ids, w, args[0], args[1][:, :0], args[2], args[3])
    with pytest.raises(nv.Nvfp4Error):
        f(x, ids, w, *args, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    ew, _, _ = _nvfp4_weights(rng, 2, 128, 128)
    x = _bf(rng, 2, 128).to(DEV)
    for name in ("q", "sf"):
        p = nv.PackedWeight(ew[0].w1.q, ew[0].w1.sf, 2, 256, 128)
        setattr(p, name, getattr(p, name)[:-64])
        with pytest.raises(ValueError):
            nv.moe_expert_forward_few(x, ids, w, nv.ExpertWeights(p, ew[0].gs_w1, ew[0].w2, ew[0].gs_w2))
    with pytest.raises(ValueError):
        nv.moe_expert_forward_few(x, ids, w, nv.mx_expert_weights(ew[0]))


def test_a_decode_block():
    """A serving step as a user strings it together: norm with FP8 rows, router,
    experts, and the next norm with the experts' output added to the residual."""
    rng = np.random.default_rng(21)
    T, H, I, E, k = 5, 512, 256, 12, 3
    args, w1, w2 = _fp8_weights(rng, E, H, I)
    attn, res, g1, g2 = _bf(rng, T, H), _bf(rng, T, H), _bf(rng, H), _bf(rng, H)
    router = _bf(rng, E, H, scale=0.1)
    q, sf, y, h, _ = nv.fp8_rmsnorm(attn.to(DEV), g1.to(DEV), residual=res.to(DEV), need_y=True)
    ids, w = nv.router_topk(y.float() @ router.to(DEV).float().t(), k)
    out = nv.moe_expert_forward_few_fp8(y, ids, w, *args)
    y2, h2, _ = nv.rmsnorm(out, g2.to(DEV), residual=h)
    _check(out, y.cpu(), host(ids), host(w), w1, w2)
    from oracle import norm as N
    assert torch.equal(h2.view(torch.int16), (out.float() + h.float()).to(torch.bfloat16).view(torch.int16))
    v, _ = N.rmsnorm(host(h2.float()), g2.float().numpy(), 1e-6)
    assert np.all(np.abs(bf16_values(host(y2)) - v) <= (2.0 ** -8 + 41 * 2.0 ** -24) * np.abs(v) + 1e-38)
    # the same experts by the quantised chain: FP8 activations are off by up to 2^-4 a value
    off, perm, inv, _ = nv.moe_route(ids, E)
    y1 = nv.fp8_grouped_gemm(q, sf, args[0], args[1], offsets=off, a_row_src=perm, a_row_div=k)
    hq, hs = nv.fp8_swiglu_quantize(y1, offsets=off)
    chain = nv.moe_combine(nv.fp8_grouped_gemm(hq, hs, args[2], args[3], offsets=off), inv, w, off)
    a, b = host(chain.float()).astype(np.float64), host(out.float()).astype(np.float64)
    assert np.linalg.norm(a - b) <= 3 * 2.0 ** -4 * np.linalg.norm(b)
