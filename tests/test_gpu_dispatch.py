"""GPU parity of dispatch, its gradient, combine's gradient and the router's
gradient, and a training pass around the experts.

Tolerances: dispatch and dy are bit-exact (a copy; one fp32 product and one
rounding to BF16).  dx: half a BF16 step (2^-8 relative) and k fp32 additions
(2^-24 of the terms' magnitudes each).  dw: H + 16 fp32 additions and fused
products.  dlogits: k + 4 fp32 operations, each 2^-24 of the magnitudes."""

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_04_amd as nv
from oracle import formats as F
from oracle import fp8 as P
from parity import host, bf16_values

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _bf(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _routing(rng, T, k, E, bad):
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[rng.random((T, k)) < bad] = -1
    off, perm, inv, _ = nv.moe_route(torch.from_numpy(ids).to(DEV), E)
    return ids, off, perm, inv


CASES = [(1, 1, 1, 8, 0.0), (1, 8, 4, 16, 0.0), (5, 2, 3, 64, 0.3), (33, 3, 9, 512, 0.1), (64, 8, 16, 520, 0.0),
         (17, 9, 5, 1000, 0.2), (40, 16, 64, 1024, 0.0), (7, 64, 300, 2048, 0.1), (30, 6, 8, 2056, 0.5),
         (9, 8, 256, 4104, 0.0), (12, 8, 256, 7168, 0.05), (6, 5, 4, 14344, 0.1), (20, 2, 4, 256, 1.0)]


@pytest.mark.parametrize("T,k,E,H,bad", CASES)
def test_dispatch_and_gradients(T, k, E, H, bad):
    print(f"[case] dispatch T={T} k={k} E={E} H={H} bad={bad}", flush=True)
    rng = np.random.default_rng(T * 131 + H)
    _, off, _, inv = _routing(rng, T, k, E, bad)
    n, hinv = int(off[-1]), host(inv)
    x, y, dout, drows = _bf(rng, T, H), _bf(rng, T * k, H), _bf(rng, T, H), _bf(rng, T * k, H)
    drows[n:] = float("nan")                             # rows of invalid pairs are not read
    y[n:] = float("inf")
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32))

    rows = nv.moe_dispatch(x.to(DEV), inv, off, k)
    assert np.array_equal(_bits(rows), P.dispatch(_bits(x), hinv, n, k))

    dx = nv.moe_dispatch_bwd(drows.to(DEV), inv, off, k)
    ref, mag = P.dispatch_bwd(drows.double().numpy(), hinv, n, k)
    assert np.all(np.abs(bf16_values(host(dx)) - ref) <= 2.0 ** -8 * np.abs(ref) + k * 2.0 ** -24 * mag)

    dy, dw = nv.moe_combine_bwd(dout.to(DEV), y.to(DEV), inv, w.to(DEV), off)
    rdy, rdw, rmag = P.combine_bwd(dout.float().numpy(), y.float().numpy(), hinv, w.numpy(), n)
    assert np.array_equal(bf16_values(host(dy)), F.bf16_bits_to_f32(F.round_to_bf16(rdy)).astype(np.float64))
    assert np.all(np.abs(host(dw) - rdw) <= (H + 16) * 2.0 ** -24 * rmag)

    only, none = nv.moe_combine_bwd(dout.to(DEV), None, inv, w.to(DEV), off, need_dw=False)
    assert none is None and torch.equal(only.view(torch.int16), dy.view(torch.int16))


@pytest.mark.parametrize("k,H", [(3, 64), (9, 1000), (4, 2056)])
def test_combine_gradient_of_non_finite_rows(k, H):
    """dout of infinities and NaN: dy and dw of pairs with an invalid expert id
    stay zero, and other tokens' stay finite."""
    T, E = 20, 5
    rng = np.random.default_rng(H)
    ids, off, _, inv = _routing(rng, T, k, E, 0.3)
    dout, y = _bf(rng, T, H), _bf(rng, T * k, H)
    dout[::3, 1], dout[1::3, H - 1] = float("inf"), float("nan")
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32) + 0.5)
    dy, dw = nv.moe_combine_bwd(dout.to(DEV), y.to(DEV), inv, w.to(DEV), off)
    bad = host(inv).reshape(T, k) >= int(off[-1])
    assert np.array_equal(bad, ids < 0) and bad.any()
    got, dy = host(dw), bf16_values(host(dy))
    assert np.all(got[bad] == 0) and np.all(dy[int(off[-1]):] == 0)
    finite = np.isfinite(dout.float().numpy()).all(1)
    assert np.isfinite(got[finite]).all() and not np.isfinite(got[~finite][~bad[~finite]]).any()


def test_more_tokens_than_a_row_of_workgroups():
    """2^26 + 5 tokens of eight columns: more threads than 2^32."""
    T = (1 << 26) + 5
    perm = torch.randperm(T, device=DEV)
    inv = torch.empty(T, dtype=torch.int32, device=DEV)
    inv[perm] = torch.arange(T, dtype=torch.int32, device=DEV)
    off = torch.tensor([0, T - 3], dtype=torch.int32, device=DEV)
    x = torch.arange(T * 8, dtype=torch.int32, device=DEV).bitwise_and_(0x3F7F).to(torch.int16).view(torch.bfloat16).view(T, 8)
    rows = nv.moe_dispatch(x, inv, off, 1)
    want = torch.cat([x[p] for p in perm.split(1 << 24)])   # indexed at once it comes out wrong at this size
    want[T - 3:] = 0
    assert torch.equal(rows.view(torch.int16), want.view(torch.int16))
    back = nv.moe_dispatch_bwd(rows, inv, off, 1)
    kept = torch.where((inv < T - 3)[:, None], x, torch.zeros_like(x))
    assert torch.equal(back.view(torch.int16), kept.view(torch.int16))
    del want, kept, back
    w = torch.full((T, 1), 0.5, device=DEV)
    dy, _ = nv.moe_combine_bwd(x, None, inv, w, off, need_dw=False)
    assert torch.equal(dy, rows * 0.5)
    ids, dw = torch.zeros((T, 1), dtype=torch.int32, device=DEV), torch.ones((T, 1), device=DEV)
    dl = nv.router_topk_bwd(ids, w, dw, 1)
    assert torch.all(dl == 0.25)                         # 0.5 * (1 - 0.5 * 1)


def test_outputs_stay_inside_their_buffers():
    rng = np.random.default_rng(3)
    for T, k, H in [(5, 3, 24), (3, 2, 1000), (2, 8, 7168)]:
        _, off, _, inv = _routing(rng, T, k, 4, 0.2)
        x, y, w = _bf(rng, T, H).to(DEV), _bf(rng, T * k, H).to(DEV), torch.rand((T, k), device=DEV)
        buf = torch.full((T * k * H + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
        mid = buf[32:32 + T * k * H].view(T * k, H)
        nv.moe_dispatch(x, inv, off, k, out=mid)
        assert torch.all(buf[:32] == 7) and torch.all(buf[-32:] == 7)
        wb = torch.full((T * k + 16,), 7.0, device=DEV)
        nv.moe_combine_bwd(x, y, inv, w, off, out=(mid, wb[8:8 + T * k].view(T, k)))
        assert torch.all(buf[:32] == 7) and torch.all(buf[-32:] == 7)
        assert torch.all(wb[:8] == 7) and torch.all(wb[-8:] == 7)
        nv.moe_dispatch_bwd(y, inv, off, k, out=buf[32:32 + T * H].view(T, H))
        assert torch.all(buf[:32] == 7) and torch.all(buf[-32:] == 7)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 4, 2), (33, 70, 3), (100, 256, 8), (9, 1024, 64), (5, 1023, 7), (64, 65, 9)])
def test_router_gradient(T, E, k):
    print(f"[case] router gradient T={T} E={E} k={k}", flush=True)
    rng = np.random.default_rng(T + E)
    ids, w = nv.router_topk(torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV), k)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    out = torch.full((T, E), 9.0, device=DEV)
    nv.router_topk_bwd(ids, w, torch.from_numpy(dw).to(DEV), E, out=out)
    ref, mag = P.router_bwd(host(ids), host(w), dw, E)
    assert np.all(np.abs(host(out) - ref) <= (k + 4) * 2.0 ** -24 * mag)
    assert np.all(host(out)[mag == 0] == 0)


def test_router_gradient_repeated_and_invalid_ids():
    ids = np.array([[3, 3, 1], [-1, 2, 9], [0, 0, 0]], np.int32)
    w = np.array([[.5, .25, .25], [.2, .3, .5], [.1, .2, .7]], np.float32)
    dw = np.array([[1, -2, 3], [4, 5, 6], [1, 1, 2]], np.float32)
    t = lambda v: torch.from_numpy(v).to(DEV)
    for E in (5, 8):
        got = host(nv.router_topk_bwd(t(ids), t(w), t(dw), E))
        ref, mag = P.router_bwd(ids, w, dw, E)
        assert np.all(np.abs(got - ref) <= 7 * 2.0 ** -24 * mag)


def test_router_gradient_unaligned_output():
    rng = np.random.default_rng(6)
    ids, w = nv.router_topk(torch.from_numpy(rng.standard_normal((9, 64)).astype(np.float32)).to(DEV), 4)
    dw = torch.from_numpy(rng.standard_normal((9, 4)).astype(np.float32)).to(DEV)
    ref = nv.router_topk_bwd(ids, w, dw, 64)
    buf = torch.full((9 * 64 + 8,), 5.0, device=DEV)
    nv.router_topk_bwd(ids, w, dw, 64, out=buf[1:1 + 9 * 64].view(9, 64))
    assert torch.equal(buf[1:1 + 9 * 64].view(9, 64), ref) and buf[0] == 5 and torch.all(buf[1 + 9 * 64:] == 5)


def test_empty_calls_and_refusals():
    i32 = torch.zeros(5, dtype=torch.int32, device=DEV)
    none = torch.zeros((0, 16), dtype=torch.bfloat16, device=DEV)
    assert nv.moe_dispatch(none, i32[:0], i32, 2).shape == (0, 16)
    assert nv.moe_dispatch_bwd(none, i32[:0], i32, 2).shape == (0, 16)
    dy, dw = nv.moe_combine_bwd(none, none, i32[:0], torch.zeros((0, 2), device=DEV), i32)
    assert dy.shape == (0, 16) and dw.shape == (0, 2)
    z = torch.zeros((0, 2), device=DEV)
    assert nv.router_topk_bwd(z.to(torch.int32), z, z, 8).shape == (0, 8)
    x = torch.zeros((2, 16), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        nv.moe_dispatch(x, i32[:3], i32, 2)
    with pytest.raises(nv.Nvfp4Error):
        nv.moe_dispatch(torch.zeros((2, 12), dtype=torch.bfloat16, device=DEV), i32[:4], i32, 2)
    with pytest.raises(ValueError):
        nv.moe_dispatch(x.t(), i32[:4], i32, 2)
    with pytest.raises(ValueError):
        nv.moe_dispatch_bwd(x, i32[:4], i32, 3)
    with pytest.raises(nv.Nvfp4Error):
        nv.moe_combine_bwd(x, torch.zeros((4, 16), dtype=torch.bfloat16, device=DEV), i32[:4],
                           torch.zeros((2, 2), device=DEV), i32[:1])                       # no expert
    y = torch.zeros((4, 16), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(nv.Nvfp4Error):
        nv.moe_combine_bwd(x, y, i32[:4], torch.zeros((2, 2), device=DEV), i32,
                           out=(y, torch.zeros((2, 2), device=DEV)))                       # dy over y


def test_a_training_pass_around_fp8_experts():
    """Router, route, dispatch, FP8 products with SwiGLU, combine, and the
    gradients back to the logits and the tokens.  Forward: equal bits whether
    the products gather compact quantised tokens or take the dispatched rows.
    Backward: every gradient kernel chained, against the same chain in float64
    on the device's own intermediates (each link's own bound)."""
    rng = np.random.default_rng(31)
    T, H, I, E, k = 48, 256, 128, 6, 3
    x = _bf(rng, T, H)
    xd = x.to(DEV)
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV)
    w1 = (_bf(rng, E, 2 * I, H) * 0.1).to(DEV)
    w2 = (_bf(rng, E, H, I) * 0.1).to(DEV)
    b1, s1 = nv.fp8_quantize_weight(w1)
    b2, s2 = nv.fp8_quantize_weight(w2)
    ids, w = nv.router_topk(logits, k)
    off, perm, inv, _ = nv.moe_route(ids, E)

    def experts(a, asf, **kw):
        y1 = nv.fp8_grouped_gemm(a, asf, b1, s1, offsets=off, **kw)
        h, hs = nv.fp8_swiglu_quantize(y1, offsets=off)
        return h, hs, nv.fp8_grouped_gemm(h, hs, b2, s2, offsets=off)

    q, sf = nv.fp8_quantize(xd)
    _, _, y_gather = experts(q, sf, M=T * k, a_row_src=perm, a_row_div=k)
    rows = nv.moe_dispatch(xd, inv, off, k)
    h, hs, y = experts(*nv.fp8_quantize(rows))
    assert torch.equal(y.view(torch.int16), y_gather.view(torch.int16))
    out = nv.moe_combine(y, inv, w, off)

    dout = _bf(rng, T, H).to(DEV)
    dy, dw = nv.moe_combine_bwd(dout, y, inv, w, off)
    dlogits = nv.router_topk_bwd(ids, w, dw, E)
    # gradient of the second product's operand: the product with the transposed weights
    b2t, s2t = nv.fp8_quantize_weight(nv.weight_layout(w2, False))
    dh = nv.fp8_grouped_gemm(*nv.fp8_quantize(dy), b2t, s2t, offsets=off)
    dxr = nv.moe_dispatch_bwd(rows, inv, off, k)
    torch.cuda.synchronize()

    hinv, n = host(inv), int(off[-1])
    rdy, rdw, mag = P.combine_bwd(bf16_values(host(dout)).astype(np.float32), bf16_values(host(y)).astype(np.float32),
                                  hinv, host(w), n)
    assert np.array_equal(bf16_values(host(dy)), F.bf16_bits_to_f32(F.round_to_bf16(rdy)).astype(np.float64))
    assert np.all(np.abs(host(dw) - rdw) <= (H + 16) * 2.0 ** -24 * mag)
    rl, lm = P.router_bwd(host(ids), host(w), host(dw), E)
    assert np.all(np.abs(host(dlogits) - rl) <= (k + 4) * 2.0 ** -24 * lm)
    # each token's rows are k copies of it: their sum is k * x, rounded once
    assert np.all(np.abs(bf16_values(host(dxr)) - k * x.double().numpy()) <= 2.0 ** -8 * k * np.abs(x.double().numpy()))
    qd, sd = P.quantize(bf16_values(host(dy)).astype(np.float32))
    wl = []
    for e in range(E):
        qt, st = P.quantize(w2[e].float().cpu().numpy().T.copy(), 128)
        wl.append(P.decode(qt, st, 128))
    ref, rm, peak = P.grouped_product(P.decode(qd, sd), wl, host(off), np.arange(T * k))
    # the product's bound, see test_gpu_fp8.py
    bound = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * ((128 + 2 + 2 + 8) * 2.0 ** -23 * rm + 7 * 2.0 ** -13 * peak)
    assert np.all(np.abs(bf16_values(host(dh)) - ref)[:n] <= bound[:n])

    # the router's gradient is the derivative of <combine, dout>: a difference
    # quotient in float64 over the logits, with the device's expert rows
    yv, dv = bf16_values(host(y)), bf16_values(host(dout))
    lg, hids = host(logits).astype(np.float64), host(ids)

    def value(lg):
        v = np.take_along_axis(lg, hids, 1)
        e = np.exp(v - v.max(1, keepdims=True))
        ww = e / e.sum(1, keepdims=True)
        return (np.einsum("tk,tkh->th", ww, yv[hinv].reshape(T, k, H)) * dv).sum(1)

    for e in range(E):
        p, m = lg.copy(), lg.copy()
        p[:, e] += 1e-5
        m[:, e] -= 1e-5
        np.testing.assert_allclose(host(dlogits)[:, e], (value(p) - value(m)) / 2e-5, rtol=1e-3, atol=2e-3)
    assert out.shape == (T, H)


def test_gradients_replay_from_a_graph():
    rng = np.random.default_rng(41)
    T, k, E, H = 21, 4, 8, 1000
    x, y, w = _bf(rng, T, H).to(DEV), _bf(rng, T * k, H).to(DEV), torch.rand((T, k), device=DEV)
    ids = torch.from_numpy(rng.integers(0, E, (T, k)).astype(np.int32)).to(DEV)

    def step():
        off, _, inv, _ = nv.moe_route(ids, E)
        rows = nv.moe_dispatch(x, inv, off, k)
        dy, dw = nv.moe_combine_bwd(x, y, inv, w, off)
        return rows, nv.moe_dispatch_bwd(y, inv, off, k), dy, dw, nv.router_topk_bwd(ids, w, dw, E)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = step()
    for r in range(4):
        x.copy_(_bf(np.random.default_rng(r), T, H))
        ids.copy_(torch.from_numpy(np.random.default_rng(r).integers(-1, E, (T, k)).astype(np.int32)))
        want = [t.clone() for t in step()]
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), r


def test_gradients_chained_from_the_output_to_the_tokens():
    """The backward pass of dispatch, product, SwiGLU, product, combine, each
    link fed the gradient that the one before gave: combine, the product with the
    transposed second weight, SwiGLU (its gradient here in PyTorch), the product
    with the transposed first weight, dispatch.  The transposed weights are the
    forward's own codes and 128 x 128 scales, both transposed.  Each link
    against float64 on its device inputs, with that link's bound, in the host's
    own order of rows and slots; pairs without an expert among them."""
    rng = np.random.default_rng(77)
    T, H, I, E, k = 45, 272, 144, 5, 3
    x = _bf(rng, T, H).to(DEV)
    ids, off, perm, inv = _routing(rng, T, k, E, 0.15)
    n, hinv, hoff = int(off[-1]), host(inv), host(off)
    assert n < T * k
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32)).to(DEV)
    b1, s1 = nv.fp8_quantize_weight((_bf(rng, E, 2 * I, H) * 0.1).to(DEV))
    b2, s2 = nv.fp8_quantize_weight((_bf(rng, E, H, I) * 0.1).to(DEV))

    def transposed(b, s):
        return b.view(torch.uint8).transpose(1, 2).contiguous().view(b.dtype), s.transpose(1, 2).contiguous()

    q, sf = nv.fp8_quantize(x)
    y1 = nv.fp8_grouped_gemm(q, sf, b1, s1, offsets=off, M=T * k, a_row_src=perm, a_row_div=k)
    h, hs = nv.fp8_swiglu_quantize(y1, offsets=off)
    y = nv.fp8_grouped_gemm(h, hs, b2, s2, offsets=off)
    dout = _bf(rng, T, H).to(DEV)
    dy, dw = nv.moe_combine_bwd(dout, y, inv, w, off)
    qy = nv.fp8_quantize(dy)
    dh = nv.fp8_grouped_gemm(*qy, *transposed(b2, s2), offsets=off)
    gate, up, d = y1[:n, :I].float(), y1[:n, I:].float(), dh[:n].float()
    sig = torch.sigmoid(gate)
    dy1 = torch.zeros((T * k, 2 * I), dtype=torch.bfloat16, device=DEV)
    dy1[:n, :I] = d * up * sig * (1 + gate * (1 - sig))
    dy1[:n, I:] = d * gate * sig
    q1 = nv.fp8_quantize(dy1)
    drows = nv.fp8_grouped_gemm(*q1, *transposed(b1, s1), offsets=off)
    dx = nv.moe_dispatch_bwd(drows, inv, off, k)
    torch.cuda.synchronize()

    f64 = lambda t: bf16_values(host(t))
    codes = lambda t: t.view(torch.uint8).cpu().numpy()
    # combine: row inv[t*k+j] is w[t][j] dout[t], rounded once
    rdy = np.zeros((T * k, H))
    for f in range(T * k):
        if hinv[f] < n:
            assert ids[f // k, f % k] == np.searchsorted(hoff, hinv[f], side="right") - 1
            rdy[hinv[f]] = float(w[f // k, f % k]) * f64(dout)[f // k]
    assert np.all(np.abs(f64(dy) - rdy) <= 2.0 ** -8 * np.abs(rdy) * (1 + 2.0 ** -16))
    # both products against the weights as they were quantised for the forward, transposed in float64
    for got, (qa, sa), (b, s) in ((dh, qy, (b2, s2)), (drows, q1, (b1, s1))):
        wl = [P.decode(codes(b)[e], host(s)[e], 128).T for e in range(E)]
        ref, mag, peak = P.grouped_product(P.decode(codes(qa), host(sa)), wl, hoff, np.arange(T * k))
        kb = -(-qa.shape[1] // 128)
        bound = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * ((128 + 2 + kb + 8) * 2.0 ** -23 * mag + 7 * 2.0 ** -13 * peak)
        assert np.all((np.abs(f64(got) - ref) <= bound)[:n])
    # dispatch: each token's rows, in its slots' order
    ref, mag = P.dispatch_bwd(f64(drows), hinv, n, k)
    assert np.all(np.abs(f64(dx) - ref) <= 2.0 ** -8 * np.abs(ref) + k * 2.0 ** -24 * mag)
    none = (hinv.reshape(T, k) >= n).all(1)
    assert np.all(f64(dx)[none] == 0) and np.any(f64(dx)[~none] != 0)
    # SwiGLU's formula above against differences, in float64
    g, u, dd = (t.double().cpu().numpy() for t in (gate, up, d))
    eps = 1e-6
    silu = lambda v: v / (1 + np.exp(-v))
    for col, diff in ((0, (silu(g + eps) - silu(g - eps)) / (2 * eps) * u * dd), (I, silu(g) * dd)):
        have = f64(dy1)[:n, col:col + I]
        # one BF16 rounding, eight fp32 operations on terms up to (1 + |g|) the factors, the quotient's own 1e-9
        assert np.all(np.abs(have - diff) <= 2.0 ** -8 * np.abs(diff) + (16 * 2.0 ** -23 + 1e-9) * (1 + np.abs(g)) ** 2 * (1 + np.abs(u)) * np.abs(dd))


def test_combine_of_more_tokens_than_a_row_of_workgroups():
    """6 million tokens of eight columns, 896 threads each: more than 2^32."""
    T = 6_000_011
    g = torch.Generator(DEV).manual_seed(2)
    inv = torch.randperm(T, device=DEV, generator=g)
    y = torch.randn((T, 8), device=DEV, generator=g).to(torch.bfloat16)
    off = torch.tensor([0, T - 3], dtype=torch.int32, device=DEV)
    out = torch.full((T, 8), 9.0, dtype=torch.bfloat16, device=DEV)
    nv.moe_combine(y, inv.to(torch.int32), torch.full((T, 1), 0.5, device=DEV), off, out=out)
    want = torch.where((inv < T - 3)[:, None], y[inv] * 0.5, torch.zeros_like(y))
    assert torch.equal(out, want)


def test_router_of_more_tokens_than_a_row_of_workgroups():
    """2^26 + 5 tokens, a wave each: more than 2^32 threads."""
    T = (1 << 26) + 5
    lg = torch.randn((T, 2), device=DEV, generator=torch.Generator(DEV).manual_seed(4))
    ids, w = nv.router_topk(lg, 1)
    assert torch.equal(ids[:, 0], (lg[:, 1] > lg[:, 0]).to(torch.int32)) and torch.all(w == 1)
