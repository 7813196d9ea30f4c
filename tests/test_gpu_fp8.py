"""GPU parity of the FP8 block quantisers and the FP8 grouped product.

Tolerances.  Quantised rows and weights: bit-exact (a fixed fp32 sequence).
SwiGLU: see `_check_swiglu`.  Product: the reference is float64 on the exactly
decoded operands; the kernel rounds once to BF16 (2^-8 relative) and sums in
fp32: 128 products a block, one product with each of two scales, at most
ceil(K/128) block sums and 8 partial sums, each at most 2^-23 of the sum of the
terms' magnitudes (2^-24 if it rounds, twice that if the matrix unit truncates).
The matrix unit adds eight consecutive products in fixed point first: measured
with one product of 2^16, its negative and a third of 2^t, the third survives
down to t = 3 inside the eight and down to 2^-7 outside them.  So each of the
seven products beside the largest loses less than 2^-13 of that one:
7 * 2^-13 of the sum over the eights of their largest term (`peak`)."""

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_04_amd as nv
from oracle import formats as F
from oracle import fp8 as P
from parity import host, bf16_values

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _acts(rng, R, C):
    x = rng.standard_normal((R, C)) * np.exp(0.5 * rng.standard_normal((R, 1)))
    x[:, ::64] *= 12
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)


def _codes(t):
    return t.view(torch.uint8).cpu().numpy()


def _f32(t):
    return t.float().numpy()


@pytest.mark.parametrize("R,C", [(1, 16), (1, 128), (3, 144), (4, 7168), (5, 112), (37, 1040), (130, 256), (257, 48)])
def test_quantize_rows_bit_exact(R, C):
    print(f"[case] fp8 rows R={R} C={C}", flush=True)
    x = _acts(np.random.default_rng(R * 10007 + C), R, C)
    if R > 2:
        x[1] = 0
        x[2, :16] = 1e-38
    q, sf = nv.fp8_quantize(x.to(DEV))
    rq, rs = P.quantize(_f32(x))
    assert q.dtype == torch.float8_e4m3fn and q.shape == (R, C) and sf.shape == rs.shape
    assert np.array_equal(host(sf).view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(_codes(q), rq)


def test_quantize_every_bf16_magnitude():
    """One block per finite positive BF16 value as the block's largest, with
    halves and small parts of it in the same block."""
    bits = np.arange(0x0000, 0x7F80, dtype=np.uint16)
    top = F.bf16_bits_to_f32(bits)
    x = np.zeros((len(top), 128), np.float32)
    for i in range(128):
        x[:, i] = top * np.float32((i - 64) / 64 if i else 1)
    x = torch.from_numpy(x).to(torch.bfloat16)
    q, sf = nv.fp8_quantize(x.to(DEV))
    rq, rs = P.quantize(_f32(x))
    assert np.array_equal(host(sf).view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(_codes(q), rq)


def test_quantize_strided_rows_and_row_count():
    rng = np.random.default_rng(2)
    big = _acts(rng, 19, 600).to(DEV)
    x = big[:, 8:8 + 272]                               # rows 600 apart, first element 16 bytes in
    q, sf = nv.fp8_quantize(x)
    rq, rs = P.quantize(x.float().cpu().numpy())
    assert np.array_equal(_codes(q), rq) and np.array_equal(host(sf), rs)
    for n in (0, 1, 13, 19, 25):                        # rows behind the count stay as they were
        off = torch.tensor([0, 1, n], dtype=torch.int32, device=DEV)
        q2 = torch.full((19, 272), 0x55, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        s2 = torch.full((19, 3), -7.0, device=DEV)
        nv.fp8_quantize(x, offsets=off, out=(q2, s2))
        m = min(n, 19)
        assert np.array_equal(_codes(q2)[:m], rq[:m]) and np.all(_codes(q2)[m:] == 0x55)
        assert np.array_equal(host(s2)[:m], rs[:m]) and np.all(host(s2)[m:] == -7.0)


@pytest.mark.parametrize("G,N,K", [(1, 1, 16), (2, 128, 128), (3, 130, 272), (1, 300, 1040), (2, 64, 112)])
def test_quantize_weight_bit_exact(G, N, K):
    print(f"[case] fp8 weight G={G} N={N} K={K}", flush=True)
    w = _acts(np.random.default_rng(N + K), G * N, K).view(G, N, K)
    q, sf = nv.fp8_quantize_weight(w.to(DEV))
    for g in range(G):
        rq, rs = P.quantize(_f32(w[g]), 128)
        assert np.array_equal(host(sf)[g], rs) and np.array_equal(_codes(q)[g], rq)


def _check_swiglu(x, q, sf):
    """h = g / (1 + exp(-g)) * u in fp32 against float64: exp2 and the reciprocal
    within an ulp (2^-23 each), four roundings of 2^-24 between, so 2^-21 relative
    covers h; the scale adds 2^-24.  A code then stands for h up to half its
    step, plus that error of h (a value within it of a midpoint may go either
    way)."""
    h = P.swiglu(_f32(x))
    m = np.maximum(P._amax_blocks(h.astype(np.float32), 1).astype(np.float64), 2.0 ** -100)
    s = host(sf).astype(np.float64)
    assert np.all(np.abs(s - m / 448) <= m / 448 * 2.0 ** -20)
    ss = np.repeat(s, 128, 1)[:, :h.shape[1]]
    v = np.abs(h) / ss
    step = np.exp2(np.floor(np.log2(np.maximum(v * (1 + 2.0 ** -20), 2.0 ** -6))) - 3)
    got = F.e4m3_decode(_codes(q)) * ss
    assert np.all(np.abs(got - h) <= ss * step / 2 + np.abs(h) * 2.0 ** -20)


@pytest.mark.parametrize("R,I", [(1, 16), (5, 128), (33, 272), (64, 2048), (3, 144)])
def test_swiglu_quantize(R, I):
    print(f"[case] fp8 swiglu R={R} I={I}", flush=True)
    x = _acts(np.random.default_rng(R + I), R, 2 * I)
    x[0, :8] = torch.tensor([0.0, -0.0, 90.0, -90.0, 300.0, -300.0, 3e38, -3e38], dtype=torch.bfloat16)
    x[0, I:I + 8] = 1e-30
    q, sf = nv.fp8_swiglu_quantize(x.to(DEV))
    assert q.shape == (R, I)
    _check_swiglu(x, q, sf)


def test_swiglu_of_every_bf16_gate():
    """One gate a row, up 1: the row's scale is |silu| / 448.  exp2 and the
    reciprocal within an ulp (2^-23 each), four roundings of 2^-24 on the way to
    silu and two of the scale: 2^-21 + 2^-23 relative, down to the floor of
    2^-100; one sign's infinity and NaN give NaN codes."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    x = torch.zeros((1 << 16, 32), dtype=torch.bfloat16)
    x[:, 0] = bits.view(torch.bfloat16)
    x[:, 16] = 1
    q, sf = nv.fp8_swiglu_quantize(x.to(DEV))
    g = x[:, 0].double().numpy()
    with np.errstate(over="ignore", invalid="ignore"):
        h = g / (1 + np.exp(-g))
    got, code = host(sf)[:, 0].astype(np.float64), _codes(q)
    ok = np.isfinite(h)
    want = np.maximum(np.abs(h[ok]), 2.0 ** -100) / 448
    assert np.all(np.abs(got[ok] - want) <= want * (2.0 ** -21 + 2.0 ** -23))
    assert np.array_equal(code[ok, 0] >= 0x80, np.signbit(g[ok]))
    assert np.all(code[~ok, 0] & 0x7F == 0x7F) and np.all(code[:, 1:] == 0)


def test_swiglu_row_count_leaves_the_rest():
    x = _acts(np.random.default_rng(8), 9, 64).to(DEV)
    ref, rs = nv.fp8_swiglu_quantize(x)
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    q = torch.full((9, 32), 0x33, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    s = torch.full((9, 1), 5.0, device=DEV)
    nv.fp8_swiglu_quantize(x, offsets=off, out=(q, s))
    assert np.array_equal(_codes(q)[:4], _codes(ref)[:4]) and np.all(_codes(q)[4:] == 0x33)
    assert np.array_equal(host(s)[:4], host(rs)[:4]) and np.all(host(s)[4:] == 5.0)


# ------------------------------------------------------------------ product

def _operands(rng, R, E, N, K, special=False):
    a, asf = P.quantize(_acts(rng, R, K).float().numpy())
    b = np.clip(np.round(rng.standard_normal((E, N, K)) * 110 * 8) / 8, -448, 448)
    b = P.e4m3_encode(b)
    bsf = (2e-4 * np.exp(0.3 * rng.standard_normal((E, -(-N // 128), -(-K // 128))))).astype(np.float32)
    if special and R > 1:
        a[0] = 0                                        # a row of zero codes
        asf[1] *= np.float32(2.0 ** 40)                 # rows and blocks of very different size
        bsf[0, 0, 0] *= np.float32(2.0 ** -60)
    return a, asf, b, bsf


def _dev(a, asf, b, bsf):
    t = lambda v: torch.from_numpy(v).to(DEV)
    return (t(a).view(torch.float8_e4m3fn), t(asf), t(b).view(torch.float8_e4m3fn), t(bsf))


def _check(c, ref, mag, peak, K, live):
    KB = -(-K // 128)
    got = bf16_values(host(c))[:live]
    sums = (128 + 2 + KB + 8) * 2.0 ** -23 * mag[:live] + 7 * 2.0 ** -13 * peak[:live]
    bound = 2.0 ** -8 * np.abs(ref[:live]) + (1 + 2.0 ** -8) * sums
    bad = np.abs(got - ref[:live]) > bound
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], np.abs(got - ref[:live])[bad][:4], bound[bad][:4])


def _run(counts, N, K, k=1, extra=0, seed=0, special=False, gather=False, bad=False):
    """Expert row counts -> operands, the call, the check; `extra` rows of c
    behind the last expert and a band around c stay as they were."""
    print(f"[case] fp8 product counts={counts if len(counts) < 12 else len(counts)} N={N} K={K} gather={gather}", flush=True)
    rng = np.random.default_rng(seed + N * 7 + K)
    E, live = len(counts), int(np.sum(counts))
    M = live + extra
    R = max(1, -(-M // k)) if gather else max(M, 1)
    a, asf, b, bsf = _operands(rng, R, E, N, K, special)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    src, rows = None, np.arange(M)
    if gather:
        src = rng.permutation(R * k)[:M].astype(np.int32)
        if bad and M > 3:
            src[1], src[2], src[M // 2] = -k * 5, -1, (R + 3) * k       # indices outside A: rows of zeros
        rows = np.where((src // k >= 0) & (src >= 0) & (src // k < R), src // k, -1)
    ref, mag, peak = P.grouped_product(P.decode(a, asf), [P.decode(b[e], bsf[e], 128) for e in range(E)], off, rows)
    da, das, db, dbs = _dev(a, asf, b, bsf)
    buf = torch.full((M * N + 128,), 3.0, dtype=torch.bfloat16, device=DEV)
    c = buf[64:64 + M * N].view(M, N)
    nv.fp8_grouped_gemm(da, das, db, dbs, offsets=torch.from_numpy(off).to(DEV), M=M,
                        a_row_src=None if src is None else torch.from_numpy(src).to(DEV), a_row_div=k, out=c)
    torch.cuda.synchronize()
    _check(c, ref, mag, peak, K, live)
    assert torch.all(buf[:64] == 3) and torch.all(buf[64 + live * N:] == 3)


@pytest.mark.parametrize("K", [16, 112, 128, 144, 272, 1024, 1040, 1152, 2320])
def test_product_depths(K):
    _run([3, 0, 5], 72, K)


@pytest.mark.parametrize("N", [1, 2, 15, 63, 64, 65, 127, 128, 129, 200, 257, 513])
def test_product_widths(N):
    _run([4, 1], N, 272)
    _run([70, 150], N, 272)


@pytest.mark.parametrize("counts", [[1], [16], [17], [33], [64], [65], [200], [257], [300, 0, 0, 1],
                                    [0, 0, 0], [0, 31, 0, 64, 129, 1], [1] * 70, [3] * 130 + [90]],
                         ids=lambda c: f"{len(c)}x{sum(c)}")
def test_product_row_counts(counts):
    _run(counts, 192, 400, extra=7)


@pytest.mark.parametrize("counts", [[5, 0, 9], [40, 41, 42], [100, 200], [513], [600, 30]])
@pytest.mark.parametrize("bad", [False, True])
def test_product_gather(counts, bad):
    _run(counts, 136, 528, k=3, extra=2, gather=True, bad=bad)


def test_product_special_values():
    _run([6, 40], 200, 272, special=True)
    _run([90, 140], 200, 272, special=True)


@pytest.mark.parametrize("M", [1, 2, 15, 16, 31, 100, 257, 700, 1300])
@pytest.mark.parametrize("N,K", [(192, 656), (1001, 128)])
def test_product_dense(M, N, K):
    print(f"[case] fp8 dense M={M} N={N} K={K}", flush=True)
    a, asf, b, bsf = _operands(np.random.default_rng(M + N), M, 1, N, K)
    c = nv.fp8_grouped_gemm(*_dev(a, asf, b, bsf))
    ref, mag, peak = P.grouped_product(P.decode(a, asf), [P.decode(b[0], bsf[0], 128)], [0, M], np.arange(M))
    assert c.shape == (M, N)
    _check(c, ref, mag, peak, K, M)


# Sizes at which each of the product's kernels is the one taken on 256 CUs: m
# tiles of 32*jv rows, one a CU; ragged experts of tiles that hold one expert
# or more; experts of few rows, many of them.

@pytest.mark.parametrize("jv", range(3, 10))
@pytest.mark.parametrize("N,K", [(200, 272), (72, 16)])
def test_product_dense_tiles(jv, N, K):
    M = 256 * 32 * jv - 19
    print(f"[case] fp8 dense tiles jv={jv} M={M} N={N} K={K}", flush=True)
    a, asf, b, bsf = _operands(np.random.default_rng(jv), M, 1, N, K, special=True)
    c = nv.fp8_grouped_gemm(*_dev(a, asf, b, bsf))
    ref, mag, peak = P.grouped_product(P.decode(a, asf), [P.decode(b[0], bsf[0], 128)], [0, M], np.arange(M))
    _check(c, ref, mag, peak, K, M)


@pytest.mark.parametrize("N,shift", [(65, 0), (70, 0), (258, 0), (72, 1), (72, 2), (3, 1), (62, 2)])
def test_product_tile_widths_and_places(N, shift):
    """Rows at 2-, 4- and 16-byte places; nothing before or behind them is written."""
    M, K = 256 * 96 - 5, 144
    print(f"[case] fp8 tile widths N={N} shift={shift}", flush=True)
    a, asf, b, bsf = _operands(np.random.default_rng(N), M, 1, N, K)
    buf = torch.full((M * N + 16,), 3.0, dtype=torch.bfloat16, device=DEV)
    c = buf[8 + shift:8 + shift + M * N].view(M, N)
    nv.fp8_grouped_gemm(*_dev(a, asf, b, bsf), out=c)
    ref, mag, peak = P.grouped_product(P.decode(a, asf), [P.decode(b[0], bsf[0], 128)], [0, M], np.arange(M))
    _check(c, ref, mag, peak, K, M)
    assert torch.all(buf[:8 + shift] == 3) and torch.all(buf[8 + shift + M * N:] == 3)


@pytest.mark.parametrize("K", [128, 144, 384, 512, 1040, 1168])
def test_product_grouped_tiles(K):
    rng = np.random.default_rng(K)
    counts = rng.integers(0, 330, 200).tolist()
    counts[3:6] = [0, 1, 700]
    _run(counts, 72, K, k=2, extra=5, gather=K % 3 == 2, special=True, bad=True)


@pytest.mark.parametrize("N,K", [(200, 16), (250, 144), (129, 640), (256, 1040), (180, 784)])
def test_product_streamed_experts(N, K):
    rng = np.random.default_rng(N + K)
    counts = np.minimum(rng.poisson(4, 600), 40)
    counts[[0, 7, 599]] = [37, 0, 16]
    _run(counts.tolist(), N, K, k=3, extra=4, gather=K > 700, special=True, bad=True)


@pytest.mark.parametrize("M,N,K", [(5, 2048, 1040), (40, 2048, 400), (100, 1500, 272), (300, 2040, 272), (500, 2000, 144)])
def test_product_few_rows_shapes(M, N, K):
    print(f"[case] fp8 few rows M={M} N={N} K={K}", flush=True)
    a, asf, b, bsf = _operands(np.random.default_rng(M + N), M, 1, N, K)
    c = nv.fp8_grouped_gemm(*_dev(a, asf, b, bsf))
    ref, mag, peak = P.grouped_product(P.decode(a, asf), [P.decode(b[0], bsf[0], 128)], [0, M], np.arange(M))
    _check(c, ref, mag, peak, K, M)


@pytest.mark.parametrize("counts,N,K", [([53, 61, 0, 64, 40] * 5, 529, 272), ([33, 20], 1735, 400), ([31, 32, 27, 9], 1030, 528),
                                        ([14, 1, 0, 16], 2050, 144), ([70, 90, 100, 30], 1030, 400), ([10, 15, 9] * 6, 129, 1040)],
                         ids=lambda v: f"{len(v)}x{sum(v)}" if isinstance(v, list) else str(v))
def test_product_few_rows_an_expert(counts, N, K):
    _run(counts, N, K, k=2, extra=3, gather=True, bad=True, special=True)


def test_product_layer_shape_against_sampled_columns():
    """A layer's own depth and width (K 7168, N 4096) with ragged experts: all
    rows, columns of every 64-wide group."""
    rng = np.random.default_rng(11)
    counts, N, K = [1, 0, 37, 64, 300], 4096, 7168
    M = sum(counts)
    x = _acts(rng, M, K).to(DEV)
    a, asf = nv.fp8_quantize(x)
    w = torch.randn((5, N, K), device=DEV, generator=torch.Generator(DEV).manual_seed(1)).mul_(0.02).to(torch.bfloat16)
    b, bsf = nv.fp8_quantize_weight(w)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    c = nv.fp8_grouped_gemm(a, asf, b, bsf, offsets=torch.from_numpy(off).to(DEV))
    cols = np.unique(np.concatenate([np.arange(0, N, 64) + rng.integers(0, 64, N // 64), [0, N - 1]]))
    ad = P.decode(_codes(a), host(asf))
    bc, bs = _codes(b), host(bsf)
    wl = [F.e4m3_decode(bc[e][cols]) * np.repeat(bs[e].astype(np.float64)[cols // 128], 128, 1) for e in range(5)]
    ref, mag, peak = P.grouped_product(ad, wl, off, np.arange(M))
    _check(c[:, torch.from_numpy(cols).to(DEV)], ref, mag, peak, K, M)


def test_product_same_bits_and_other_stream():
    rng = np.random.default_rng(12)
    for counts in ([3, 20], [200, 70]):
        ops = _dev(*_operands(rng, sum(counts), 2, 320, 656))
        off = torch.tensor([0, counts[0], sum(counts)], dtype=torch.int32, device=DEV)
        ref = nv.fp8_grouped_gemm(*ops, offsets=off)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            again = [nv.fp8_grouped_gemm(*ops, offsets=off) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(x.view(torch.int16), ref.view(torch.int16)) for x in again)


def test_product_empty_calls():
    ops = _dev(*_operands(np.random.default_rng(1), 4, 2, 32, 128))
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert nv.fp8_grouped_gemm(ops[0][:0], ops[1][:0], *ops[2:], offsets=off).shape == (0, 32)
    c = torch.full((4, 32), 2.0, dtype=torch.bfloat16, device=DEV)
    nv.fp8_grouped_gemm(*ops, offsets=off, out=c)                    # no expert has rows
    assert torch.all(c == 2)
    q, sf = nv.fp8_quantize(torch.zeros((0, 32), dtype=torch.bfloat16, device=DEV))
    assert q.shape == (0, 32) and sf.shape == (0, 1)


def test_binding_refusals():
    ops = _dev(*_operands(np.random.default_rng(1), 4, 2, 32, 128))
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        nv.fp8_grouped_gemm(*ops, offsets=off, M=5)
    with pytest.raises(ValueError):
        nv.fp8_grouped_gemm(*ops, offsets=off[:2])
    with pytest.raises(nv.Nvfp4Error):
        nv.fp8_grouped_gemm(*ops)                                    # two experts, no offsets
    with pytest.raises(TypeError):
        nv.fp8_grouped_gemm(ops[0].view(torch.uint8), *ops[1:], offsets=off)
    with pytest.raises(ValueError):
        nv.fp8_grouped_gemm(ops[0], ops[1].t(), *ops[2:], offsets=off)
    with pytest.raises(ValueError):
        nv.fp8_quantize(torch.zeros((2, 32), dtype=torch.bfloat16, device=DEV), offsets=off[:0])
    with pytest.raises(nv.Nvfp4Error):
        nv.fp8_quantize(torch.zeros((2, 24), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        nv.fp8_swiglu_quantize(torch.zeros((2, 33), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        nv.fp8_grouped_gemm(*ops, offsets=off, out=torch.zeros((4, 33), dtype=torch.bfloat16, device=DEV))


def test_product_and_quantise_replay_from_a_graph():
    rng = np.random.default_rng(21)
    x = _acts(rng, 96, 656).to(DEV)
    _, _, b, bsf = _dev(*_operands(rng, 1, 2, 320, 656))
    off = torch.tensor([0, 20, 96], dtype=torch.int32, device=DEV)
    out = torch.zeros((96, 320), dtype=torch.bfloat16, device=DEV)
    hq = (torch.zeros((96, 160), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn), torch.zeros((96, 2), device=DEV))

    def step():
        a, asf = nv.fp8_quantize(x)
        nv.fp8_grouped_gemm(a, asf, b, bsf, offsets=off, out=out)
        nv.fp8_swiglu_quantize(out, out=hq)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for r in range(4):
        x.copy_(_acts(np.random.default_rng(100 + r), 96, 656))
        if r == 2:
            off.copy_(torch.tensor([0, 90, 96], dtype=torch.int32))
        step()
        torch.cuda.synchronize()
        want = out.clone(), _codes(hq[0]).copy(), host(hq[1]).copy()
        out.zero_()
        hq[1].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want[0].view(torch.int16)), r
        assert np.array_equal(_codes(hq[0]), want[1]) and np.array_equal(host(hq[1]), want[2])


@pytest.mark.parametrize("K", [272, 640, 784, 1040])
@pytest.mark.parametrize("counts", [[30, 2], [3] * 700, [250] * 200])
def test_product_bad_row_stays_its_own(counts, K):
    """NaN and infinite scales of one A row, and of rows that no expert takes,
    reach no other row (odd numbers of K blocks, a gather of neighbours)."""
    print(f"[case] fp8 bad rows K={K} experts={len(counts)}", flush=True)
    rng = np.random.default_rng(K)
    M, E, N = sum(counts), len(counts), 72
    R = M + 3
    a, asf, b, bsf = _operands(rng, R, E, N, K)
    asf[5], asf[M - 2], asf[M:] = np.nan, np.inf, np.nan
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    src = rng.permutation(M).astype(np.int32)
    ops = _dev(a, asf, b, bsf)
    for s in (src, None):
        c = nv.fp8_grouped_gemm(*ops, offsets=torch.from_numpy(off).to(DEV), M=M,
                                a_row_src=None if s is None else torch.from_numpy(s).to(DEV))
        rows = np.arange(M) if s is None else s
        good = np.isfinite(asf[rows]).all(1)
        clean = np.where(np.isfinite(asf), asf, 0).astype(np.float32)
        ref, mag, peak = P.grouped_product(P.decode(a, clean), [P.decode(b[e], bsf[e], 128) for e in range(E)], off, rows)
        got = bf16_values(host(c))
        assert np.isfinite(got[good]).all() and not np.isfinite(got[~good]).any()
        sums = (128 + 2 + K // 128 + 9) * 2.0 ** -23 * mag + 7 * 2.0 ** -13 * peak
        assert np.all((np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * sums)[good])


def _ones(R, K):
    """(R, K) codes of 1.0, made in pieces: R * K may pass 2^32."""
    q = torch.empty((R, K), dtype=torch.uint8, device=DEV)
    for part in q.split(1 << 26):
        part.fill_(0x38)
    return q.view(torch.float8_e4m3fn)


@pytest.mark.parametrize("grouped", [False, True])
def test_product_of_nearly_two_to_the_31_rows(grouped):
    """2^31 - 100 rows, one column: row d is 16 times its scale, 1 .. 7 in turn
    (52 GB of operands and output)."""
    M = (1 << 31) - 100
    print(f"[case] fp8 rows M={M} grouped={grouped}", flush=True)
    a, asf = _ones(M, 16), torch.empty((M, 1), device=DEV)
    for i, part in enumerate(asf.view(-1).split(1 << 26)):
        part.copy_((torch.arange(len(part), device=DEV) + (i << 26)) % 7 + 1)
    c = torch.zeros((M + 8, 1), dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, M], dtype=torch.int32, device=DEV) if grouped else None
    nv.fp8_grouped_gemm(a, asf, _ones(1, 16)[None], torch.ones((1, 1, 1), device=DEV), offsets=off, out=c[:M])
    for got, s in zip(c[:M].view(-1).split(1 << 26), asf.view(-1).split(1 << 26)):
        assert torch.equal(got, (16 * s).to(torch.bfloat16))
    assert torch.all(c[M:] == 0)


def test_quantize_more_weight_blocks_than_a_row_of_workgroups():
    """2^24 + 5 weights of one block each: more threads than 2^32.  Column 0 is
    448 times a power of two, which is the scale."""
    G = (1 << 24) + 5
    s = torch.exp2((torch.arange(G, device=DEV) % 9 - 4).float())
    w = torch.zeros((G, 1, 16), dtype=torch.bfloat16, device=DEV)
    w[:, 0, 0], w[:, 0, 15] = 448 * s, -2 * s
    q, sf = nv.fp8_quantize_weight(w)
    assert torch.equal(sf.view(-1), s)
    q = q.view(torch.uint8).view(G, 16)
    assert torch.all(q[:, 0] == 0x7E) and torch.all(q[:, 15] == 0xC0) and not q[:, 1:15].any()


@pytest.mark.parametrize("rows", [1, 13])
def test_product_of_more_tiles_than_a_row_of_workgroups(rows):
    """17 experts of 2^27 - 128 columns with 1 and 13 rows each: more than 2^32
    threads of the streaming and of the tile kernel (42 and 96 GB)."""
    E, N, K = 17, (1 << 27) - 128, 16
    M = E * rows
    print(f"[case] fp8 wide experts rows={rows} N={N}", flush=True)
    a, asf = _ones(M, K), torch.ones((M, 1), device=DEV)
    b = _ones(E * N, K).view(E, N, K)
    bsf = (torch.arange(E * (N // 128), device=DEV) % 7 + 1).float().view(E, N // 128, 1)
    off = torch.arange(0, M + 1, rows, dtype=torch.int32, device=DEV)
    c = torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)
    nv.fp8_grouped_gemm(a, asf, b, bsf, offsets=off, out=c)
    for d in range(M):
        want = (16 * bsf[d // rows]).to(torch.bfloat16)
        assert torch.equal(c[d].view(-1, 128), want.expand(-1, 128)), d


@pytest.mark.parametrize("K", [128, 272, 512, 784])
@pytest.mark.parametrize("counts", [[30, 2], [3] * 700, [250] * 200], ids=["few_rows", "streamed", "tiles"])
@pytest.mark.parametrize("last", [False, True])
def test_product_infinite_weight_scale(counts, K, last):
    """One block of one expert's weight with an infinite scale: its columns are
    infinite with the sign of that block's sum, and no other output changes."""
    print(f"[case] fp8 infinite weight scale K={K} experts={len(counts)} last={last}", flush=True)
    rng = np.random.default_rng(K + len(counts))
    M, E, N = sum(counts), len(counts), 136
    a, asf, b, bsf = _operands(rng, M, E, N, K)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    e, kb = E // 2, bsf.shape[2] - 1 if last else 0
    offd = torch.from_numpy(off).to(DEV)
    clean = bf16_values(host(nv.fp8_grouped_gemm(*_dev(a, asf, b, bsf), offsets=offd)))
    bsf[e, 0, kb] = np.inf
    got = bf16_values(host(nv.fp8_grouped_gemm(*_dev(a, asf, b, bsf), offsets=offd)))
    lo, hi, k0, k1 = off[e], off[e + 1], kb * 128, min(K, kb * 128 + 128)
    x, w = F.e4m3_decode(a[lo:hi, k0:k1]), F.e4m3_decode(b[e, :128, k0:k1])
    dot = x @ w.T
    sure = np.abs(dot) > 2.0 ** -8 * (np.abs(x) @ np.abs(w).T)      # far from what the sum may be off by
    assert sure.any() and np.array_equal(got[lo:hi, :128][sure], np.sign(dot[sure]) * np.inf)
    got[lo:hi, :128] = clean[lo:hi, :128]
    assert np.array_equal(got, clean)


def _odd_values(rng, R, C):
    """Activations with NaN (quiet and signalling, both signs) in every third
    row, infinities in every fifth, and one block of nothing but NaN."""
    x = _acts(rng, R, C)
    for i, bits in enumerate([0x7FC0, 0xFFC0, 0x7F81, 0xFF81]):
        x.view(torch.int16)[::3, 5 + 7 * i] = bits - (0x10000 if bits & 0x8000 else 0)
    x[1::5, C - 3], x[2::5, 2] = float("inf"), float("-inf")
    x[0, :128] = float("nan")
    return x


def _same_codes(got, want):
    nan = want & 0x7F == 0x7F                            # of either sign
    return np.array_equal(got & 0x7F == 0x7F, nan) and np.array_equal(got[~nan], want[~nan])


@pytest.mark.parametrize("R,C", [(17, 272), (600, 16384)])
def test_quantize_nan_and_infinity(R, C):
    """Bit-exact, but for a NaN code's sign: one and four rows a lane group."""
    print(f"[case] fp8 odd values R={R} C={C}", flush=True)
    x = _odd_values(np.random.default_rng(R), R, C)
    q, sf = nv.fp8_quantize(x.to(DEV))
    rq, rs = P.quantize(_f32(x))
    assert np.array_equal(host(sf), rs) and _same_codes(_codes(q), rq)
    assert np.isinf(rs).any() and (rq & 0x7F == 0x7F).any()


@pytest.mark.parametrize("N,K", [(130, 272), (300, 160)])
def test_quantize_weight_nan_and_infinity(N, K):
    x = _odd_values(np.random.default_rng(N), N, K)
    x[:128, :128].nan_to_num_(nan=float("nan"), posinf=3.0, neginf=-3.0)   # NaN alone in the first block
    q, sf = nv.fp8_quantize_weight(x[None].to(DEV))
    rq, rs = P.quantize(_f32(x), 128)
    assert np.array_equal(host(sf)[0], rs) and _same_codes(_codes(q)[0], rq)
    assert np.isfinite(rs[0, 0]) and np.isinf(rs).any()


def test_swiglu_quantize_nan_and_infinity():
    """A NaN gate or up value has the NaN code and leaves its block's others; an
    infinite product takes its block."""
    x = _acts(np.random.default_rng(5), 6, 2 * 256)
    y = x.clone()
    y[0, 3], y[1, 256 + 200] = float("nan"), float("nan")
    y[2, 140], y[2, 256 + 140] = 3e38, 3e38
    small = [(0, 3), (1, 200)]
    for r, c in small:
        x[r, c] = 0                                      # what the others' scale is made from
    ref, rs = nv.fp8_swiglu_quantize(x.to(DEV))
    q, sf = nv.fp8_swiglu_quantize(y.to(DEV))
    got, want, s, ws = _codes(q), _codes(ref).copy(), host(sf), host(rs).copy()
    for r, c in small:
        assert got[r, c] & 0x7F == 0x7F
        want[r, c] = got[r, c]
    assert got[2, 140] & 0x7F == 0x7F and np.isinf(s[2, 1]) and not (np.delete(got[2, 128:], 12) & 0x7F).any()
    want[2, 128:], ws[2, 1] = got[2, 128:], np.inf
    assert np.array_equal(got, want) and np.array_equal(s, ws)
