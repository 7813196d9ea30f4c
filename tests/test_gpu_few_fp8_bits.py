"""The expert layer for a few tokens, FP8 weights: h enters the second product
with 16 bits.

Every output is p * h_i - q * h_j with codes p, q that let the two terms nearly
cancel, so that the rounding of h is what is left.  The first product has one
term, exact in fp32: h is off by expf (2^-23), its sum, the division (2^-22) and
two products, 12 * 2^-24 at most, and by 2^-8 of 2^-8 of its rounding to a BF16
pair.  The terms of the second product are exact (8 bits by 4), their sums lose
2^-23 of what has gone in a few times, 24 at most."""

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_04_amd as nv
from oracle import formats as F
from parity import bf16_values, host

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _round_bits(h, bits):
    m, e = np.frexp(h)
    return np.ldexp(np.round(m * 2.0 ** bits), e - bits)


@pytest.mark.parametrize("T", [1, 3, 7])
def test_few_fp8_keeps_sixteen_bits_of_h(T):
    rng = np.random.default_rng(T)
    H = I = 256
    x = np.zeros((T, H), np.float32)
    x[:, 5] = rng.integers(129, 256, T) / 128.0            # eight bits each
    c1 = rng.integers(0x28, 0x48, (2 * I, H)).astype(np.uint8)   # codes between 2^-2 and 4
    a = F.e4m3_decode(c1[:, 5])[None] * x[:, 5:6].astype(np.float64)
    g, u = a[:, :I], a[:, I:]
    coef = rng.uniform(0.5, 2, (T, 1)).astype(np.float32)
    h = g / (1 + np.exp(-g)) * u * coef
    codes = np.arange(0x30, 0x40, dtype=np.uint8)          # between 2^-1 and 2: eight steps each
    c2 = np.zeros((H, I), np.uint8)
    for n in range(H):
        ht = h[n % T]
        best = None
        for _ in range(40):
            i, p = rng.integers(I), rng.choice(codes)
            first = F.e4m3_decode(p) * ht[i]
            off = np.abs(F.e4m3_decode(codes)[None] * ht[:, None] / first - 1)
            off[np.abs(ht / ht[i] - 1) < 2.0 ** -20] = np.inf     # not the same h
            j, q = np.unravel_index(np.argmin(off), off.shape)
            if best is None or off[j, q] < best[0]:
                best = off[j, q], i, p, j, codes[q]
        _, i, p, j, q = best
        c2[n, i], c2[n, j] = p, q | 0x80
    b = F.e4m3_decode(c2)
    ref, mag = h @ b.T, np.abs(h) @ np.abs(b).T
    bound = lambda out: mag * (2.0 ** -16 + 12 * 2.0 ** -24 + 24 * 2.0 ** -23) + 2.0 ** -8 * np.abs(out) * (1 + 2.0 ** -6)
    # the bound tells 16 bits from 12
    assert np.mean(np.abs(_round_bits(h, 11) @ b.T - ref) > bound(ref)) > 0.5 / T
    f8 = lambda c: torch.from_numpy(c[None]).view(torch.float8_e4m3fn).to(DEV)
    out = nv.moe_expert_forward_few_fp8(torch.from_numpy(x).to(torch.bfloat16).to(DEV), torch.zeros((T, 1), dtype=torch.int32, device=DEV),
                                        torch.from_numpy(coef).to(DEV), f8(c1), torch.ones((1, 4, 2), device=DEV), f8(c2),
                                        torch.ones((1, 2, 2), device=DEV))
    worst = np.max(np.abs(bf16_values(host(out)) - ref) / bound(ref))
    print(f"[worst share of the bound] {worst:.3f}", flush=True)
    assert worst <= 1.0
