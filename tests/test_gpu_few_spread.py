"""The expert layer for a few tokens, NVFP4 weights, where columns of h that share
a power of two lie far apart.

h is FP16 with a power of two for each 16 columns, and the second product brings
the eight groups of 128 columns to the largest of them.  In units in which that
group's largest lies between 2^14 and 2^15 each step of this rounds to a multiple
of 2^-24 at worst, half of it off: at most 2^-25 for the last step and half as
much for those in front, together below 2^-38 of the largest of the 128."""

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_04_amd as nv
from oracle import few as W
from oracle import formats as F
from parity import bf16_values, host

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _weights(w1, w2):
    """w1 (1, H, 2I) [gate | up] columns, w2 (1, I, H) -> the call's weights and what
    they stand for, w1 (2I, H) and w2 (H, I) in float64."""
    w = nv.prepare_expert_weights([torch.from_numpy(w1).to(torch.bfloat16).to(DEV)], [torch.from_numpy(w2).to(torch.bfloat16).to(DEV)], DEV)
    I = w1.shape[2] // 2
    vals = []
    for name, gs in (("w1", w.gs_w1), ("w2", w.gs_w2)):
        q, sf = host(w.rowmajor[name + "_q"])[0], host(w.rowmajor[name + "_sf"])[0]
        codes = np.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)
        vals.append(F.e2m1_decode(codes).astype(np.float64) * np.repeat(F.e4m3_decode(sf), 16, 1) / np.float64(host(gs)[0]))
    n = np.arange(2 * I)
    a = np.empty_like(vals[0])
    a[np.where(n % 16 < 8, 8 * (n // 16) + n % 8, I + 8 * (n // 16) + n % 8)] = vals[0]
    return w, a, vals[1]


@pytest.mark.parametrize("apart", [6, 8, 9, 10, 11, 12, 14, 17, 20, 21, 22, 24])
@pytest.mark.parametrize("large,small", [(0, 1), (7, 0), (3, 6)])
def test_few_groups_of_h_far_apart(apart, large, small):
    """Group `large` of 16 columns holds about 2^14, group `small` of the same 128 about
    2^(-1 - apart); half of out reads the small one alone, and a second 128 holds
    small ones only."""
    print(f"[case] apart={apart} large={large} small={small}", flush=True)
    rng = np.random.default_rng(100 * apart + large)
    H, I = 256, 256
    x = torch.zeros((2, H))
    x[0, 0], x[0, 16] = 1, 16
    x[1, 0], x[1, 16] = 1, -16
    w1, w2 = np.zeros((1, H, 2 * I), np.float32), np.zeros((1, I, H), np.float32)
    A, B, C = (slice(16 * g, 16 * g + 16) for g in (large, small, 8 + small))
    for half, m in ((0, apart // 2), (I, apart - apart // 2)):
        for g in (B, C):
            w1[0, 0, half:][g] = 2.0 ** -m * rng.uniform(0.7, 1.4, 16)
        w1[0, 0, half:][A] = w1[0, 16, half:][A] = rng.uniform(6, 8, 16)
    w2[0, B] = rng.uniform(0.5, 1, (16, H)) * rng.choice([-1, 1], (16, H))
    w2[0, C, ::4] = 2.0 ** -6
    w2[0, A, 1::2] = rng.uniform(0.5, 1, (16, H // 2))
    w, a, b = _weights(w1, w2)
    assert np.all(a[B, 0] != 0) and np.all(a[I:][B, 0] != 0) and np.all(b[::2, A] == 0) and np.all(b[:, B] != 0)
    ids, tw = np.zeros((2, 1), np.int32), np.array([[1.0], [0.75]], np.float32)
    x = x.to(torch.bfloat16)
    out = nv.moe_expert_forward_few(x.to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(tw).to(DEV), w)
    ref, err = W.forward(x.float().numpy(), ids, tw, lambda e: a, lambda e: b, h_bits=12, h_floor=2.0 ** -38)
    worst = np.max(np.abs(bf16_values(host(out)) - ref) / err)
    print(f"[worst share of the bound] {worst:.3f}", flush=True)
    assert worst <= 1.0
