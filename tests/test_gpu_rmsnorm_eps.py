"""RMS norm at the smallest eps: rows whose squares, times 2^-16, reach fp32's
subnormal numbers.

These are kept, each rounding 2^-150 off at most; that is 2^-134 in the mean for
each of a lane's sums, 2^-34 of an eps of 1e-30 (2^-99.7), far below the 40
roundings of 2^-24 that 1/rms is counted with otherwise."""

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_04_amd as nv
from oracle import norm as N
from parity import bf16_values, host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("size", [1e-20, 1e-17, 1e-16, 1e-15, 1e-14, 1e-10])
@pytest.mark.parametrize("T,H", [(5, 128), (3, 528), (4, 2048), (2, 7168), (1, 32768)])
def test_rmsnorm_smallest_eps(T, H, size):
    rng = np.random.default_rng(H)
    x = torch.from_numpy((size * rng.standard_normal((T, H))).astype(np.float32)).to(torch.bfloat16)
    w = torch.from_numpy(rng.uniform(0.5, 2, H).astype(np.float32))
    y, _, rstd = nv.rmsnorm(x.to("cuda:0"), w.to("cuda:0"), eps=1e-30, need_rstd=True)
    v, s = N.rmsnorm(x.float().numpy(), w.numpy(), float(np.float32(1e-30)))
    assert np.all(np.abs(host(rstd) - s) <= 40 * U * s)
    assert np.all(np.abs(bf16_values(host(y)) - v) <= (2.0 ** -8 + 41 * U) * np.abs(v) + 1e-38)
