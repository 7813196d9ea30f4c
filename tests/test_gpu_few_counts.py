"""Counts that a C int cannot hold are refused, not cut to their low bits."""

import pytest
import torch

import nvfp4_block_scaled_04_amd as nv

BIG = (1 << 32) + 2


def test_few_workspace_refuses_a_k_beyond_32_bits():
    with pytest.raises(ValueError):
        nv.few_workspace(1, 128, BIG, "cpu")


@pytest.mark.gpu
def test_few_refuses_a_k_beyond_32_bits():
    dev = "cuda:0"
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=dev)
    ids, w = torch.empty((0, BIG), dtype=torch.int32, device=dev), torch.empty((0, BIG), device=dev)
    w1, w2 = torch.zeros((2, 64, 64), device=dev).to(torch.float8_e4m3fn), torch.zeros((2, 64, 32), device=dev).to(torch.float8_e4m3fn)
    one = torch.ones((2, 1, 1), device=dev)
    assert nv.moe_expert_forward_few_fp8(x, ids[:, :2], w[:, :2], w1, one, w2, one).shape == (0, 64)
    with pytest.raises(ValueError):
        nv.moe_expert_forward_few_fp8(x, ids, w, w1, one, w2, one)
