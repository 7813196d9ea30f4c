"""Refusals of the FP8 and gradient entry points on the CPU: every bad call is
turned down on the host before any HIP call (the addresses are never used)."""

import os

import pytest
import torch

FAKE = 1 << 20          # distinct, aligned, never dereferenced
P = [FAKE << i for i in range(10)]


@pytest.fixture(scope="module")
def L():
    from nvfp4_block_scaled_04_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from nvfp4_block_scaled_04_amd import build
        build.build(verbose=False)
    return binding.lib()


def _gemm(**kw):
    a = dict(a=P[0], asf=P[1], rows=64, src=None, div=1, off=P[2], E=4, M=64, N=64, K=128, b=P[3],
             bsf=P[4], c=P[5], stream=None)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(E=0), -2), (dict(E=4097), -2), (dict(M=-1), -2), (dict(M=1 << 31), -2),
    (dict(K=0), -2), (dict(K=24), -2), (dict(K=1 << 22), -2), (dict(N=0), -2),
    (dict(N=1 << 20, K=2048), -2),                                  # an expert's weight of 2^31
    (dict(rows=63), -2),                                            # fewer A rows than M
    (dict(rows=-1, M=0), -2),
    (dict(src=P[6], div=0), -2),
    (dict(src=P[6], rows=1 << 24, K=128), -2),                      # gathered A of 2 GiB
    (dict(off=None), -1),                                           # dense with four experts
    (dict(a=None), -1), (dict(asf=None), -1), (dict(b=None), -1), (dict(bsf=None), -1),
    (dict(c=None), -1), (dict(a=P[0] + 8), -1), (dict(b=P[3] + 4), -1), (dict(asf=P[1] + 2), -1),
    (dict(c=P[5] + 1), -1), (dict(off=P[2] + 2), -1), (dict(src=P[6] + 1), -1),
    (dict(c=P[0] + 64), -1), (dict(c=P[1]), -1), (dict(c=P[3] + 16), -1), (dict(c=P[4]), -1),   # c over an input
    (dict(src=P[6], c=P[6]), -1), (dict(c=P[2] + 2), -1),
    (dict(M=(1 << 31) - 1, rows=(1 << 31) - 1, N=1 << 20, K=16), -2),   # too many tiles
])
def test_fp8_grouped_gemm_rejects(L, kw, status):
    assert L.nvfp4_fp8_grouped_gemm(*_gemm(**kw)) == status
    assert L.nvfp4_last_error() != b""


@pytest.mark.parametrize("name,two", [("nvfp4_fp8_quantize", 1), ("nvfp4_fp8_swiglu_quantize", 2)])
def test_fp8_quantize_rejects(L, name, two):
    f = getattr(L, name)
    for args, status in [((P[0], -1, 16, 32, None, P[1], P[2]), -2),
                         ((P[0], 1, 8, 32, None, P[1], P[2]), -2),
                         ((P[0], 1, 0, 32, None, P[1], P[2]), -2),
                         ((P[0], 1, 40, 80, None, P[1], P[2]), -2),
                         ((P[0], 1, 1 << 24, 1 << 25, None, P[1], P[2]), -2),
                         ((P[0], 1, 32, 32 * two - 8, None, P[1], P[2]), -2),
                         ((P[0], 1, 32, 32 * two + 4, None, P[1], P[2]), -2),
                         ((P[0], 1 << 30, 256, 512, None, P[1], P[2]), -2),
                         ((None, 1, 32, 64, None, P[1], P[2]), -1),
                         ((P[0], 1, 32, 64, None, None, P[2]), -1),
                         ((P[0], 1, 32, 64, None, P[1], None), -1),
                         ((P[0] + 8, 1, 32, 64, None, P[1], P[2]), -1),
                         ((P[0], 1, 32, 64, None, P[1] + 4, P[2]), -1),
                         ((P[0], 1, 32, 64, None, P[1], P[2] + 2), -1),
                         ((P[0], 1, 32, 64, None, P[0] + 8, P[2]), -1),
                         ((P[0], 9, 32, 64, None, P[1], P[0] + 1024), -1),
                         ((P[0], 9, 32, 64, None, P[1], P[1] + 32), -1),
                         ((P[0], (1 << 31) - 1, 32, (1 << 40) - 8, None, P[1], P[2]), -2),
                         ((P[0], 1, 32, 64, P[1], P[1], P[2]), -1), ((P[0], 1, 32, 64, P[2], P[1], P[2]), -1),
                         ((P[0], 1, 32, 64, P[3] + 2, P[1], P[2]), -1)]:
        assert f(*args, None) == status, args
        assert L.nvfp4_last_error() != b""
    assert f(None, 0, 32, 64, None, None, None, None) == 0      # no rows: nothing to do


def test_fp8_quantize_weight_rejects(L):
    f = L.nvfp4_fp8_quantize_weight
    for args, status in [((P[0], -1, 4, 16, P[1], P[2]), -2), ((P[0], 1, -1, 16, P[1], P[2]), -2),
                         ((P[0], 1, 4, 8, P[1], P[2]), -2), ((P[0], 1, 4, 1 << 24, P[1], P[2]), -2),
                         ((P[0], 1 << 31, 1, 16, P[1], P[2]), -2), ((P[0], 1 << 30, 256, 128, P[1], P[2]), -2),
                         ((None, 1, 4, 16, P[1], P[2]), -1), ((P[0], 1, 4, 16, None, P[2]), -1),
                         ((P[0], 1, 4, 16, P[0] + 64, P[2]), -1), ((P[0], 1, 4, 16, P[1], P[1] + 8), -1),
                         ((P[0], 1, 4, 16, P[1], None), -1), ((P[0] + 2, 1, 4, 16, P[1], P[2]), -1)]:
        assert f(*args, None) == status, args
    assert f(None, 0, 4, 16, None, None, None) == 0 and f(None, 4, 0, 16, None, None, None) == 0


def test_dispatch_and_gradients_reject(L):
    for T, k, E, H in [(-1, 2, 4, 16), (4, 0, 4, 16), (4, 65, 4, 16), (4, 2, 0, 16), (4, 2, 4097, 16),
                       (4, 2, 4, 0), (4, 2, 4, 12), (4, 2, 4, 1 << 24), (1 << 30, 2, 4, 16), (1 << 62, 4, 4, 16)]:
        assert L.nvfp4_moe_dispatch(P[0], P[1], P[2], T, k, E, H, P[9], None) == -2
        assert L.nvfp4_moe_dispatch_bwd(P[9], P[1], P[2], T, k, E, H, P[0], None) == -2
        assert L.nvfp4_moe_combine_bwd(P[0], P[9], P[1], P[3], P[2], T, k, E, H, P[8], P[4], None) == -2
    good = (4, 2, 4, 16)
    for i in range(4):
        ptr = [P[0], P[1], P[2], P[9]]
        ptr[i] = None
        assert L.nvfp4_moe_dispatch(ptr[0], ptr[1], ptr[2], *good, ptr[3], None) == -1
        assert L.nvfp4_moe_dispatch_bwd(ptr[0], ptr[1], ptr[2], *good, ptr[3], None) == -1
    assert L.nvfp4_moe_dispatch(P[0] + 8, P[1], P[2], *good, P[9], None) == -1
    assert L.nvfp4_moe_dispatch(P[0], P[1], P[2], *good, P[0] + 112, None) == -1       # x is 128 bytes
    assert L.nvfp4_moe_dispatch(P[0], P[1], P[2], *good, P[0] - 16, None) == -1
    assert L.nvfp4_moe_dispatch_bwd(P[9], P[1], P[2], *good, P[9] + 16, None) == -1
    for bad in ((P[1] + 2, P[2]), (P[1], P[2] + 2), (P[9], P[2]), (P[1], P[9])):         # misaligned, or over an output
        assert L.nvfp4_moe_dispatch(P[0], *bad, *good, P[9], None) == -1
        assert L.nvfp4_moe_dispatch_bwd(P[0], *bad, *good, P[9], None) == -1
        assert L.nvfp4_moe_combine_bwd(P[0], P[8], bad[0], P[3], bad[1], *good, P[9], P[4], None) == -1
    assert L.nvfp4_moe_combine_bwd(P[0], P[8], P[4], P[3], P[2], *good, P[9], P[4], None) == -1
    assert L.nvfp4_moe_combine_bwd(P[0], P[8], P[1], P[3] + 2, P[2], *good, P[9], P[4], None) == -1
    for i in (0, 1, 2, 3, 4, 5):
        ptr = [P[0], P[9], P[1], P[3], P[2], P[8]]
        ptr[i] = None
        assert L.nvfp4_moe_combine_bwd(*ptr[:5], *good, ptr[5], P[4], None) == -1
    assert L.nvfp4_moe_combine_bwd(P[0], P[9], P[1], P[3], P[2], *good, P[9], P[4], None) == -1     # in place
    assert L.nvfp4_moe_combine_bwd(P[0], P[9], P[1], P[3], P[2], *good, P[8], P[3], None) == -1     # dw over w
    assert L.nvfp4_moe_combine_bwd(P[0], P[9], P[1], P[3], P[2], *good, P[8], P[4] + 2, None) == -1
    assert L.nvfp4_moe_dispatch(None, None, None, 0, 2, 4, 16, None, None) == 0


def test_router_bwd_rejects(L):
    f = L.nvfp4_router_topk_bwd
    for T, E, k in [(-1, 4, 1), (4, 0, 1), (4, 1025, 1), (4, 4, 0), (4, 4, 5), (4, 100, 65), (1 << 32, 4, 2)]:
        assert f(P[0], P[1], P[2], T, E, k, P[3], None) == -2
    for i in range(4):
        ptr = P[:4]
        ptr[i] = None
        assert f(*ptr[:3], 4, 4, 2, ptr[3], None) == -1
        ptr[i] = P[i] + 2
        assert f(*ptr[:3], 4, 4, 2, ptr[3], None) == -1
    assert f(P[0], P[1], P[2], 4, 4, 2, P[2], None) == -1       # dlogits over dw
    assert f(None, None, None, 0, 4, 2, None, None) == 0


def test_bindings_reject_host_tensors():
    import nvfp4_block_scaled_04_amd as nv
    bf, f32, i32 = torch.zeros((2, 16), dtype=torch.bfloat16), torch.zeros((2, 1)), torch.zeros(3, dtype=torch.int32)
    q = torch.zeros((2, 16), dtype=torch.float8_e4m3fn)
    for call in (lambda: nv.fp8_quantize(bf), lambda: nv.fp8_swiglu_quantize(bf),
                 lambda: nv.fp8_quantize_weight(bf[None]),
                 lambda: nv.fp8_grouped_gemm(q, f32, q[None], f32[None]),
                 lambda: nv.moe_dispatch(bf, i32, i32, 1), lambda: nv.moe_dispatch_bwd(bf, i32, i32, 1),
                 lambda: nv.moe_combine_bwd(bf, bf, i32, f32, i32),
                 lambda: nv.router_topk_bwd(i32[None], f32, f32, 4)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("v", [1 << 31, (1 << 32) + 1, -(1 << 31) - 1, (1 << 32) + 3])
def test_bindings_reject_counts_beyond_32_bits(v):
    """A count that C's int cannot hold is refused, not cut to its low bits
    (2^32 + 1 rows a source row would read as 1)."""
    import nvfp4_block_scaled_04_amd as nv
    bf, f32, i32 = torch.zeros((2, 16), dtype=torch.bfloat16), torch.zeros((2, 1)), torch.zeros(3, dtype=torch.int32)
    q = torch.zeros((2, 16), dtype=torch.float8_e4m3fn)
    for name, call in (("a_row_div", lambda: nv.fp8_grouped_gemm(q, f32, q[None], f32[None], a_row_src=i32, a_row_div=v)),
                       ("k", lambda: nv.moe_dispatch(bf, i32, i32, v)),
                       ("k", lambda: nv.moe_dispatch_bwd(bf, i32, i32, v)),
                       ("E", lambda: nv.router_topk_bwd(i32[None], f32, f32, v))):
        with pytest.raises(ValueError, match=f"{name} .* 32 bits"):
            call()
