"""Refusals of the RMS norm and of the expert layer for a few tokens on the CPU:
every bad call is turned down on the host before any HIP call (the addresses
are never used)."""

import os

import pytest

P = [1 << (24 + i) for i in range(14)]          # distinct, aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    from nvfp4_block_scaled_04_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from nvfp4_block_scaled_04_amd import build
        build.build(verbose=False)
    return binding.lib()


def _norm(**kw):
    a = dict(x=P[0], ld_x=64, res=P[1], ld_r=64, w=P[2], wide=0, rows=8, cols=64, eps=1e-6, h=P[3], y=P[4], q=P[5],
             sf=P[6], rstd=P[7], stream=None)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), -2), (dict(rows=1 << 31), -2), (dict(cols=0, ld_x=64), -2), (dict(cols=12), -2),
    (dict(cols=32776, ld_x=32776, ld_r=32776), -2), (dict(cols=24), -2),              # FP8 of 24 columns
    (dict(ld_x=56), -2), (dict(ld_r=60), -2), (dict(ld_x=68), -2), (dict(ld_x=1 << 40), -2),
    (dict(rows=(1 << 31) - 1, ld_r=(1 << 40) - 8), -2),
    (dict(eps=0.0), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(eps=9e-31), -1),
    (dict(wide=2), -1), (dict(x=None), -1), (dict(w=None), -1), (dict(y=None, q=None, sf=None), -1),
    (dict(sf=None), -1), (dict(q=None), -1), (dict(h=None), -1), (dict(res=None), -1),
    (dict(x=P[0] + 8), -1), (dict(res=P[1] + 2), -1), (dict(w=P[2] + 4), -1), (dict(h=P[3] + 8), -1),
    (dict(y=P[4] + 8), -1), (dict(q=P[5] + 4), -1), (dict(sf=P[6] + 2), -1), (dict(rstd=P[7] + 1), -1),
    (dict(y=P[0]), -1), (dict(y=P[1] + 16), -1), (dict(h=P[0] + 16), -1), (dict(h=P[1] + 128), -1),
    (dict(h=P[1], ld_r=72), -1), (dict(h=P[0], ld_x=72), -1),                         # in place, rows apart
    (dict(q=P[2]), -1), (dict(sf=P[5] + 8), -1), (dict(rstd=P[3] + 4), -1), (dict(y=P[3]), -1), (dict(rstd=P[2]), -1),
])
def test_rmsnorm_rejects(L, kw, status):
    assert L.nvfp4_rmsnorm(*_norm(**kw)) == status
    assert L.nvfp4_last_error() != b""


def test_rmsnorm_of_no_rows(L):
    assert L.nvfp4_rmsnorm(*_norm(rows=0, x=None, res=None, w=None, h=None, y=None, q=None, sf=None, rstd=None)) == 0


def _bwd(**kw):
    a = dict(dy=P[0], dh=P[1], h=P[2], rstd=P[3], w=P[4], wide=1, rows=8, cols=64, dx=P[5], dw=P[6], ws=P[7],
             wsb=1 << 20, stream=None)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), -2), (dict(rows=1 << 31), -2), (dict(cols=4), -2), (dict(cols=32776), -2), (dict(wide=-1), -1),
    (dict(dy=None), -1), (dict(h=None), -1), (dict(rstd=None), -1), (dict(w=None), -1), (dict(dx=None), -1),
    (dict(rows=0, w=None), -1),                           # dw of no rows is written all the same
    (dict(ws=None), -3), (dict(wsb=64), -3), (dict(ws=P[7] + 8), -3), (dict(rows=0, ws=None), -3),
    (dict(dy=P[0] + 8), -1), (dict(dh=P[1] + 8), -1), (dict(h=P[2] + 8), -1), (dict(w=P[4] + 8), -1),
    (dict(dx=P[5] + 8), -1), (dict(rstd=P[3] + 2), -1), (dict(dw=P[6] + 2), -1),
    (dict(dx=P[0] + 16), -1), (dict(dx=P[1] + 16), -1), (dict(dx=P[2]), -1), (dict(dx=P[4]), -1), (dict(dw=P[4]), -1),
    (dict(dw=P[5]), -1), (dict(ws=P[0]), -1), (dict(ws=P[5] + 64), -1), (dict(ws=P[6]), -1), (dict(dw=P[3]), -1),
    (dict(dx=P[0], dw=P[0]), -1), (dict(dx=P[0], ws=P[0]), -1),
])
def test_rmsnorm_bwd_rejects(L, kw, status):
    assert L.nvfp4_rmsnorm_bwd(*_bwd(**kw)) == status
    assert L.nvfp4_last_error() != b""


def test_rmsnorm_bwd_workspace(L):
    f = L.nvfp4_rmsnorm_bwd_workspace_size
    assert f(-1, 64) == 0 and f(4, 0) == 0 and f(4, 32776) == 0
    assert f(0, 64) >= 4 * 64 and f(8192, 7168) >= 4 * 7168
    assert L.nvfp4_rmsnorm_bwd(*_bwd(rows=0, dw=None, dy=None, h=None, w=None, rstd=None, dx=None, ws=None)) == 0


def _few(fp8, **kw):
    a = dict(x=P[0], T=4, H=256, I=128, E=4, k=2, ids=P[1], w=P[2], w1=P[3], s1=P[4], g1=P[5], w2=P[6], s2=P[7], g2=P[8],
             out=P[9], ws=P[10], wsb=1 << 20, stream=None)
    a.update(kw)
    if fp8:
        del a["g1"], a["g2"]
    return tuple(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -2), (dict(T=17), -2), (dict(H=0), -2), (dict(I=0), -2), (dict(H=120), -2), (dict(I=72), -2),
    (dict(H=1 << 20), -2), (dict(I=1 << 20), -2), (dict(H=1 << 16, I=1 << 14), -2), (dict(E=0), -2), (dict(E=4097), -2),
    (dict(k=0), -2), (dict(k=65), -2),
    (dict(x=None), -1), (dict(ids=None), -1), (dict(w=None), -1), (dict(w1=None), -1), (dict(s1=None), -1),
    (dict(w2=None), -1), (dict(s2=None), -1), (dict(out=None), -1),
    (dict(x=P[0] + 8), -1), (dict(w1=P[3] + 8), -1), (dict(w2=P[6] + 8), -1), (dict(s1=P[4] + 2), -1),
    (dict(s2=P[7] + 2), -1), (dict(out=P[9] + 8), -1), (dict(ids=P[1] + 2), -1), (dict(w=P[2] + 1), -1),
    (dict(ws=None), -3), (dict(ws=P[10] + 8), -3), (dict(wsb=4 * 4 * 2 * 128 - 1), -3),
    (dict(out=P[0] + 64), -1), (dict(out=P[1]), -1), (dict(out=P[3] + 16), -1), (dict(out=P[7]), -1), (dict(ws=P[9]), -1),
    (dict(ws=P[6]), -1), (dict(ws=P[0]), -1), (dict(ws=P[2]), -1),
])
@pytest.mark.parametrize("fp8", [False, True])
def test_few_rejects(L, fp8, kw, status):
    f = L.moe_expert_forward_few_fp8 if fp8 else L.moe_expert_forward_few
    assert f(*_few(fp8, **kw)) == status
    assert L.nvfp4_last_error() != b""


def test_few_rejects_by_format(L):
    assert L.moe_expert_forward_few(*_few(False, H=144)) == -2          # NVFP4: multiples of 128
    assert L.moe_expert_forward_few(*_few(False, I=144)) == -2
    assert L.moe_expert_forward_few(*_few(False, g1=None)) == -1
    assert L.moe_expert_forward_few(*_few(False, g2=None)) == -1
    assert L.moe_expert_forward_few(*_few(False, s1=P[4] + 4)) == -1
    assert L.moe_expert_forward_few(*_few(False, g2=P[9])) == -1        # under out


def test_few_of_no_tokens_and_workspace(L):
    for fp8, f in ((False, L.moe_expert_forward_few), (True, L.moe_expert_forward_few_fp8)):
        assert f(*_few(fp8, T=0, x=None, ids=None, w=None, w1=None, s1=None, w2=None, s2=None, out=None, ws=None)) == 0
    f = L.moe_expert_forward_few_workspace_size
    assert f(0, 128, 2) == 0 and f(17, 128, 2) == 0 and f(1, 0, 2) == 0 and f(1, 128, 0) == 0
    assert f(16, 2048, 8) >= 16 * 8 * 2048 * 4


def test_binding_refuses_on_the_host():
    """Shapes and types are refused by the Python layer before any call."""
    import torch

    import nvfp4_block_scaled_04_amd as nv
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    w = torch.zeros((64,))
    with pytest.raises(ValueError, match="device"):
        nv.rmsnorm(x, w)
    with pytest.raises(TypeError):
        nv.fp8_rmsnorm(None, w)
    with pytest.raises(ValueError, match="device"):
        nv.rmsnorm_bwd(x, x, w, w)
    with pytest.raises(ValueError, match="device"):
        nv.moe_expert_forward_few_fp8(x, None, None, torch.zeros((1, 32, 64)).to(torch.float8_e4m3fn), w, x, w)
