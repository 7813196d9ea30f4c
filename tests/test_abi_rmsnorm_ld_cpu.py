"""Refusals of the gradient of the RMS norm with rows of h spaced apart, on the
host before any HIP call (the addresses are never used)."""

import os

import pytest

P = [1 << (24 + i) for i in range(9)]           # distinct, aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    from nvfp4_block_scaled_04_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from nvfp4_block_scaled_04_amd import build
        build.build(verbose=False)
    return binding.lib()


def _bwd(**kw):
    a = dict(dy=P[0], dh=P[1], h=P[2], ld_h=72, rstd=P[3], w=P[4], wide=1, rows=8, cols=64, dx=P[5], dw=P[6], ws=P[7],
             wsb=1 << 20, stream=None)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(ld_h=56), -2), (dict(ld_h=0), -2), (dict(ld_h=-72), -2), (dict(ld_h=68), -2), (dict(ld_h=1 << 40), -2),
    (dict(ld_h=(1 << 40) - 8, rows=(1 << 31) - 1), -2), (dict(rows=0, ld_h=56), -2), (dict(cols=72, ld_h=64), -2),
    (dict(dx=P[2]), -1), (dict(dx=P[2] + 128), -1),       # between the rows of h
    (dict(dx=P[2] + 2 * (7 * 72 + 64) - 16), -1), (dict(dw=P[2] + 2 * (7 * 72 + 64) - 4), -1), (dict(ws=P[2] + 1024), -1),
    (dict(h=None), -1), (dict(h=P[2] + 8), -1), (dict(w=None), -1), (dict(ws=None), -3),
])
def test_rmsnorm_bwd_ld_rejects(L, kw, status):
    assert L.nvfp4_rmsnorm_bwd_ld(*_bwd(**kw)) == status
    assert L.nvfp4_last_error() != b""


def test_rmsnorm_bwd_ld_of_no_rows(L):
    assert L.nvfp4_rmsnorm_bwd_ld(*_bwd(rows=0, dw=None, dy=None, h=None, w=None, rstd=None, dx=None, ws=None)) == 0


@pytest.mark.parametrize("kw", [dict(dw=P[4]), dict(dw=P[4] + 128), dict(ws=P[4]), dict(dw=P[7] + 16)])
def test_rmsnorm_bwd_of_no_rows_keeps_its_weight(L, kw):
    """dw of no rows is written, so it may not lie over w or the workspace either."""
    a = dict(rows=0, dy=None, dh=None, h=None, rstd=None, dx=None)
    a.update(kw)
    assert L.nvfp4_rmsnorm_bwd_ld(*_bwd(**a)) == -1
    a["ld_h"] = 64
    b = _bwd(**a)
    assert L.nvfp4_rmsnorm_bwd(*b[:3], *b[4:]) == -1
