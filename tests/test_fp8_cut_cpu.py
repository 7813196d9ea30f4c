"""The FP8 product's cut of an expert's rows into tiles, on the CPU: the
function the kernels use, called on the host.  Every row lies in exactly one
tile, up to the largest row count the entry point takes."""

import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def cut():
    from nvfp4_block_scaled_04_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from nvfp4_block_scaled_04_amd import build
        build.build(verbose=False)
    f = ctypes.CDLL(binding.LIB_PATH).nvfp4_internal_fp8_cut
    f.restype = ctypes.c_int
    f.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                  ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int)]

    def call(M, lo, hi, bm, i):
        row0, nrows = ctypes.c_int64(), ctypes.c_int()
        n = f(M, lo, hi, bm, i, ctypes.byref(row0), ctypes.byref(nrows))
        return n, row0.value, nrows.value
    return call


HEIGHTS = [16, 32, 64, 96, 128, 160, 192, 224, 256, 288]


@pytest.mark.parametrize("bm", HEIGHTS)
@pytest.mark.parametrize("lo,rows", [(0, 1), (3, 15), (0, 16), (7, 17), (0, 64), (1, 272), (0, 300), (5, 577), (0, 4593)])
def test_tiles_partition_the_rows(cut, bm, lo, rows):
    n, at = -(-rows // bm), lo
    for i in range(n):
        count, row0, size = cut(lo + rows + 4, lo, lo + rows, bm, i)
        assert count == n and row0 == at and 0 < size <= bm
        at += size
    assert at == lo + rows
    assert cut(lo + rows + 4, lo, lo + rows, bm, n)[2] == 0       # none behind the last


@pytest.mark.parametrize("bm", HEIGHTS)
@pytest.mark.parametrize("lo,hi", [(0, (1 << 31) - 1), (0, (1 << 31) - 100), (0, (1 << 31) - 287), (0, (1 << 31) - 288),
                                   (5, (1 << 31) - 1), ((1 << 30) + 3, (1 << 31) - 1)])
def test_tiles_of_the_largest_calls(cut, bm, lo, hi):
    n = -(-(hi - lo) // bm)
    for i in [0, 1, 2, n // 3, n // 2, n - 3, n - 2, n - 1]:
        count, row0, size = cut(hi, lo, hi, bm, i)
        assert count == n and 0 < size <= bm and lo <= row0 and row0 + size <= hi, (i, count, row0, size)
        if i + 1 < n:
            assert cut(hi, lo, hi, bm, i + 1)[1] == row0 + size
    assert cut(hi, lo, hi, bm, 0)[1] == lo and sum(cut(hi, lo, hi, bm, n - 1)[1:]) == hi
