"""Test-only choice of the integer product's kernel: the testing library's fgt_force_int8 puts this
thread's calls inside a ``with`` block on one compiled tile, the two-shape dense kernel or the
run-following contiguous one, with at most `grid` workgroups where these walk their tiles; "... columns" is the weight-streaming kernel, on
blocks of 16 `grid` rows (0: of all rows up to 128)."""
import contextlib
import ctypes

import moe_grouped_gemm_02_amd as fg
from fgtesting import testing_lib

TILES = {"256x256": 0, "256x128": 1, "128x256": 2, "128x128": 3, "64x128": 4, "128x160": 5,
         "split": 6, "runs": 7, "16 columns": 8, "32 columns": 9, "64 columns": 10}


@contextlib.contextmanager
def forced_int8(kernel, grid=0):
    L = testing_lib()
    L.fgt_force_int8.argtypes = [ctypes.c_int, ctypes.c_int]
    L.fgt_force_int8.restype = ctypes.c_int
    saved = fg.lib()
    assert L.fgt_force_int8(TILES[kernel], grid) == 0
    fg._lib = L
    try:
        yield
    finally:
        fg._lib = saved
        L.fgt_force_int8(-1, 0)
