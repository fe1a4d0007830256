"""The sizes at which gemm_e4m3_block is tested in every output mode reach each of its kernels (the library's own
rule is asked; no compute call is made here)."""
import ctypes
import os

import pytest

from block_modes import MODES
from test_block_choice import LIB, TILES


def test_every_kernel_in_every_mode():
    if not os.path.exists(LIB):
        pytest.skip("libql.so not built")
    kernel = ctypes.CDLL(LIB).ql_gemm_e4m3_block_kernel
    kernel.argtypes = [ctypes.c_int64] * 3
    seen = {k: [] for k in range(len(TILES))}
    for s in MODES:
        seen[kernel(*s)].append(s)
    for k, sizes in seen.items():
        rows, cols = TILES[k]
        assert any(n % cols == 0 for _, n, _ in sizes) and any(n % 2 for _, n, _ in sizes), (k, sizes)
        assert any(m % rows for m, _, _ in sizes) and any(kk % 128 for _, _, kk in sizes), (k, sizes)
    for k in (0, 1, 4, 5, 6, 8, 10):   # a block of K alone
        assert any(kk <= 128 for _, _, kk in seen[k]), k
