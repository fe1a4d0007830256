"""gemm_e4m3_block takes a few-row kernel for no more groups of rows than a grid has in y (the library's own rule is
asked; no compute call is made here)."""
import ctypes
import os
import random

import pytest

from test_block_choice import LIB, TILES


def test_few_row_kernels_stay_within_the_grid():
    if not os.path.exists(LIB):
        pytest.skip("libql.so not built")
    kernel = ctypes.CDLL(LIB).ql_gemm_e4m3_block_kernel
    kernel.argtypes = [ctypes.c_int64] * 3
    rng = random.Random(0)
    sizes = [(m, n, k) for m in (1 << 20, (1 << 20) + 1, 65535 * 16 + 1, 65535 * 32 + 1, 65535 * 64 + 1, (1 << 30) - 15, 1 << 30)
             for n in (*range(1, 34), 48, 64, 65, 128, 129, 192, 193, 256, 1000, 1 << 23) for k in (64, 128, 192, 4096, 65536, 131008)]
    sizes += [(65535 * 16 + int(2 ** rng.uniform(0, 29.9)), int(2 ** rng.uniform(0, 12)), 64 * int(2 ** rng.uniform(0, 11)))
              for _ in range(100000)]
    for s in sizes:
        k = kernel(*s)
        assert k >= 6 or -(-s[0] // TILES[k][0]) <= 65535, (s, k)
