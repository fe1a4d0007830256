"""Which kernel gemm_e4m3_block takes for the sizes of the GPU tests: every one is reached, at full and at
ragged tiles (the library's own rule is asked; no compute call is made here)."""
import ctypes
import os

import pytest

from block_shapes import LARGE, SHAPES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "int8_quantized_linear_amd", "libql.so")
# rows and columns of a workgroup of each kernel, the last but one a mix of the two before
TILES = [(16, 16), (16, 32), (32, 16), (32, 32), (32, 64), (64, 32), (128, 128), (128, 192), (256, 192), (256, 192),
         (64, 64)]


@pytest.fixture(scope="module")
def kernel():
    if not os.path.exists(LIB):
        pytest.skip("libql.so not built")
    f = ctypes.CDLL(LIB).ql_gemm_e4m3_block_kernel
    f.argtypes = [ctypes.c_int64] * 3
    return f


def test_every_kernel_is_reached(kernel):
    seen = {}
    for M, N, K in SHAPES + LARGE:
        k = kernel(M, N, K)
        r, c = TILES[k]
        seen.setdefault(k, set()).add((M % r != 0, N % c != 0, K % 128 != 0))
    assert sorted(seen) == list(range(len(TILES)))
    for k, kinds in seen.items():
        assert any(a for a, _, _ in kinds) and any(b for _, b, _ in kinds) and any(c for _, _, c in kinds), (k, kinds)


def test_largest_sizes(kernel):
    for s in ((1, 1, 64), ((1 << 31) - 1, 1, 64), (1, 1 << 23, 64), (2 ** 14, 1 << 23, 131008), ((1 << 31) - 1, 64, 64)):
        assert 0 <= kernel(*s) < len(TILES)


def test_grids_stay_below_2_to_32_threads(kernel):
    """At the most rows, with as many columns as 288 GB hold beside them: few-row kernels split their rows over launches."""
    for M in (1 << 30, (1 << 30) - 77, 1 << 28, 1 << 24):
        for K in (64, 128, 4096):
            for N in (1, 48, 64, 130, 700, 1 << 23):
                if M * K + M * N * 2 + N * K > 288 << 30:
                    continue
                k = kernel(M, N, K)
                r, c = TILES[k]
                threads = 256 if k == len(TILES) - 1 else 512
                assert k < 6 or -(-M // r) * -(-N // c) * threads < 1 << 32, (M, N, K, k)
