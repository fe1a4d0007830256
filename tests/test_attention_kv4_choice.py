"""Which attention kernel the GPU tests' batches reach: those written for the prompt kernel, in either
of its shapes, and for the decode kernel go there."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "int8_quantized_linear_amd", "libql.so")
DECODE, ONE, TWO = 0, 1, 2


@pytest.fixture(scope="module")
def kernel():
    if not os.path.exists(LIB):
        pytest.skip("libql.so not built")
    f = ctypes.CDLL(LIB).ql_attention_kv4_kernel
    f.argtypes = [ctypes.c_int64] + [ctypes.c_int] * 7
    f.restype = ctypes.c_int

    def choice(H, R, D, rows, max_q, max_len, window=0):
        return f(sum(rows), H * R, H, D, len(rows), max_q, max_len, window)

    return choice


@pytest.mark.parametrize("H,R,D,rows,max_q,max_len,window,want", [
    # test_gpu_attention_kv4_prompt.py
    (128, 4, 64, (64, 50, 1), 64, 500, 0, ONE), (128, 4, 128, (64, 50, 1), 64, 500, 0, TWO),
    (128, 4, 256, (64, 50, 1), 64, 500, 0, ONE), (64, 4, 128, (64, 41), 64, 500, 0, ONE),
    *[(128, 4, 128, (64, 64), 64, 450, w, TWO) for w in (1, 63, 64, 200, 5000)],
    (64, 7, 128, (36, 30, 1, 20), 36, 400, 0, TWO), (128, 4, 128, (64, 64), 64, 300, 0, TWO),
    (64, 4, 128, (64, 64), 64, 500, 0, ONE), (128, 4, 128, (64, 64), 64, 500, 0, TWO),
    (128, 4, 64, (64, 64), 64, 500, 0, ONE), (128, 4, 256, (64, 64), 64, 500, 0, ONE),
    # test_gpu_attention_kv4_range.py, _small_q, _scale, _large_scores
    (64, 4, 128, (64, 64), 64, 300, 0, ONE), (128, 4, 128, (64, 64), 64, 300, 0, TWO),
    *[(128, 4, D, (64, 64), 64, 300, 0, TWO if D == 128 else ONE) for D in (64, 128, 256)],
    (256, 4, 64, (64,), 64, 304, 0, ONE),
    # test_gpu_attention_kv4_longest.py, _starts, _weights
    (256, 4, 64, (64,), 64, 300, 90, ONE), (256, 4, 64, (64, 0), 64, 300, 0, ONE), (256, 4, 64, (64,), 64, 300, 0, ONE),
])
def test_prompts(kernel, H, R, D, rows, max_q, max_len, window, want):
    assert kernel(H, R, D, rows, max_q, max_len, window) == want


@pytest.mark.parametrize("D", [64, 128, 256])
def test_few_rows(kernel, D):
    for H, R, rows, max_len in ((2, 4, (1,) * 11, 272), (2, 3, (5, 9, 8, 17, 0), 320), (1, 4, (1,), 70016), (32, 1, (1, 1), 160),
                                (2, 2, (8, 3), 208), (1, 71, (3, 2), 160), (8, 4, (1,) * 64, 16384)):
        assert kernel(H, R, D, rows, max(1, max(rows)), max_len) == DECODE
