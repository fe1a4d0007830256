"""The entry points with a scale for each block of 128 refuse bad arguments with the documented
status codes before any HIP call (no compute call is made here)."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "int8_quantized_linear_amd", "libql.so")
OK, NULL, SHAPE, ALIGN, DTYPE = 0, 1, 2, 3, 4
F32, F16 = 0, 1
A, MIS = 0x10000, 0x10001   # fake addresses: never dereferenced on error paths


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.skip("libql.so not built")
    L = ctypes.CDLL(LIB)
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.quantize_per_row_block_e4m3.argtypes = [P, I, I64, I64, P, P, P]
    L.quantize_weight_block_e4m3.argtypes = [P, I64, I64, I64, P, P, P]
    L.gemm_e4m3_block.argtypes = [P, P, P, P, P, I, P, I, I64, I64, I64, P]
    return L


def test_quantize_rows(lib):
    def f(x=A, dt=F16, M=4, K=64, q=A, s=A):
        return lib.quantize_per_row_block_e4m3(x, dt, M, K, q, s, None)

    for kw in (dict(x=None), dict(q=None), dict(s=None)):
        assert f(**kw) == NULL
    for kw in (dict(x=MIS), dict(x=A + 8), dict(q=A + 8), dict(s=A + 2)):
        assert f(**kw) == ALIGN
    for kw in (dict(M=-1), dict(K=0), dict(K=-16), dict(K=24), dict(M=1 << 31), dict(K=1 << 31), dict(M=1 << 30, K=256)):
        assert f(**kw) == SHAPE, kw
    assert f(dt=2) == DTYPE
    assert f(M=0, x=None, q=None, s=None) == OK


def test_quantize_weight(lib):
    def f(w=A, E=2, K=64, N=40, q=A, s=A):
        return lib.quantize_weight_block_e4m3(w, E, K, N, q, s, None)

    for kw in (dict(w=None), dict(q=None), dict(s=None)):
        assert f(**kw) == NULL
    for kw in (dict(w=MIS), dict(q=A + 8), dict(s=A + 2)):
        assert f(**kw) == ALIGN
    for kw in (dict(E=-1), dict(E=(1 << 20) + 1), dict(K=0), dict(K=24), dict(N=-1), dict(N=1 << 31)):
        assert f(**kw) == SHAPE, kw
    assert f(E=0, w=None) == OK and f(N=0, w=None) == OK


def test_gemm(lib):
    def f(x=A, xs=A, w=A, ws=A, bias=None, act=0, y=A, dt=F16, M=4, N=200, K=256):
        return lib.gemm_e4m3_block(x, xs, w, ws, bias, act, y, dt, M, N, K, None)

    for kw in (dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(y=None)):
        assert f(**kw) == NULL
    for kw in (dict(x=A + 8), dict(w=MIS), dict(y=A + 8), dict(xs=A + 2), dict(ws=A + 1), dict(bias=A + 3)):
        assert f(**kw) == ALIGN
    for kw in (dict(M=-1), dict(N=-1), dict(K=0), dict(K=32), dict(K=200), dict(K=131072), dict(N=(1 << 23) + 1),
               dict(M=1 << 31)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(dt=2), dict(act=3), dict(act=-1)):
        assert f(**kw) == DTYPE
    assert f(M=0, x=None) == OK and f(N=0, w=None) == OK
