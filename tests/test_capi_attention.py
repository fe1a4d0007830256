"""The norm, 4-bit cache and attention entry points refuse bad arguments with the documented
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
    P, I64, I, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    L.rms_norm_quantize_int8.argtypes = [P, I, P, I, P, F, I64, I64, P, P, P, P]
    L.rms_norm_quantize_e4m3.argtypes = [P, I, P, I, P, F, I64, I64, P, P, P, P]
    L.kv4_append.argtypes = [P, P, I, I64, I64, I64, P, I64, I64, I64, I64, I64, P, I64, P, P, I64, P]
    L.kv4_read.argtypes = [P, I64, I64, I64, I64, I64, P, I64, P, P, I64, I64, I, P, P, P]
    L.attention_kv4.argtypes = [P, I64, P, I64, I64, P, I64, I64, I64, I64, I64, P, I64, P, P, I64, I64, I64, F, I64,
                                P, I64, P]
    L.attention_kv4_workspace_bytes.argtypes = [I64, I64, I64, I64, I64, I64, I64, I64, ctypes.POINTER(I64)]
    return L


@pytest.mark.parametrize("name", ["rms_norm_quantize_int8", "rms_norm_quantize_e4m3"])
def test_norm(lib, name):
    def f(x=A, xt=F16, res=A, rt=F16, gamma=A, eps=1e-6, M=4, K=64, ro=A, q=A, s=A):
        return getattr(lib, name)(x, xt, res, rt, gamma, eps, M, K, ro, q, s, None)

    for kw in (dict(x=None), dict(gamma=None), dict(q=None), dict(s=None), dict(res=None), dict(ro=None)):
        assert f(**kw) == NULL
    for kw in (dict(x=MIS), dict(res=MIS), dict(gamma=A + 4), dict(ro=MIS), dict(q=MIS), dict(s=MIS)):
        assert f(**kw) == ALIGN
    for kw in (dict(M=-1), dict(K=0), dict(K=24), dict(M=1 << 31), dict(eps=0.0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf"))):
        assert f(**kw) == SHAPE
    assert f(xt=2) == DTYPE and f(rt=7) == DTYPE
    assert f(res=None, rt=7, ro=None, q=None) == NULL      # res_dtype is not looked at
    assert f(x=None, gamma=None, q=None, M=0) == OK


def _bad_cache(f):
    for kw in (dict(P=8), dict(P=24), dict(P=8192), dict(P=0), dict(H=0), dict(D=96), dict(D=512), dict(G=16),
               dict(G=0), dict(D=64, G=128), dict(rows=-1), dict(rows=(1 << 24) + 1), dict(pages=-1), dict(pages=0),
               dict(pages=1 << 31), dict(width=-1), dict(width=1 << 40), dict(width=1 << 27), dict(batch=0),
               dict(batch=-1), dict(batch=1 << 21), dict(H=4096, rows=1 << 20)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(cache=None), dict(table=None), dict(lens=None), dict(starts=None)):
        assert f(**kw) == NULL, kw
    for kw in (dict(cache=MIS), dict(table=MIS), dict(lens=MIS), dict(starts=MIS)):
        assert f(**kw) == ALIGN, kw
    assert f(rows=0, cache=None, lens=None, batch=0, pages=0) == OK


def test_append(lib):
    def f(k=A, v=A, dt=F16, ks=None, vs=None, rows=4, cache=A, pages=9, P=16, H=2, D=128, G=64, table=A, width=3,
          lens=A, starts=A, batch=2):
        return lib.kv4_append(k, v, dt, H * D if ks is None else ks, H * D if vs is None else vs, rows, cache, pages, P,
                              H, D, G, table, width, lens, starts, batch, None)

    _bad_cache(f)
    assert f(k=None) == NULL and f(v=None) == NULL
    assert f(dt=3) == DTYPE
    assert f(ks=255) == SHAPE and f(vs=0) == SHAPE and f(ks=1 << 31) == SHAPE
    assert f(k=MIS) == ALIGN and f(v=A + 8) == ALIGN
    assert f(ks=260) == ALIGN and f(vs=258, dt=F32) == ALIGN


def test_read(lib):
    def f(cache=A, pages=9, P=16, H=2, D=128, G=64, table=A, width=3, lens=A, starts=A, batch=2, rows=4, dt=F16, k=A,
          v=A):
        return lib.kv4_read(cache, pages, P, H, D, G, table, width, lens, starts, batch, rows, dt, k, v, None)

    _bad_cache(f)
    assert f(k=None) == NULL and f(v=None) == NULL
    assert f(dt=2) == DTYPE
    assert f(k=MIS) == ALIGN and f(v=A + 8) == ALIGN


def test_attention(lib):
    def need(**kw):
        n = ctypes.c_int64(-1)
        a = dict(rows=4, HQ=4, H=2, D=128, batch=2, max_q=3, max_len=40, window=0)
        a.update({k: v for k, v in kw.items() if k in a})
        st = lib.attention_kv4_workspace_bytes(a["rows"], a["HQ"], a["H"], a["D"], a["batch"], a["max_q"], a["max_len"],
                                               a["window"], ctypes.byref(n))
        return st, n.value

    def f(q=A, qs=None, out=A, rows=4, HQ=4, cache=A, pages=9, P=16, H=2, D=128, G=64, table=A, width=3, lens=A,
          starts=A, batch=2, max_q=3, max_len=40, scale=0.1, window=0, ws=A, wb=1 << 40):
        if HQ % max(H, 1):
            HQ = H
        return lib.attention_kv4(q, HQ * D if qs is None else qs, out, rows, HQ, cache, pages, P, H, D, G, table, width,
                                 lens, starts, batch, max_q, max_len, scale, window, ws, wb, None)

    _bad_cache(f)
    assert f(q=None) == NULL and f(out=None) == NULL and f(ws=None) == NULL
    assert f(q=A + 2) == ALIGN and f(out=A + 8) == ALIGN and f(ws=A + 4) == ALIGN and f(qs=516) == ALIGN
    assert f(qs=511) == SHAPE and f(max_q=0) == SHAPE and f(max_len=0) == SHAPE and f(window=-1) == SHAPE
    assert f(scale=float("nan")) == SHAPE and f(scale=float("inf")) == SHAPE and f(wb=-1) == SHAPE
    assert lib.attention_kv4(A, 512, A, 4, 3, A, 9, 16, 2, 128, 64, A, 3, A, A, 2, 1, 40, 0.1, 0, A, 1 << 40, None) == SHAPE
    st, n = need(rows=1, batch=1, max_q=1, max_len=1 << 17)
    assert st == OK and n >= 0 and n % 4 == 0
    if n:
        assert f(rows=1, batch=1, max_q=1, max_len=1 << 17, wb=n - 4) == SHAPE
    assert need(D=100)[0] == SHAPE and need(HQ=3)[0] == SHAPE and need(max_q=0)[0] == SHAPE and need(window=-1)[0] == SHAPE
    assert lib.attention_kv4_workspace_bytes(4, 4, 2, 128, 2, 3, 40, 0, None) == NULL
