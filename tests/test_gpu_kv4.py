"""kv4_append and kv4_read against the plain implementation: the whole cache byte for byte after
a write (places that no row writes keep their bytes), and the rows read back bit for bit (a value
is one fused multiply-add of exact numbers, rounded to the output)."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_util import Guarded, dev, host

pytestmark = pytest.mark.gpu

DG = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]


@pytest.fixture(scope="module")
def ql():
    import int8_quantized_linear_amd as ql

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return ql


def _rows(rng, n, H, D, dtype):
    x = rng.standard_normal((n, H, D), dtype=np.float32)
    x[..., 3::29] *= 4
    return x.astype(dtype)


def _expected(cache, b, D, G, k, v):
    want = cache.copy()
    for s, (n, m) in enumerate(zip(b.lens, b.rows)):
        for i in range(m):
            pos = min(max(n, 0), b.width * b.P) - m + i
            if pos >= 0:
                for h in range(cache.shape[1]):
                    ref.write_token(want[b.table[s, pos // b.P], h], b.P, D, G, pos % b.P,
                                    k[b.starts[s] + i, h], v[b.starts[s] + i, h])
    return want


def _append(ql, cache, b, G, k, v):
    d = dev(cache)
    ql.kv4_append(dev(k), dev(v), d, *(dev(a) for a in b.arrays()), page_size=b.P, group=G)
    return d


def _case(seed, lens, rows, P, H, D, G, dtype):
    rng = np.random.default_rng(seed)
    b = ref.Batch(rng, lens, rows, P)
    cache = rng.integers(0, 256, (b.pages, H, ref.page_bytes(P, D, G)), dtype=np.uint8)
    return b, cache, _rows(rng, b.total, H, D, dtype), _rows(rng, b.total, H, D, dtype)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("D,G", DG)
def test_write_and_read(ql, D, G, dtype):
    """One row, several rows over pages that start and end inside a run of 8, a whole prompt from
    position 0, a sequence without rows, and one of length 0 with a row that has no position."""
    b, cache, k, v = _case(D + G, [1, 45, 19, 30, 0, 64], [1, 7, 19, 0, 1, 33], 16, 3, D, G, dtype)
    got = _append(ql, cache, b, G, k, v)
    want = _expected(cache, b, D, G, k, v)
    assert np.array_equal(host(got), want)
    # everything back, in both types
    back = ref.Batch(np.random.default_rng(0), b.lens, b.lens, b.P)
    back.table = np.ascontiguousarray(b.table)
    ks, vs = zip(*(ref.read_rows(want, b.table[s], b.P, D, G, n) for s, n in enumerate(b.lens)))
    written = np.concatenate([np.arange(n) >= n - m for n, m in zip(b.lens, b.rows)])
    for out in (torch.float16, torch.float32):
        gk, gv = ql.kv4_read(got, *(dev(a) for a in (b.table, np.array(b.lens, np.int32), back.starts)), back.total, D,
                             b.P, G, out)
        for g, w in ((gk, np.concatenate(ks)), (gv, np.concatenate(vs))):
            w32 = w[written].astype(np.float32)
            with np.errstate(over="ignore"):
                assert np.array_equal(host(g)[written], w32.astype(np.float16) if out == torch.float16 else w32)


@pytest.mark.parametrize("P", [16, 32, 128, 1024])
@pytest.mark.parametrize("H", [1, 8])
def test_page_sizes(ql, P, H):
    b, cache, k, v = _case(P + H, [3, 2 * P, P + 5], [3, 9, P // 2 + 3], P, H, 128, 64, np.float16)
    assert np.array_equal(host(_append(ql, cache, b, 64, k, v)), _expected(cache, b, 128, 64, k, v))


def test_rows_without_position(ql):
    """More rows than the length (the first have no position), a negative length, and a length
    past what the table holds: nothing but the rows' own places changes, and such rows read 0."""
    b, cache, k, v = _case(1, [5, 4, 3], [5, 7, 2], 16, 2, 64, 32, np.float16)
    b.lens[2] = -9
    got = _append(ql, cache, b, 32, k, v)
    assert np.array_equal(host(got), _expected(cache, b, 64, 32, k, v))
    gk, gv = ql.kv4_read(got, *(dev(a) for a in b.arrays()), b.total, 64, 16, 32)
    for g in (gk, gv):
        assert not host(g)[5:8].any() and not host(g)[12:].any()
        assert host(g)[:5].any() and host(g)[8:12].any()
    b, cache, k, v = _case(2, [32, 8], [3, 1], 16, 1, 64, 64, np.float16)
    b.table, b.width = np.ascontiguousarray(b.table[:, :2]), 2
    b.lens[0] = 1000                                  # taken as 2 pages of 16
    assert np.array_equal(host(_append(ql, cache, b, 64, k, v)), _expected(cache, b, 64, 64, k, v))


def test_values(ql):
    """Constant rows, zeros, the largest and smallest fp16 numbers, both signs, and fp32 values
    past fp16's range (the scale and low saturate)."""
    H, D, G = 2, 128, 32
    b, cache, k, v = _case(4, [12], [12], 16, H, D, G, np.float32)
    k[0], v[0] = 0, -0.0
    k[1], v[1] = 1.5, -2.25
    k[2], v[2] = 65504, -65504
    k[3, :, ::2], v[3, :, ::2] = 65504, -65504
    k[4], v[4] = 6e-8, -6e-8
    k[5, :, ::3] = 1e-7
    k[6], v[6] = k[6] * 1e6, v[6] * 1e30
    k[7, 0, 5] = 3e38
    v[8] = np.abs(v[8]) + 100
    for dtype in (np.float32, np.float16):
        with np.errstate(over="ignore"):
            kk, vv = (np.clip(x, -65504, 65504).astype(dtype) if dtype == np.float16 else x for x in (k, v))
        assert np.array_equal(host(_append(ql, cache, b, G, kk, vv)), _expected(cache, b, D, G, kk, vv))


def test_slices_of_a_projection(ql):
    """k and v as slices of one [rows, (q + 2 kv) heads, D] projection, read through their strides."""
    b, cache, k, v = _case(6, [40, 7], [11, 7], 32, 2, 128, 64, np.float16)
    wide = np.zeros((b.total, 7, 128), np.float16)
    wide[:, 3:5], wide[:, 5:7] = k, v
    w, d = dev(wide), dev(cache)
    ql.kv4_append(w[:, 3:5], w[:, 5:7], d, *(dev(a) for a in b.arrays()), page_size=32, group=64)
    assert np.array_equal(host(d), _expected(cache, b, 128, 64, k, v))


def test_pages_past_4_gib(ql):
    """Pages whose bytes lie beyond 2^32 from the cache's start."""
    P, H, D, G = 1024, 8, 256, 64
    per = ref.page_bytes(P, D, G) * H
    pages = (1 << 32) // per + 3
    d = torch.zeros((pages, H, ref.page_bytes(P, D, G)), dtype=torch.uint8, device="cuda:0")
    rng = np.random.default_rng(9)
    k, v = _rows(rng, 5, H, D, np.float16), _rows(rng, 5, H, D, np.float16)
    table = np.array([[pages - 1, 0]], np.int32)
    meta = [dev(a) for a in (table, np.array([5], np.int32), np.array([0, 5], np.int32))]
    ql.kv4_append(dev(k), dev(v), d, *meta, page_size=P, group=G)
    blk = np.zeros((1, H, ref.page_bytes(P, D, G)), np.uint8)
    for i in range(5):
        for h in range(H):
            ref.write_token(blk[0, h], P, D, G, i, k[i, h], v[i, h])
    assert np.array_equal(host(d[-1]), blk[0])
    assert not d[:-1].any()
    gk, gv = ql.kv4_read(d, *meta, 5, D, P, G)
    wk, wv = ref.read_rows(blk, [0], P, D, G, 5)
    assert np.array_equal(host(gk), wk.astype(np.float32).astype(np.float16))
    assert np.array_equal(host(gv), wv.astype(np.float32).astype(np.float16))


def test_page_numbers_outside_the_cache(ql):
    """A page number outside the cache does not lead outside its array."""
    n = 3 * 2 * ref.page_bytes(16, 64, 64)
    buf = torch.full((n + 2 * 65536,), 77, dtype=torch.uint8, device="cuda:0")
    cache = buf[65536:65536 + n].view(3, 2, -1)
    k = dev(np.ones((2, 2, 64), np.float16))
    for bad in (3, -1, 2 ** 31 - 1):
        meta = [dev(a) for a in (np.array([[bad], [bad]], np.int32), np.array([1, 16], np.int32),
                                 np.array([0, 1, 2], np.int32))]
        ql.kv4_append(k, k, cache, *meta, page_size=16, group=64)
        ql.kv4_read(cache, *meta, 2, 64, 16, 64)
    torch.cuda.synchronize()
    assert bool((buf[:65536] == 77).all()) and bool((buf[65536 + n:] == 77).all())


def test_refusals(ql):
    b, cache, k, v = _case(7, [20], [4], 16, 2, 128, 64, np.float16)
    c, k, v, t, n, s = dev(cache), dev(k), dev(v), *(dev(a) for a in b.arrays())
    ok = dict(page_size=16, group=64)
    for bad in ((k[0], v, c, t, n, s), (k, v[:3], c, t, n, s), (k[:, :1], v, c, t, n, s), (k, v, c[:, :, :-16], t, n, s),
                (k, v, c, t[0], n, s), (k, v, c, t, n[:0], s), (k, v, c, t, n, s[:1]), (k.cpu(), v, c, t, n, s),
                (k.transpose(0, 1).contiguous().transpose(0, 1)[:, :, ::2], v, c, t, n, s)):
        with pytest.raises(ValueError):
            ql.kv4_append(*bad, **ok)
    for bad in ((k.bfloat16(), v.bfloat16(), c, t, n, s), (k, v.float(), c, t, n, s), (k, v, c.view(torch.int8), t, n, s),
                (k, v, c, t.long(), n, s)):
        with pytest.raises(TypeError):
            ql.kv4_append(*bad, **ok)
    with pytest.raises(ValueError):
        ql.kv4_append(k, v, c, t, n, s, page_size=32, group=64)
    with pytest.raises(ValueError):
        ql.kv4_append(k, v, c, t, n, s, page_size=16, group=48)
    with pytest.raises(TypeError):
        ql.kv4_read(c, t, n, s, 4, 128, 16, 64, torch.bfloat16)
    odd = torch.zeros((2, 1, ref.page_bytes(24, 128, 64)), dtype=torch.uint8, device="cuda:0")
    with pytest.raises(ql.QLError):
        ql.kv4_append(k[:, :1], v[:, :1], odd, t, n, s, page_size=24, group=64)
    wide = torch.zeros((4, 2 * 128 + 4), dtype=torch.float16, device="cuda:0")[:, :256].unflatten(1, (2, 128))
    with pytest.raises(ql.QLError):
        ql.kv4_append(wide, v, c, t, n, s, **ok)     # rows not 16-byte aligned
    ql.kv4_append(k[:0], v[:0], c, t, n, torch.zeros_like(s), **ok)
    assert torch.equal(c, dev(cache))
