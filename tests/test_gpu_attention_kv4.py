"""attention_kv4 against the plain implementation in 64 bits over the same cache.

Tolerance, elementwise. With u = 2^-11 (half a unit of fp16's last place, relative): the weights
and the values enter the matrix cores as fp16, so each product is off by at most 2 u of its
magnitude, the output's rounding adds u |o|, and the sum of the weights is of what was rounded or
of the fp32 weights, u again. A score is off by at most (D + 8) roundings of fp32 of the products'
magnitudes, at most top = max_j sum_d |q_d k_jd| scale, and so is a weight, relatively, by 2 e with
e = (D + 8) 2^-24 top: weights p_j (1 + d_j), |d_j| <= 2 e + 2^-20 (the exponential), moves o by at
most twice that of sum_j p_j |v_j|. Weights below fp16's normal range are off by 2^-25 of the
largest instead, at most n 2^-25 max|v| over n positions.
"""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_util import Guarded, dev, host

pytestmark = pytest.mark.gpu

DG = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]
U = 2.0 ** -11


@pytest.fixture(scope="module")
def ql():
    import int8_quantized_linear_amd as ql

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return ql


def _cache(rng, b, H, D, G):
    """A cache whose every token is a normal value's codes; scales and lows of its own draw."""
    P, pages = b.P, b.pages
    cache = rng.integers(0, 256, (pages, H, ref.page_bytes(P, D, G)), dtype=np.uint8)
    n = P * (D // G)
    for which in range(2):
        at = P * D // 2 * (1 + which) + which * 4 * n
        par = np.empty((pages, H, D // G, 2, P), np.float16)
        par[..., 0, :] = rng.uniform(0.1, 0.4, (pages, H, D // G, P))
        par[..., 1, :] = -7.5 * par[..., 0, :] + rng.standard_normal((pages, H, D // G, P)) * 0.3
        cache[:, :, at:at + 4 * n] = par.reshape(pages, H, -1).view(np.uint8)
    return cache


def _poison(cache, b, D, G, window=0):
    """NaN and infinite scales and lows at every position that no row sees."""
    P = b.P
    seen = np.zeros((b.pages, P), bool)
    for s, (n, m) in enumerate(zip(b.lens, b.rows)):
        first = max(0, n - m - window + 1) if window else 0
        for pos in range(first, n):
            seen[b.table[s, pos // P], pos % P] = True
    for which in range(2):
        at = P * D // 2 * (1 + which) + which * 4 * P * (D // G)
        par = cache[:, :, at:at + 4 * P * (D // G)].copy().view(np.float16).reshape(b.pages, -1, D // G, 2, P)
        hide = np.broadcast_to(~seen[:, None, None, None, :], par.shape)
        par[hide] = np.resize(np.array([np.nan, np.inf, -np.inf, np.nan, 65504], np.float16), int(hide.sum()))
        cache[:, :, at:at + 4 * P * (D // G)] = par.reshape(b.pages, par.shape[1], -1).view(np.uint8)


def _check(ql, seed, lens, rows, P, H, R, D, G, window=0, scale=None, gain=1.0, max_q=None, max_len=None, poison=True,
           samples=None):
    rng = np.random.default_rng(seed)
    b = ref.Batch(rng, lens, rows, P)
    cache = _cache(rng, b, H, D, G)
    if poison:
        _poison(cache, b, D, G, window)
    q = (gain * rng.standard_normal((b.total, H * R, D))).astype(np.float16)
    out = Guarded((b.total, H * R, D), torch.float16)
    ql.attention_kv4(dev(q), dev(cache), *(dev(a) for a in b.arrays()), page_size=P, group=G, scale=scale,
                     window=window, max_q=max_q, max_len=max_len, out=out.view)
    torch.cuda.synchronize()
    out.check()
    got = host(out.view).astype(np.float64)
    assert np.isfinite(got).all()
    sc = D ** -0.5 if scale is None else scale
    for s, (n, m) in enumerate(zip(b.lens, b.rows)):
        n = max(n, 0)
        k, v = ref.read_rows(cache, b.table[s], P, D, G, n)
        a, e = b.starts[s], b.starts[s + 1]
        pick = np.arange(m) if samples is None else np.unique(rng.integers(0, m, samples))
        for i in pick:
            length = n - m + i + 1                 # this row alone: the last of its own positions
            if length <= 0:
                assert not got[a + i].any()
                continue
            o, mag, top = ref.attention64(q[a + i:a + i + 1], k[:length], v[:length], length, sc, window)
            d = 2 * (D + 8) * 2.0 ** -24 * top[0][:, None] + 2.0 ** -20
            far = min(length, window) if window else length
            vmax = np.abs(v[length - far:length]).max()
            tol = U * np.abs(o[0]) + (3 * U + 2 * d) * mag[0] + far * 2.0 ** -25 * vmax
            off = np.abs(got[a + i] - o[0])
            assert np.all(off <= tol), "sequence %d row %d: %.3g of %.3g" % (s, i, off.max(), tol[off > tol].min())


@pytest.mark.parametrize("D,G", DG)
def test_one_token(ql, D, G):
    """Single tokens over lengths around the tiles' and the pages' ends, and idle slots."""
    _check(ql, D + G, [1, 2, 15, 16, 17, 31, 33, 64, 100, 0, 257], [1] * 11, 16, 2, 4, D, G)


@pytest.mark.parametrize("H,R", [(1, 1), (32, 1), (2, 3), (1, 7), (2, 8), (1, 16), (1, 17), (1, 71)])
def test_head_layouts(ql, H, R):
    _check(ql, H + R, [77, 130], [1, 1], 32, H, R, 128, 64)
    _check(ql, H + R, [77, 130], [3, 2], 32, H, R, 64, 32)


@pytest.mark.parametrize("P", [16, 32, 64, 1024])
@pytest.mark.parametrize("D,G", [(64, 64), (128, 32), (256, 128)])
def test_pages(ql, P, D, G):
    _check(ql, P, [5, 300, P, 2 * P + 1, P - 1], [1, 2, 1, 4, 3], P, 2, 2, D, G)


@pytest.mark.parametrize("D,G", DG)
def test_several_rows(ql, D, G):
    """Rows of one sequence see one position more each; more rows than positions; no rows."""
    _check(ql, D * G, [40, 9, 5, 300, 12], [5, 9, 8, 17, 0], 16, 2, 3, D, G)


@pytest.mark.parametrize("D,G", DG)
def test_prompt(ql, D, G):
    """Prompts from position 0 and after a prefix, with ends inside tiles."""
    _check(ql, D - G, [150, 333, 1], [150, 129, 1], 64, 2, 2, D, G)


@pytest.mark.parametrize("window", [1, 2, 31, 32, 100, 5000])
@pytest.mark.parametrize("rows", [1, 6, 90])
def test_window(ql, rows, window):
    """Only the last `window` positions of each row; pages before the first row's window hold
    NaN scales."""
    _check(ql, rows + window, [400, 200, 95], [rows] * 3, 16, 2, 2, 128, 64, window=window)


def test_long(ql):
    """One sequence split over the whole chip, and a ragged pair beside it."""
    _check(ql, 1, [70001], [1], 64, 1, 4, 128, 64, poison=True)
    _check(ql, 2, [20000, 3, 129], [1, 1, 1], 16, 2, 8, 64, 32)
    _check(ql, 3, [9000, 50], [4, 2], 128, 1, 2, 256, 64)


def test_long_prompt(ql):
    _check(ql, 4, [3000], [1000], 64, 1, 4, 128, 64, samples=12)
    _check(ql, 5, [1100, 700], [1100, 650], 16, 2, 1, 128, 128, samples=12)


@pytest.mark.parametrize("max_q,max_len", [(1, 1), (1, 10 ** 6), (500, 1), (64, 300)])
def test_wrong_hints(ql, max_q, max_len):
    """max_q and max_len shape the launch only: any values give the rows' results."""
    _check(ql, 6, [300, 41], [37, 2], 32, 2, 4, 128, 64, max_q=max_q, max_len=max_len)
    _check(ql, 7, [1300, 41], [1, 1], 32, 2, 4, 128, 64, max_q=max_q, max_len=max_len)


@pytest.mark.parametrize("gain,scale", [(40.0, None), (1e-4, None), (1.0, 3.0), (1.0, -0.2), (0.0, None)])
def test_scores(ql, gain, scale):
    """Scores that make one weight 1 and the rest 0, equal weights, a negative scale."""
    _check(ql, 8, [500, 33, 210], [1, 2, 40], 32, 2, 4, 128, 64, gain=gain, scale=scale)


def test_rising_scores(ql):
    """Scores that rise along the sequence, so that the running maximum moves at every step."""
    P, D, G, n = 32, 64, 64, 640
    rng = np.random.default_rng(2)
    b = ref.Batch(rng, [n], [1], P)
    cache = np.zeros((b.pages, 1, ref.page_bytes(P, D, G)), np.uint8)
    k = np.zeros((n, 1, D), np.float32)
    k[:, 0, 0] = np.arange(n) * 0.5
    v = rng.standard_normal((n, 1, D)).astype(np.float32)
    for i in range(n):
        ref.write_token(cache[b.table[0, i // P], 0], P, D, G, i % P, k[i, 0], v[i, 0])
    q = np.zeros((1, 1, D), np.float16)
    for lead in (1.0, -1.0, 0.05):
        q[0, 0, 0] = lead
        got = host(ql.attention_kv4(dev(q), dev(cache), *(dev(a) for a in b.arrays()), page_size=P, group=G, scale=1.0))
        kk, vv = ref.read_rows(cache, b.table[0], P, D, G, n)
        o, mag, top = ref.attention64(q, kk, vv, n, 1.0, 0)
        d = 2 * (D + 8) * 2.0 ** -24 * top[..., None] + 2.0 ** -20
        assert np.all(np.abs(got - o) <= U * np.abs(o) + (3 * U + 2 * d) * mag + n * 2.0 ** -25 * np.abs(vv).max())


def test_small_and_large_values(ql):
    """V of 1e-4 and of thousands: the weights' fp16 does not depend on V's size."""
    for gain in (2e-4, 3000.0):
        P, D, G, n = 16, 128, 64, 90
        rng = np.random.default_rng(3)
        b = ref.Batch(rng, [n], [1], P)
        cache = np.zeros((b.pages, 1, ref.page_bytes(P, D, G)), np.uint8)
        k = rng.standard_normal((n, D)).astype(np.float32)
        v = (gain * rng.standard_normal((n, D))).astype(np.float32)
        for i in range(n):
            ref.write_token(cache[b.table[0, i // P], 0], P, D, G, i % P, k[i], v[i])
        q = rng.standard_normal((1, 2, D)).astype(np.float16)
        got = host(ql.attention_kv4(dev(q), dev(cache), *(dev(a) for a in b.arrays()), page_size=P, group=G))
        kk, vv = ref.read_rows(cache, b.table[0], P, D, G, n)
        o, mag, top = ref.attention64(q, kk, vv, n, D ** -0.5, 0)
        # fp16 values below 2^-14 are off by up to 2^-25 where larger ones are off by U relatively
        tol = U * np.abs(o) + (3 * U + 2.0 ** -15) * mag + n * 2.0 ** -25 * np.abs(vv).max() + 2 * 2.0 ** -25
        assert np.all(np.abs(got - o) <= tol), gain


def test_strided_rows(ql):
    """q as a slice of a wider projection."""
    rng = np.random.default_rng(5)
    P, H, R, D, G = 16, 2, 2, 128, 64
    b = ref.Batch(rng, [50, 20], [3, 1], P)
    cache, meta = dev(_cache(rng, b, H, D, G)), [dev(a) for a in b.arrays()]
    wide = dev(rng.standard_normal((b.total, 8, D)).astype(np.float16))
    a = ql.attention_kv4(wide[:, :4], cache, *meta, page_size=P, group=G)
    c = ql.attention_kv4(wide[:, :4].contiguous(), cache, *meta, page_size=P, group=G)
    assert torch.equal(a, c)


def test_repeats_bit_for_bit(ql):
    rng = np.random.default_rng(6)
    P, H, R, D, G = 16, 4, 4, 128, 64
    for lens, rows in (([3000, 700, 0, 45], [1, 1, 1, 1]), ([900, 333], [300, 20])):
        b = ref.Batch(rng, lens, rows, P)
        cache, meta = dev(_cache(rng, b, H, D, G)), [dev(a) for a in b.arrays()]
        q = dev(rng.standard_normal((b.total, H * R, D)).astype(np.float16))
        first = ql.attention_kv4(q, cache, *meta, page_size=P, group=G)
        for _ in range(10):
            assert torch.equal(ql.attention_kv4(q, cache, *meta, page_size=P, group=G), first)


def test_page_numbers_outside_the_cache(ql):
    """Page numbers outside the cache and lengths past the table lead to no access outside."""
    rng = np.random.default_rng(7)
    b = ref.Batch(rng, [40, 40], [1, 20], 16)
    b.table[:] = np.array([2 ** 31 - 1, -1, b.pages, -2 ** 31])[None, :b.table.shape[1]]
    b.lens = [10 ** 9, -5]
    cache, q = dev(_cache(rng, b, 2, 64, 64)), dev(rng.standard_normal((21, 4, 64)).astype(np.float16))
    out = ql.attention_kv4(q, cache, *(dev(a) for a in b.arrays()), page_size=16, group=64)
    assert not host(out)[1:].any()


def test_refusals(ql):
    rng = np.random.default_rng(8)
    b = ref.Batch(rng, [20], [4], 16)
    c, t, n, s = dev(_cache(rng, b, 2, 128, 64)), *(dev(a) for a in b.arrays())
    q = torch.zeros((4, 4, 128), dtype=torch.float16, device="cuda:0")
    f, ok = ql.attention_kv4, dict(page_size=16, group=64)
    for bad in (q[0], q[:, :3], q[:, :, :64], q.cpu(), torch.zeros((4, 4, 256), dtype=torch.float16, device="cuda:0")[:, :, ::2]):
        with pytest.raises(ValueError):
            f(bad, c, t, n, s, **ok)
    with pytest.raises(TypeError):
        f(q.float(), c, t, n, s, **ok)
    with pytest.raises(TypeError):
        f(q, c, t, n.long(), s, **ok)
    with pytest.raises(ValueError):
        f(q, c, t, n, s, page_size=16, group=128)
    with pytest.raises(ValueError):
        f(q, c, t, n, s, out=q[:2], **ok)
    for kw in (dict(window=-1), dict(scale=float("nan")), dict(max_q=0), dict(max_len=0)):
        with pytest.raises(ql.QLError):
            f(q, c, t, n, s, **ok, **kw)
    assert f(q[:0], c, t, n, torch.zeros_like(s), **ok).shape == (0, 4, 128)
