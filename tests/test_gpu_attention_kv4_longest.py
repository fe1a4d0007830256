"""The 4-bit cache and attention at the longest lengths that a table can hold, close to 2^31 positions:
sums of positions, stretches and blocks pass 31 bits there. Few pages serve all of a sequence, so the
results are known from theirs."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_util import dev, host
from test_gpu_attention_kv4 import U, _cache, ql  # noqa: F401

pytestmark = pytest.mark.gpu

H, D, G = 1, 64, 64


def _setup(seed, P, pages, H=1):
    rng = np.random.default_rng(seed)
    b = ref.Batch(rng, [pages * P], [1], P, spare=0, extra_width=0)
    return rng, _cache(rng, b, H, D, G)


def _table(P, width, last):
    """Page 0 throughout, then the pages `last` at the sequence's end."""
    t = torch.zeros((1, width), dtype=torch.int32, device="cuda:0")
    t[0, width - len(last):] = torch.tensor(last, dtype=torch.int32, device="cuda:0")
    return t


def _tol(o, mag, top, far, vmax):
    d = 2 * (D + 8) * 2.0 ** -24 * top + 2.0 ** -20
    return U * np.abs(o) + (3 * U + 2 * d) * mag + far * 2.0 ** -25 * vmax


@pytest.mark.parametrize("rows", [1, 3])
def test_every_position_counts(ql, rows):  # noqa: F811
    """Split over the whole length. The last 2048 of 2^19 - 1 pages have half of the weight: they are
    what the last of 256 splits holds. Each of a wave's 2^16 steps rounds its running sums once, of values and of weights."""
    P, width, many = 4096, (1 << 19) - 1, 2048
    n = P * width
    rng, cache = _setup(1, P, 2)
    par = cache[:, :, P * D // 2:P * D // 2 + 4 * P].copy().view(np.float16).reshape(2, 1, 1, 2, P)
    par[..., 0, :] *= np.float16(0.05)           # K: little but a low, which tells the pages apart
    par[0, ..., 1, :], par[1, ..., 1, :] = 0, 0.6875
    cache[:, :, P * D // 2:P * D // 2 + 4 * P] = par.reshape(2, 1, -1).view(np.uint8)
    k, v = zip(*(ref.read_rows(cache, [p], P, D, G, P) for p in (0, 1)))
    q = (1 + 0.1 * rng.standard_normal((rows, 1, D))).astype(np.float16)
    got = host(ql.attention_kv4(dev(q), dev(cache), _table(P, width, [1] * many), dev(np.array([n], np.int32)),
                                dev(np.array([0, rows], np.int32)), page_size=P, group=G))
    for i in range(rows):
        m = P - rows + i + 1                     # of the last page
        w = [np.exp(k[p][:, 0] @ q[i, 0].astype(np.float64) * D ** -0.5) for p in (0, 1)]
        w = [w[0] * (width - many), w[1] * (many - 1 + (np.arange(P) < m))]
        total = w[0].sum() + w[1].sum()
        assert 0.3 < w[1].sum() / total < 0.7
        o = (w[0] @ v[0][:, 0] + w[1] @ v[1][:, 0]) / total
        mag = (w[0] @ np.abs(v[0][:, 0]) + w[1] @ np.abs(v[1][:, 0])) / total
        top = D ** -0.5 * max((np.abs(k[p][:, 0]) @ np.abs(q[i, 0].astype(np.float64))).max() for p in (0, 1))
        assert np.all(np.abs(got[i, 0] - o) <= _tol(o, mag, top, 0, 0) + 2.0 ** -8 * mag), i


@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("rows", [1, 40])
def test_windows_at_the_end(ql, P, rows):  # noqa: F811
    """Written, read back and attended over at the last positions, through a window."""
    width = (1 << 31) // P - 1
    n, pages, window = P * width, 160 // P, 90
    rng, cache = _setup(2 + P, P, pages + 1)
    table, lens = _table(P, width, list(range(1, pages + 1))), dev(np.array([n], np.int32))
    starts = dev(np.array([0, rows], np.int32))
    d = dev(cache)
    new = [dev(rng.standard_normal((rows, H, D)).astype(np.float16)) for _ in range(2)]
    ql.kv4_append(*new, d, table, lens, starts, page_size=P, group=G)
    m = (pages + 1) * P                          # the sequence's last positions, page 0 the first of them
    k, v = ref.read_rows(host(d), list(range(pages + 1)), P, D, G, m)
    want = cache.copy()
    for i in range(rows):
        at = m - rows + i
        ref.write_token(want[at // P, 0], P, D, G, at % P, host(new[0])[i, 0], host(new[1])[i, 0])
    assert np.array_equal(host(d), want)
    for g, w in zip(ql.kv4_read(d, table, lens, starts, rows, D, P, G, torch.float32), (k, v)):
        assert np.array_equal(host(g), w[m - rows:].astype(np.float32))
    q = rng.standard_normal((rows, 2, D)).astype(np.float16)
    got = host(ql.attention_kv4(dev(q), d, table, lens, starts, page_size=P, group=G, window=window))
    o, mag, top = ref.attention64(q, k, v, m, D ** -0.5, window)
    assert np.all(np.abs(got - o) <= _tol(o, mag, top[..., None], window, np.abs(v).max()))


def test_a_prompt_at_the_end(ql):  # noqa: F811
    """The prompt kernel on the last 64 rows, through a window, and with the longest window there is."""
    P, rows, heads, window, pages = 64, 64, 256, 90, 3
    width = (1 << 31) // P - 1
    n = P * width
    rng, cache = _setup(9, P, pages + 1, heads)
    table, lens = _table(P, width, [1, 2, 3]), dev(np.array([n], np.int32))
    starts, d = dev(np.array([0, rows], np.int32)), dev(cache)
    q = rng.standard_normal((rows, heads * 4, D)).astype(np.float16)
    got = host(ql.attention_kv4(dev(q), d, table, lens, starts, page_size=P, group=G, window=window, max_q=rows,
                                max_len=300))
    k, v = ref.read_rows(cache, [1, 2, 3], P, D, G, pages * P)
    for i in (0, 1, 31, 63):
        m = pages * P - rows + i + 1
        o, mag, top = ref.attention64(q[i:i + 1, :8], k[:m, :2], v[:m, :2], m, D ** -0.5, window)
        assert np.all(np.abs(got[i, :8] - o[0]) <= _tol(o[0], mag[0], top[0][:, None], window, np.abs(v).max()))
    short = dev(np.array([70], np.int32))
    near = torch.tensor([[1, 2]], dtype=torch.int32, device="cuda:0")
    call = lambda w: ql.attention_kv4(dev(q), d, near, short, starts, page_size=P, group=G, window=w, max_q=rows,  # noqa: E731
                                      max_len=300)
    assert torch.equal(call((1 << 31) - 2), call(0))
