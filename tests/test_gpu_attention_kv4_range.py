"""attention_kv4 over caches whose V passes fp16's range: scale * code + low of a stored pair goes up
to 15 * 65504 + 65504 = 1048064, from fp32 rows that large as well as from the rounding of the pair
for fp16 rows near 65504. A row has to match the 64-bit form whatever lies at positions that it
does not see and others of its tile do, and whatever it sees.

Tolerance: test_gpu_attention_kv4.py's, and 2^-20 more: V next to values that pass 65504 enters
divided by 16, where fp16 numbers lie 2^-24 apart at least; low / 16 and the value each round by half of that,
16 times in the output.
"""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_util import Guarded, dev, host
from test_gpu_attention_kv4 import DG, U, ql  # noqa: F401

pytestmark = pytest.mark.gpu


def _spike(kind, rng, shape):
    """One token's V [H, D]."""
    v = rng.standard_normal(shape).astype(np.float32)
    if kind == "top":
        v[:, ::3] = np.abs(v[:, ::3])
        v[:, 1::32] = 65504
        v[:, 2::32] = 0
        return np.maximum(v, 0)
    if kind == "both":
        v[:, 1::32], v[:, 2::32] = 65504, -65504
        return v
    if kind == "large":
        return v * 2.5e5                         # past fp16, within the stored pair
    v[:, 1::16] = 3e38                           # past the stored pair, which saturates
    return v


def _check(ql, seed, lens, rows, P, H, R, D, G, spikes, kind, window=0, samples=None, **hints):  # noqa: F811
    rng = np.random.default_rng(seed)
    full = ref.Batch(rng, lens, lens, P)
    k = rng.standard_normal((full.total, H, D)).astype(np.float32)
    v = rng.standard_normal((full.total, H, D)).astype(np.float32)
    for s, pos in spikes:
        v[full.starts[s] + pos] = _spike(kind, rng, (H, D))
    cache = torch.zeros((full.pages, H, ref.page_bytes(P, D, G)), dtype=torch.uint8, device="cuda:0")
    ql.kv4_append(dev(k), dev(v), cache, *(dev(a) for a in full.arrays()), page_size=P, group=G)
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    q = (0.1 * rng.standard_normal((starts[-1], H * R, D))).astype(np.float16)
    out = Guarded((int(starts[-1]), H * R, D), torch.float16)
    ql.attention_kv4(dev(q), cache, dev(full.table), dev(np.array(lens, np.int32)), dev(starts), page_size=P, group=G,
                     window=window, out=out.view, **hints)
    torch.cuda.synchronize()
    out.check()
    got, cache = host(out.view).astype(np.float64), host(cache)
    seen = hidden = 0
    for s, (n, m) in enumerate(zip(lens, rows)):
        kk, vv = ref.read_rows(cache, full.table[s], P, D, G, n)
        for i in range(m) if samples is None else np.unique(rng.integers(0, m, samples)):
            length = n - m + i + 1
            if length <= 0:
                assert not got[starts[s] + i].any()
                continue
            o, mag, top = ref.attention64(q[starts[s] + i][None], kk[:length], vv[:length], length, D ** -0.5, window)
            far = min(length, window) if window else length
            vmax = np.abs(vv[length - far:length]).max()
            d = 2 * (D + 8) * 2.0 ** -24 * top[0][:, None] + 2.0 ** -20
            tol = U * np.abs(o[0]) + (3 * U + 2 * d) * mag[0] + far * 2.0 ** -25 * vmax + 2.0 ** -20
            off = np.abs(got[starts[s] + i] - o[0])
            large = vmax > 60000
            seen, hidden = seen + large, hidden + (not large)
            assert np.abs(o).max() < 65504
            # comparisons with NaN are false
            assert np.all(off <= tol), "sequence %d row %d: %s of %d" % (s, i, np.sum(~(off <= tol)), off.size)
    return seen, hidden


KINDS = ["top", "both", "large", "past"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,G", DG)
def test_a_later_rows_value(ql, D, G, kind):  # noqa: F811
    """Drafted tokens: a value that only the tile's later rows see."""
    seen, hidden = _check(ql, D + G, [200, 90], [8, 3], 16, 2, 2, D, G, [(0, 196), (1, 89)], kind)
    assert seen and hidden


@pytest.mark.parametrize("kind", KINDS)
def test_a_value_left_of_the_window(ql, kind):  # noqa: F811
    """Rows whose window has passed the value beside rows that still see it."""
    seen, hidden = _check(ql, 3, [300], [6], 32, 2, 4, 128, 64, [(0, 300 - 6 - 97)], kind, window=100)
    assert seen and hidden


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,G", DG)
def test_a_later_rows_value_in_a_prompt(ql, D, G, kind):  # noqa: F811
    """The prompt kernel, in both of its shapes (D = 128 with 64 and 128 heads)."""
    for H in (64, 128) if D == 128 else (128,):
        seen, hidden = _check(ql, H + G, [300, 64], [64, 64], 64, H, 4, D, G,
                              [(0, 270), (1, 40), (1, 63)], kind, samples=4, max_q=64, max_len=300)
        assert seen or hidden


@pytest.mark.parametrize("kind", KINDS)
def test_a_value_in_one_wave_or_split(ql, kind):  # noqa: F811
    """Single tokens over lengths that several waves and splits share, one of which meets the value."""
    _check(ql, 5, [3000, 700, 130], [1, 1, 2], 16, 2, 4, 128, 64, [(0, 1500), (1, 2), (2, 129)], kind)
    _check(ql, 6, [20000], [1], 64, 1, 8, 64, 32, [(0, 19999)], kind)
