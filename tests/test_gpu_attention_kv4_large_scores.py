"""attention_kv4 with scores far past 2^24, where neighbouring fp32 numbers lie 2 and more apart:
finite outputs, the largest score's value, and zeros for rows without a position."""
import numpy as np
import pytest

import kv4_ref as ref
from gpu_util import dev, host
from test_gpu_attention_kv4 import U, _cache, _check, ql  # noqa: F401

pytestmark = pytest.mark.gpu

SCALES = [1e5, -1e7, 1e8, 1e10, -1e20, 1e34]


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("D,G", [(64, 32), (128, 64), (256, 128)])
def test_decode(ql, D, G, scale):  # noqa: F811
    _check(ql, D, [5, 300, 12, 0], [8, 6, 17, 2], 16, 2, 3, D, G, scale=scale)
    _check(ql, D, [700, 0, 3], [1, 1, 1], 16, 2, 3, D, G, scale=scale)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("H,D,G", [(128, 64, 32), (128, 128, 64), (64, 128, 64), (128, 256, 128)])
def test_prompt(ql, H, D, G, scale):  # noqa: F811
    _check(ql, D, [300, 20], [64, 64], 64, H, 4, D, G, scale=scale, max_q=64, max_len=300, samples=6)


@pytest.mark.parametrize("scale", [1e8, -1e8, 1e12, 1e32, -1e32])
@pytest.mark.parametrize("rows,H", [(4, 1), (64, 256)])
def test_scores_of_one_sign(ql, rows, H, scale):  # noqa: F811
    """Scores around 10 to 20 times the scale, all positive or all negative (q along K's mean direction): the largest has
    all the weight wherever the next one is further away than fp32's roundings of it."""
    P, D, G, n, R = 16, 64, 32, 300, 4
    rng = np.random.default_rng(7)
    b = ref.Batch(rng, [n], [rows], P)
    cache = _cache(rng, b, H, D, G)
    n_par = P * (D // G)
    par = cache[:, :, :4 * n_par + P * D // 2][:, :, P * D // 2:].copy().view(np.float16).reshape(b.pages, H, D // G, 2, P)
    par[..., 1, :] += np.float16(8)              # K around 8
    cache[:, :, P * D // 2:P * D // 2 + 4 * n_par] = par.reshape(b.pages, H, -1).view(np.uint8)
    k, v = ref.read_rows(cache, b.table[0], P, D, G, n)
    q = np.abs(rng.standard_normal((rows, H * R, D))).astype(np.float16)
    got = host(ql.attention_kv4(dev(q), dev(cache), *(dev(a) for a in b.arrays()), page_size=P, group=G, scale=scale))
    assert np.isfinite(got).all()
    sure = 0
    for i in range(0, rows, max(1, rows // 4)):
        for h in range(min(H * R, 6)):
            s = k[:n - rows + i + 1, h // R] @ q[i, h].astype(np.float64) * scale
            assert np.all(s * scale > 0)
            first, second = np.sort(s)[::-1][:2]
            if first - second > 1e-4 * np.abs(s).max():
                sure += 1
                want = v[np.argmax(s), h // R]
                assert np.all(np.abs(got[i, h] - want) <= 2 * U * np.abs(want) + 2.0 ** -24)
    assert sure
