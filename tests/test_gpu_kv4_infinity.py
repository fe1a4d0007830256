"""Infinite rows in kv4_append: the scale and low saturate as the definition says, bit for bit, and
the finite values of other groups and tokens are untouched."""
import numpy as np
import pytest

from gpu_util import host
from test_gpu_kv4 import DG, _append, _case, _expected, ql  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("D,G", DG)
def test_infinities(ql, D, G, dtype):  # noqa: F811
    """One and several +inf, -inf, both in one group, a group of nothing else; single rows and runs."""
    for lens, rows in (([12, 30], [12, 9]), ([5, 9, 1], [1, 1, 1])):
        b, cache, k, v = _case(D + G, lens, rows, 16, 2, D, G, dtype)
        inf = np.array(np.inf, dtype)
        k[0, 0, 5], v[0, 1, D - 1] = inf, -inf
        k[1, :, ::7], v[1, :, 3::5] = -inf, inf
        k[2, :, 1], k[2, :, 2], v[2, :, :G], v[2, 0, -1] = inf, -inf, inf, -inf
        if b.total > 4:
            k[3], v[3] = -inf, inf
            v[4, :, ::2] = np.array(65504, dtype)
        with np.errstate(invalid="ignore", over="ignore"):
            want = _expected(cache, b, D, G, k, v)
        assert np.array_equal(host(_append(ql, cache, b, G, k, v)), want)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("D,G", DG)
def test_nan_is_not_kept(ql, D, G, dtype):  # noqa: F811
    """Single NaN, groups of nothing else, and NaN beside infinities: what is stored for them is finite,
    and every other group's bytes are the definition's."""
    b, cache, k, v = _case(D * G, [12], [12], 16, 2, D, G, dtype)
    clean = _expected(cache, b, D, G, k, v)
    k[0, 0, 3], v[1, 1, ::2] = np.nan, np.nan
    k[2, 0, :G], v[3, :, :G] = np.nan, np.nan
    k[4, 0, 1], k[4, 0, 2], v[5, 1, 0], v[5, 1, 1] = np.nan, np.inf, -np.inf, np.nan
    got = host(_append(ql, cache, b, G, k, v))
    hit = {0: np.isnan(k.astype(np.float64)).reshape(12, 2, -1, G).any(-1),
           1: np.isnan(v.astype(np.float64)).reshape(12, 2, -1, G).any(-1)}
    P = 16
    for which in (0, 1):
        at = P * D // 2 * (1 + which) + which * 4 * P * (D // G)
        par, ref_par = (c[b.table[0, 0], :, at:at + 4 * P * (D // G)].copy().view(np.float16).reshape(2, D // G, 2, P)
                        for c in (got, clean))
        par, ref_par = par[..., :12].transpose(3, 0, 1, 2), ref_par[..., :12].transpose(3, 0, 1, 2)
        assert np.isfinite(par).all()
        assert np.array_equal(par[~hit[which]], ref_par[~hit[which]])
