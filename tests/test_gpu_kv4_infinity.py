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
