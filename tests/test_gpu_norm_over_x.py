"""The residual of the norm written over x itself: the same bits as into a tensor of its own, for rows
kept in registers and rows read twice."""
import numpy as np
import pytest
import torch

from gpu_util import dev
from test_gpu_norm import _inputs, ql  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("t", [np.float16, np.float32])
@pytest.mark.parametrize("M,K", [(1, 16), (9, 4096), (300, 11008), (7, 20480)])
def test_over_x(ql, M, K, t, e4m3):  # noqa: F811
    x, res, gamma = (dev(a) for a in _inputs(M + K, M, K, t, t))
    call = ql.rms_norm_quantize_e4m3 if e4m3 else ql.rms_norm_quantize_int8
    want = call(x, gamma, res)
    got = call(x, gamma, res, res_out=x)
    assert got[2] is x
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
