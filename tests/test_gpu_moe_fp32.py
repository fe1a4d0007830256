"""fp32 outputs of the experts have fp32's precision: within the elementwise bound of three terms of h, and of a
relative norm that two terms would pass (test_moe_terms.py)."""
import numpy as np
import pytest
import torch

import block_ref as ref
from gpu_util import Guarded, dev, host
from moe_cases import NARROW, NORM, TOKEN_NORM, inputs, norm_errors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    import int8_quantized_linear_amd as ql

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return ql


def _check(got, inp, k, renorm):
    want, err = ref.moe64(*inp, k, renorm, h_error=2.0 ** -25)
    got = got.astype(np.float64)
    assert (np.abs(got - want) <= err * (1 + 2.0 ** -24) + 2.0 ** -24 * np.abs(want) + 1e-37).all()
    whole, row = norm_errors(got, want)
    assert whole < NORM and row < TOKEN_NORM, (whole, row)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,K,I", NARROW)
def test_few_tokens_an_expert(ql, T, E, k, K, I, renorm):
    inp = inputs(T, E, K, I)
    out = Guarded((T, K), torch.float32)
    ql.moe_e4m3_block(*map(dev, inp), k, renorm, torch.float32, out.view)
    out.check()
    _check(host(out.view), inp, k, renorm)


@pytest.mark.parametrize("T,E,k,K,I", [(33, 3, 2, 2048, 8256), (64, 6, 2, 1984, 4160), (20, 2, 1, 4096, 12416),
                                       (64, 65, 16, 2112, 512)])
def test_many_tokens_an_expert(ql, T, E, k, K, I):
    assert T * k >= 8 * E and E * K * I >= 40 << 20 and E * -(-I // 128) >= 192
    rng = np.random.default_rng(K + I)
    q = lambda *s: ql.quantize_weight_block_e4m3(dev(rng.standard_normal(s, dtype=np.float32) / np.float32(np.sqrt(s[-1]))))  # noqa: E731,E501
    weights = (*q(E, 2 * I, K), *q(E, K, I))
    x, lg = rng.standard_normal((T, K)).astype(np.float16), rng.standard_normal((T, E)).astype(np.float32)
    out = host(ql.moe_e4m3_block(dev(x), dev(lg), *weights, k, True, torch.float32))
    some = sorted({0, 7, 17, min(34, T - 1), min(51, T - 1), T - 1})
    codes = [host(a.view(torch.uint8)) if a.dtype is not torch.float32 else host(a) for a in weights]
    _check(out[some], (x[some], lg[some], *codes), k, True)
