"""The tests of the experts' fp32 outputs tell three terms of h from two: on the CPU, with h cut in the reference."""
import pytest

import block_ref as ref
from moe_cases import NARROW, NORM, TOKEN_NORM, inputs, norm_errors


@pytest.mark.parametrize("T,E,k,K,I", NARROW)
def test_two_terms_fail(T, E, k, K, I):
    inp = inputs(T, E, K, I)
    want, _ = ref.moe64(*inp, k, True)
    whole, row = norm_errors(ref.moe64(*inp, k, True, terms=2)[0], want)
    assert whole > 2 * NORM and row > TOKEN_NORM
    whole, row = norm_errors(ref.moe64(*inp, k, True, terms=3)[0], want)
    assert whole < NORM / 20 and row < TOKEN_NORM / 20
