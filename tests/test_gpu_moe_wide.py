"""The experts' kernels for many tokens an expert: every token of a batch, bit for bit as in calls of so few that the
other kernels take them, with experts that all tokens, some and none take; a sample of the tokens, one at least of each
16 pairs of the expert that all take, against 64 bits."""
import numpy as np
import pytest
import torch

import block_ref as ref
from gpu_util import Guarded, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    import int8_quantized_linear_amd as ql

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return ql


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("T,E,k,K,I", [(33, 3, 2, 2048, 8256), (64, 6, 2, 1984, 4160), (70, 7, 7, 1600, 4096),
                                       (128, 8, 2, 1088, 4928), (20, 2, 1, 4096, 12352), (64, 65, 16, 2112, 512)])
def test_every_token(ql, T, E, k, K, I, f16):
    assert T * k >= 8 * E and E * K * I >= 40 << 20 and E * -(-I // 128) >= 192
    rng = np.random.default_rng(T + I)
    q = lambda *s: ql.quantize_weight_block_e4m3(dev(rng.standard_normal(s, dtype=np.float32) / np.float32(np.sqrt(s[-1]))))  # noqa: E731,E501
    (w13, s13), (w2, s2) = q(E, 2 * I, K), q(E, K, I)
    x = rng.standard_normal((T, K)).astype(np.float16)
    lg = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    lg[:, 0] += 100          # all tokens
    if E > k:
        lg[:, E - 1] = -np.inf
    dt = torch.float16 if f16 else torch.float32
    args = (w13, s13, w2, s2, k, f16, dt)
    out = Guarded((T, K), dt)
    ql.moe_e4m3_block(dev(x), dev(lg), *args, out.view)
    out.check()
    few = (8 * E - 1) // k   # tokens of a call of the other kernels
    for n in (few, 1, 7):
        for t in range(0, T, n):
            part = ql.moe_e4m3_block(dev(x[t:t + n]), dev(lg[t:t + n]), *args)
            assert torch.equal(part, out.view[t:t + n]), (n, t)
    some = sorted({t for t in (0, 15, 16, 31, 32, 47, 48, 63, 64, T - 1) if t < T})
    codes = [host(a.view(torch.uint8)) if a.dtype is not torch.float32 else host(a) for a in (w13, s13, w2, s2)]
    want, err = ref.moe64(x[some], lg[some], *codes, k, f16, h_error=2.0 ** -17 if f16 else 2.0 ** -25)
    half, least = (2.0 ** -11, 2.0 ** -25) if f16 else (2.0 ** -24, 1e-37)
    diff = np.abs(host(out.view)[some].astype(np.float64) - want)
    assert (diff <= err * (1 + half) + half * np.abs(want) + least).all()
