"""attention_kv4 with queries far below 1 and a scale that makes ordinary scores of them, down to
fp16's subnormal numbers, and with queries of very different sizes in one tile: at the tolerance of
test_gpu_attention_kv4.py, whose scores count fp32's roundings only."""
import numpy as np
import pytest

import test_gpu_attention_kv4 as base
from test_gpu_attention_kv4 import DG, ql  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gain", [2e-3, 1e-4, 1e-5, 1e-6])
@pytest.mark.parametrize("D,G", DG)
def test_decode(ql, D, G, gain):  # noqa: F811
    base._check(ql, D + G, [90, 33, 400], [1, 2, 5], 32, 2, 4, D, G, gain=gain, scale=2.0 / (gain * D ** 0.5))


@pytest.mark.parametrize("gain", [1e-4, 1e-6])
@pytest.mark.parametrize("D,G", DG)
def test_prompt(ql, D, G, gain):  # noqa: F811
    base._check(ql, D + G, [300, 64], [64, 64], 64, 128, 4, D, G, gain=gain, scale=2.0 / (gain * D ** 0.5),
                max_q=64, max_len=300, samples=3)


@pytest.mark.parametrize("H", [2, 64, 128])
def test_sizes_beside_each_other(ql, H, monkeypatch):  # noqa: F811
    """Every (row, head) a size of its own, from subnormal to thousands, over scores of its own size."""
    draw = np.random.default_rng

    class Rng:
        def __init__(self, seed):
            self.r = draw(seed)

        def __getattr__(self, name):
            return getattr(self.r, name)

        def standard_normal(self, shape):
            x = self.r.standard_normal(shape)
            if len(shape) == 3:   # q [rows, heads, D]
                x *= 10.0 ** self.r.uniform(-6, 3.5, shape[:2])[..., None]
            return x

    monkeypatch.setattr(base.np.random, "default_rng", Rng)
    for scale in (1e-3, 1.0, 1e3):
        base._check(ql, 5, [200, 64], [64 if H > 2 else 4, 64 if H > 2 else 1], 32, H, 4, 128, 64, scale=scale,
                    samples=4, max_q=64 if H > 2 else None, max_len=300 if H > 2 else None)
