"""attention_kv4 with a scale of 0 and with very small ones: rows without a position
give zeros next to rows that have one, and hidden positions no weight."""
import pytest

from test_gpu_attention_kv4 import _check, ql  # noqa: F401

pytestmark = pytest.mark.gpu

SCALES = [0.0, -0.0, 1e-45, -1e-40, 1e-30, 1e-20, -1e-17, 1e-10]


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("D,G", [(64, 32), (128, 64), (256, 128)])
def test_decode(ql, D, G, scale):  # noqa: F811
    _check(ql, D, [5, 300, 12, 0], [8, 6, 17, 2], 16, 2, 3, D, G, scale=scale)
    _check(ql, D, [700, 0, 3], [1, 1, 1], 16, 2, 3, D, G, scale=scale)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("H,D,G", [(128, 64, 32), (128, 128, 64), (64, 128, 64), (128, 256, 128)])
def test_prompt(ql, H, D, G, scale):  # noqa: F811
    _check(ql, D, [300, 20], [64, 64], 64, H, 4, D, G, scale=scale, max_q=64, max_len=300, samples=6)
