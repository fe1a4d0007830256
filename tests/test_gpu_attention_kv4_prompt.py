"""attention_kv4 on batches large enough for the prompt kernel, with 16 and with 32 (row, head)
pairs a wave: the same comparison in 64 bits, on sampled rows, at the same tolerance as the small
batches'."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_util import dev
from test_gpu_attention_kv4 import DG, _cache, _check, ql  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("D,G", DG)
def test_head_sizes(ql, D, G, P):  # noqa: F811
    """A chunk after a prefix, a prompt from position 0 with its end inside a tile, a row without a
    position."""
    _check(ql, D + G + P, [500, 50, 0], [64, 50, 1], P, 128, 4, D, G, max_q=64, max_len=500, samples=3)


@pytest.mark.parametrize("P", [32, 256])
@pytest.mark.parametrize("G", [32, 64, 128])
def test_few_workgroups(ql, G, P):  # noqa: F811
    """Half as many heads: 16 pairs a wave for D = 128 too."""
    _check(ql, G + P, [500, 41], [64, 41], P, 64, 4, 128, G, max_q=64, max_len=500, samples=4)


@pytest.mark.parametrize("window", [1, 63, 64, 200, 5000])
def test_window(ql, window):  # noqa: F811
    _check(ql, window, [450, 64], [64, 64], 16, 128, 4, 128, 64, window=window, max_q=64, max_len=450, samples=4)


def test_uneven_rows(ql):  # noqa: F811
    """Tiles that end between a row's heads, more rows than positions, single positions."""
    _check(ql, 11, [400, 36, 1, 9], [36, 30, 1, 20], 32, 64, 7, 128, 64, max_q=36, max_len=400, samples=6)


@pytest.mark.parametrize("gain,scale", [(40.0, None), (1e-4, None), (1.0, -0.2), (0.0, None)])
def test_scores(ql, gain, scale):  # noqa: F811
    _check(ql, 12, [300, 64], [64, 64], 64, 128, 4, 128, 64, gain=gain, scale=scale, max_q=64, max_len=300, samples=3)


@pytest.mark.parametrize("H,D", [(64, 128), (128, 128), (128, 64), (128, 256)])
def test_repeats_bit_for_bit(ql, H, D):  # noqa: F811
    rng = np.random.default_rng(H + D)
    P, G = 16, 64
    b = ref.Batch(rng, [500, 77], [64, 64], P)
    cache, meta = dev(_cache(rng, b, H, D, G)), [dev(a) for a in b.arrays()]
    q = dev(rng.standard_normal((b.total, H * 4, D)).astype(np.float16))
    call = lambda: ql.attention_kv4(q, cache, *meta, page_size=P, group=G, max_q=64, max_len=500)  # noqa: E731
    first = call()
    for _ in range(10):
        assert torch.equal(call(), first)
