"""Starts that break attention_kv4's contract (below 0, past the rows, falling, far apart) lead to no read
of q and no write of out or of the workspace outside them, in either kernel and with splits, and leave the rows that valid
sequences own right."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_util import Guarded, dev, host
from test_gpu_attention_kv4 import _cache, ql  # noqa: F401

pytestmark = pytest.mark.gpu

BIG = 2 ** 31 - 1
STARTS = [[-3, 2, 6], [-5, -2, 6], [0, 9, 6], [4, 1, 6], [-BIG, BIG, 6], [BIG, -BIG, 6], [-BIG - 1, 0, 6],
          [7, 8, 9], [0, 6, -BIG], [BIG - 2, BIG, 6]]


@pytest.mark.parametrize("H,rows,lens", [(2, 6, [40, 30]), (2, 6, [3000, 2000]), (256, 64, [90, 300])])
@pytest.mark.parametrize("starts", STARTS)
def test_nothing_outside(ql, H, rows, lens, starts):  # noqa: F811
    P, D, G, R = 32, 64, 32, 4
    starts = [rows if s == 6 else s for s in starts]
    rng = np.random.default_rng(1)
    b = ref.Batch(rng, lens, [3, 3], P)
    q = Guarded((rows, H * R, D), torch.float16)
    q.view.normal_()
    out = Guarded((rows, H * R, D), torch.float16)
    cache = dev(_cache(rng, b, H, D, G))
    before = cache.clone()
    meta = [dev(b.table), dev(np.array(lens, np.int32)), dev(np.array(starts, np.int64).astype(np.int32))]
    ql.attention_kv4(q.view, cache, *meta, page_size=P, group=G, out=out.view, max_q=rows, max_len=max(lens))
    torch.cuda.synchronize()
    out.check()
    assert torch.equal(cache, before)


def test_valid_sequences_beside(ql):  # noqa: F811
    P, D, G, H, R = 32, 64, 32, 2, 2
    rng = np.random.default_rng(2)
    b = ref.Batch(rng, [50, 70, 40], [2, 3, 2], P)
    cache, q = dev(_cache(rng, b, H, D, G)), dev(rng.standard_normal((5, H * R, D)).astype(np.float16))
    call = lambda n, s: host(ql.attention_kv4(q, cache, dev(b.table), dev(np.array(n, np.int32)),  # noqa: E731
                                              dev(np.array(s, np.int32)), page_size=P, group=G))
    good = call([50, 70, 40], [0, 2, 5, 5])
    bad = call([50, 70, 40], [0, 2, 5, -BIG])
    assert np.array_equal(good, bad)
