"""The weights of attention_kv4 enter the matrix cores as two fp16 terms, so that with values that are
exact in fp16 the output's own rounding is the only one to fewer bits than fp32's. V here is
(code - 8) / 8, exact, with sums close to 0, where an error of the weights is not hidden by the output's rounding.

Bound. Output: U |o|, or 2^-25 below fp16's normal range. Weights: two terms hold 22 bits, 2^-22 of
each weight in the sum of values and in that of weights, and 2^-25 where a term is below fp16's normal
range, beside a largest weight of 2^6 and more: n 2^-31 max|v|. Scores: e = 2 (D + 8) 2^-24 top relative to each
weight and 2^-20 for the exponential, twice (values and weights). The sums' fp32 roundings: n 2^-24 each.
"""
import numpy as np
import pytest
import torch

import kv4_ref as ref

U = 2.0 ** -11
D, G, P = 64, 64, 16


def _inputs(seed, H, n, rows, R):
    rng = np.random.default_rng(seed)
    pages = -(-n // P)
    cache = rng.integers(0, 256, (pages, H, ref.page_bytes(P, D, G)), dtype=np.uint8)
    for which in range(2):
        at = P * D // 2 * (1 + which) + which * 4 * P
        par = np.empty((pages, H, 2, P), np.float16)
        par[:, :, 0], par[:, :, 1] = 0.125, -1.0
        cache[:, :, at:at + 4 * P] = par.reshape(pages, H, -1).view(np.uint8)
    q = np.zeros((rows, H * R, D), np.float16)
    q[:, :, 5] = rng.uniform(-0.7, 0.7, (rows, H * R))
    q[:, :, 40] = rng.uniform(-0.7, 0.7, (rows, H * R))
    return rng.permutation(pages).astype(np.int32)[None], cache, q


def _bound(o, mag, top, n, vmax):
    d = 2 * (D + 8) * 2.0 ** -24 * top[..., None] + 2.0 ** -20
    return np.maximum(U * np.abs(o), 2.0 ** -25) + (2 * d + 2 * 2.0 ** -22 + 2 * n * 2.0 ** -24) * mag + n * 2.0 ** -31 * vmax


def _weights(q, k, v, terms):
    """One row's output with its weights rounded to `terms` fp16 terms, in 64 bits otherwise."""
    s = k @ q.astype(np.float64)
    w = 64 * np.exp(s - s.max())
    hi = w.astype(np.float16).astype(np.float64)
    p = hi + (w - hi).astype(np.float16) if terms == 2 else hi
    return p @ v / p.sum()


def test_the_bound_tells_one_term_from_two():
    """On the CPU: the bound holds with two terms and fails with one, on most rows."""
    table, cache, q = _inputs(1, 4, 7, 1, 2)
    k, v = ref.read_rows(cache, table[0], P, D, G, 7)
    o, mag, top = ref.attention64(q, k, v, 7, 1.0, 0)
    failed = 0
    for h in range(8):
        tol = _bound(o, mag, top, 7, 1.0)[0, h]
        out = [_weights(q[0, h], k[:, h // 2], v[:, h // 2], t).astype(np.float16) for t in (1, 2)]
        assert np.all(np.abs(out[1] - o[0, h]) <= tol)
        failed += not np.all(np.abs(out[0] - o[0, h]) <= tol)
    assert failed >= 6


@pytest.mark.gpu
@pytest.mark.parametrize("H,n,rows,max_q,max_len", [(4, 7, 1, 1, 7), (2, 5, 3, 3, 5), (8, 30, 2, 2, 30),
                                                    (256, 64, 64, 64, 300), (256, 70, 64, 64, 300)])
def test_two_terms(H, n, rows, max_q, max_len):
    """Single tokens, drafts and the prompt kernel."""
    import int8_quantized_linear_amd as ql
    from gpu_util import dev, host

    R = 2 if H < 256 else 4
    table, cache, q = _inputs(H + n, H, n, rows, R)
    got = host(ql.attention_kv4(dev(q), dev(cache), dev(table), dev(np.array([n], np.int32)),
                                dev(np.array([0, rows], np.int32)), page_size=P, group=G, scale=1.0, max_q=max_q,
                                max_len=max_len)).astype(np.float64)
    assert torch.cuda.is_available()
    some = slice(0, min(H, 8))
    k, v = (x[:, some] for x in ref.read_rows(cache, table[0], P, D, G, n))
    heads = slice(0, min(H, 8) * R)
    for i in range(0, rows, max(1, rows // 12)):
        m = n - rows + i + 1
        o, mag, top = ref.attention64(q[i:i + 1, heads], k[:m], v[:m], m, 1.0, 0)
        assert np.all(np.abs(got[i:i + 1, heads] - o) <= _bound(o, mag, top, m, 1.0)), i
