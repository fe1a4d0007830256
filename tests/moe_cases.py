"""Inputs of the tests of the experts' precision and of a bound that tells the number of h's terms apart."""
import numpy as np

import block_ref as ref

# Relative error of the norm of fp32 outputs, whole and of any token. Three terms leave h 2^-25, and the rest is fp32
# arithmetic: sums of n additions in a row, whose roundings (2^-24 / 3^(1/2) of a partial sum) are independent, are off
# by (n / 2)^(1/2) of one; at most 160 for a block's products, the blocks and the join give 3.1e-7 for each of the three
# products, 5.3e-7 together; silu, the products of h and the softmax of logits a few apart add a few 2^-24. Two terms alone leave h 2.4e-6 in the
# mean square (test_moe_terms.py).
NORM, TOKEN_NORM = 1e-6, 1.5e-6

# T, E, top_k, K, I: K and I of whole and of half blocks, one to eight tokens (routes by rank) and more
NARROW = [(1, 8, 2, 2048, 1536), (4, 64, 8, 512, 256), (5, 6, 2, 448, 704), (8, 70, 3, 1984, 320), (17, 9, 3, 320, 1344),
          (40, 12, 4, 1024, 640), (64, 5, 2, 704, 448), (70, 40, 2, 256, 384)]


def inputs(T, E, K, I):
    rng = np.random.default_rng(T + 3 * E + K + I)
    w = lambda *s: ref.quant_weight(rng.standard_normal(s, dtype=np.float32) / np.float32(np.sqrt(s[-1])))  # noqa: E731
    x = rng.standard_normal((T, K)).astype(np.float16)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    return (x, logits, *w(E, 2 * I, K), *w(E, K, I))


def norm_errors(got, want):
    """Of the whole, and the largest of a row."""
    d = got - want
    rows = np.linalg.norm(d, axis=1) / np.linalg.norm(want, axis=1)
    return np.linalg.norm(d) / np.linalg.norm(want), rows.max()
