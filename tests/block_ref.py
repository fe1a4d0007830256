"""A plain numpy implementation of the layers with a scale for each block of 128: the quantizers in
the fp32 operations of their definitions, the products and the mixture-of-experts layer in 64 bits."""
import numpy as np
import torch

F32 = np.float32
B = 128


def blocks(n):
    return -(-n // B)


def e4m3(v):
    """Codes of fp32 values of at most 448, round to nearest even."""
    return torch.from_numpy(np.ascontiguousarray(v, F32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def _table():
    out = np.zeros(256)
    for c in range(256):
        e, f = c >> 3 & 15, c & 7
        out[c] = (-1 if c & 128 else 1) * (f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
    return out


TABLE = _table()


def decode(codes):
    return TABLE[codes]


def quant_rows(x):
    """codes uint8 [M, K], scales fp32 [blocks, M]."""
    x = x.astype(F32)
    q = np.zeros(x.shape, np.uint8)
    s = np.zeros((blocks(x.shape[1]), x.shape[0]), F32)
    for b in range(s.shape[0]):
        v = x[:, b * B:(b + 1) * B]
        s[b] = np.maximum(np.abs(v).max(1), F32(1e-10)) / F32(448)
        q[:, b * B:(b + 1) * B] = e4m3(np.clip(v / s[b][:, None], F32(-448), F32(448)))
    return q, s


def quant_weight(w):
    """codes uint8 [E, N, K], scales fp32 [E, blocks of N, blocks of K]."""
    w = w.astype(F32)
    E, N, K = w.shape
    q = np.zeros(w.shape, np.uint8)
    s = np.zeros((E, blocks(N), blocks(K)), F32)
    for e in range(E):
        for i in range(s.shape[1]):
            for j in range(s.shape[2]):
                at = np.s_[e, i * B:(i + 1) * B, j * B:(j + 1) * B]
                s[e, i, j] = np.maximum(np.abs(w[at]).max(), F32(1e-10)) / F32(448)
                q[at] = e4m3(np.clip(w[at] / s[e, i, j], F32(-448), F32(448)))
    return q, s


def weight64(q, s):
    """What codes [N, K] with scales [blocks, blocks] stand for."""
    N, K = q.shape
    return decode(q) * np.repeat(np.repeat(s.astype(np.float64), B, 0)[:N], B, 1)[:, :K]


def gemm64(xq, xs, wq, ws):
    """With a row of scales for each column (ws [N, blocks of K]): the product before the bias,
    and a bound on the kernel's error, both [M, N]. Per group of 8 consecutive k the matrix cores truncate each product to a multiple of 2^(E - 13), E the group's
    largest sum of exponents; 16 groups a block are added in fp32, the block's scales multiplied
    and the block added, up to 8 partial sums joined."""
    M, K = xq.shape
    N = wq.shape[0]
    x, w = decode(xq), decode(wq)
    y, err, mag = (np.zeros((M, N)) for _ in range(3))
    exp = lambda v: np.where(v == 0, -99, np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))).astype(np.int32)  # noqa: E731
    ex, ew = exp(x), exp(w)
    for b in range(blocks(K)):
        sc = xs[b].astype(np.float64)[:, None] * ws[:, b].astype(np.float64)[None]
        lo, hi = b * B, min(K, b * B + B)
        y += sc * (x[:, lo:hi] @ w[:, lo:hi].T)
        mag += np.abs(sc) * (np.abs(x[:, lo:hi]) @ np.abs(w[:, lo:hi]).T)
        for g in range(lo, hi, 8):
            e = np.max(ex[:, None, g:g + 8] + ew[None, :, g:g + 8], axis=2)
            err += np.abs(sc) * np.where(e > -60, 8 * 2.0 ** (e - 13.0), 0)
    return y, err + mag * (16 + 3 + blocks(K) + 8) * 2.0 ** -24


def activate64(y, act):
    from math import erfc
    if act == "gelu":
        return y * 0.5 * np.vectorize(erfc)(-y / np.sqrt(2.0))
    if act == "silu":
        return y / (1 + np.exp(-y))
    return y


def gemm_tolerance(pre, err, bias, act, f16):
    """Bound on |y - exact| from the bound `err` on the product `pre` [M, N] without the bias."""
    v = pre if bias is None else pre + bias.astype(np.float64)
    err = err + (0 if bias is None else 2.0 ** -24 * np.abs(v))
    y = activate64(v, act)
    if act == "gelu":      # |gelu'| <= 1.13; the kernel's own evaluation: 1.5e-5 |v| before fp16, 2e-7 |v| else
        err = 1.13 * err + (1.5e-5 if f16 else 2e-7) * np.abs(v)
    elif act == "silu":    # |silu'| <= 1.1; exponential, reciprocal, sum and product
        err = 1.1 * err + (np.abs(v) + 4) * 2.0 ** -23 * np.abs(y) + 1e-30
    half = 2.0 ** -11 if f16 else 2.0 ** -24
    return y, err * (1 + half) + half * np.abs(y) + (2.0 ** -25 if f16 else 1e-37)


def routes(logits, k, renorm):
    """Per token the chosen experts (fewer than k where -inf or NaN leave fewer), their weights in 64
    bits, and a bound on the relative error of the kernel's fp32 weights."""
    out = []
    for row in logits:
        ok = [e for e in range(row.size) if row[e] > -np.inf]
        ids = sorted(ok, key=lambda e: (-row[e], e))[:k]
        if not ids:
            out.append(([], np.zeros(0), np.zeros(0)))
            continue
        d = row.astype(np.float64) - float(row[ids[0]])
        w = np.where(np.isnan(d), 0, np.exp(np.where(np.isnan(d), 0, d)))
        among = np.array(ids) if renorm else np.array(ok)
        total = w[among].sum()
        # an exponential of d: |d| + 4 units of 2^-23; up to 48 additions of positive terms; division
        one = lambda e: (np.abs(d[e]) + 4) * 2.0 ** -23  # noqa: E731
        rel = one(ids) + (w[among] * one(among)).sum() / total + 50 * 2.0 ** -24
        out.append((ids, w[ids] / total, rel))
    return out


def bf16_terms(h, terms):
    """h rounded to fp32, as the sum of so many bf16 terms, each the nearest to what those before leave."""
    rest = torch.from_numpy(np.ascontiguousarray(h, F32))
    out = torch.zeros(rest.shape, dtype=torch.float64)
    for _ in range(terms):
        t = rest.bfloat16().float()
        out += t.double()
        rest = rest - t
    return out.numpy()


def moe64(x, logits, w13, s13, w2, s2, k, renorm, h_error=2.0 ** -17, terms=None):
    """The layer in 64 bits, and a bound on the kernel's error before the output's rounding, both
    [T, K]. h_error: of h's terms, 2^-17 for two (fp16 outputs), 2^-25 for three (fp32). With `terms`, the result is that
    of h cut to so many terms, for tests of what a comparison tells apart. fp16 (bf16) products with codes are exact in fp32; a sum of n products in any order, each
    addition at most one unit off, has an error of n 2^-23 of the sum of magnitudes: 128 and 4 more
    in a block, one a block, 8 at the join."""
    T, K = x.shape
    E, I2, _ = w13.shape
    I = I2 // 2
    x = x.astype(np.float64)
    y, err = np.zeros((T, K)), np.zeros((T, K))
    up = (132 + blocks(K) + 8) * 2.0 ** -23
    route = routes(logits, k, renorm)
    down = (132 + blocks(I) * k + k + 8) * 2.0 ** -23
    for e in range(E):
        rows = [t for t in range(T) if e in route[t][0]]
        if not rows:
            continue
        a, b = weight64(w13[e], s13[e]), weight64(w2[e], s2[e])
        p = np.array([route[t][1][route[t][0].index(e)] for t in rows])[:, None]
        prel = np.array([route[t][2][route[t][0].index(e)] for t in rows])[:, None]
        gu, mag = x[rows] @ a.T, np.abs(x[rows]) @ np.abs(a).T
        g, u, eg, eu = gu[:, :I], gu[:, I:], up * mag[:, :I], up * mag[:, I:]
        with np.errstate(over="ignore"):
            s = g / (1 + np.exp(-g))
        es = 1.1 * eg + (np.abs(g) + 4) * 2.0 ** -23 * np.abs(s) + 1e-30
        h = p * s * u
        # both factors' errors, the weight's, three roundings, the bf16 terms
        eh = p * (es * (np.abs(u) + eu) + np.abs(s) * eu) + np.abs(h) * (prel + 3 * 2.0 ** -24 + h_error)
        if terms is not None:
            h = bf16_terms(h, terms)
        y[rows] += h @ b.T
        err[rows] += eh @ np.abs(b).T + down * (np.abs(h) + eh) @ np.abs(b).T
    return y, err
