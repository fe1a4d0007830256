"""A plain numpy implementation of the operators around the quantized layer -- the norm written
as 8-bit codes, the paged 4-bit K/V cache and attention over it -- in 64 bits where the library
sums, and in the fp32 and fp16 operations of the definitions where a code is decided. Every
element's place in a page is worked out by itself, from the layout stated in csrc/kv4.h."""
import numpy as np

F32 = np.float32


def norm_codes(x, res, gamma, most):
    """fp32 h, t / s before rounding, and s, each operation of the definition rounded on its own."""
    h = x.astype(F32) if res is None else res.astype(F32) + x.astype(F32)
    t = h * gamma[None, :]
    s = np.maximum(np.abs(t).max(1), F32(1e-10)) / F32(most)
    return h, t / s[:, None], s


def norm_scale64(h, s, eps):
    return s.astype(np.float64) / np.sqrt((h.astype(np.float64) ** 2).mean(1) + np.float64(F32(eps)))


def page_bytes(P, D, G):
    return P * (D + 8 * (D // G))


def quantize4(x, G):
    """codes uint8 [..., D], scale and low fp16 [..., D / G]."""
    x = x.astype(F32)
    g = x.reshape(*x.shape[:-1], -1, G)
    low = np.clip(g.min(-1), F32(-65504), F32(65504)).astype(np.float16)
    with np.errstate(over="ignore"):
        s = np.clip((g.max(-1) - low.astype(F32)) / F32(15), F32(0), F32(65504)).astype(np.float16)
    s = np.maximum(s, np.float16(2.0 ** -24))
    c = np.rint((g - low.astype(F32)[..., None]) / s.astype(F32)[..., None])
    return np.clip(c, 0, 15).astype(np.uint8).reshape(x.shape), s, low


def _k_place(P, D, slot, d):
    """Byte and shift of K's element d of token `slot`."""
    i, kg, e = d // 32, d % 32 // 8, d % 8
    bit = 16 * (e % 2) + 4 * (e // 2)
    return slot * (D // 2) + (kg * (D // 32) + i) * 4 + bit // 8, bit % 8


def _v_place(P, D, G, slot, d):
    quad, part = d // 64 * 16 + d % 32 // 2, 2 * (d % 64 // 32) + d % 2
    bit = 4 * part
    return P * D // 2 + 4 * P * (D // G) + slot // 8 * 4 * D + quad * 16 + slot % 8 * 2 + bit // 8, bit % 8


def _params(P, D, G, which, slot, g):
    base = (P * D // 2) * (1 + which) + which * 4 * P * (D // G)
    at = base + g * 4 * P + 2 * slot
    return at, at + 2 * P


def write_token(block, P, D, G, slot, k, v):
    """Writes one token's k and v [D] into a page of one head, uint8 [page bytes]."""
    d = np.arange(D)
    for which, x in ((0, k), (1, v)):
        c, s, low = quantize4(x, G)
        at, sh = _k_place(P, D, slot, d) if which == 0 else _v_place(P, D, G, slot, d)
        for byte, shift, code in zip(at, sh, c):
            block[byte] = (int(block[byte]) & ~(15 << shift)) | (int(code) << shift)
        for g in range(D // G):
            a, b = _params(P, D, G, which, slot, g)
            block[a:a + 2] = np.frombuffer(s[g].tobytes(), np.uint8)
            block[b:b + 2] = np.frombuffer(low[g].tobytes(), np.uint8)


def read_rows(cache, pages, P, D, G, n):
    """k and v float64 [n, H, D] of the first n tokens of a sequence with these pages."""
    H = cache.shape[1]
    k, v = np.zeros((n, H, D)), np.zeros((n, H, D))
    d = np.arange(D)
    for first in range(0, n, P):
        blk = cache[pages[first // P]]
        m = min(P, n - first)
        slot = np.arange(m)[:, None]
        for which, out in ((0, k), (1, v)):
            at, sh = _k_place(P, D, slot, d[None]) if which == 0 else _v_place(P, D, G, slot, d[None])
            code = (blk[:, at] >> sh) & 15
            a, b = _params(P, D, G, which, slot, d[None] // G)
            s = (blk[:, a].astype(np.uint16) | blk[:, a + 1].astype(np.uint16) << 8).view(np.float16)
            low = (blk[:, b].astype(np.uint16) | blk[:, b + 1].astype(np.uint16) << 8).view(np.float16)
            out[first:first + m] = (code * s.astype(np.float64) + low.astype(np.float64)).transpose(1, 0, 2)
    return k, v


def attention64(q, k, v, length, scale, window):
    """o and sum_j p_j |v_j| and max_j |score| of rows q [n, HQ, D], the last n of `length`
    positions, over k and v [length, H, D]; all float64."""
    n, HQ, D = q.shape
    R = HQ // k.shape[1]
    o, mag, top = np.zeros((n, HQ, D)), np.zeros((n, HQ, D)), np.zeros((n, HQ))
    for i in range(n):
        p = length - n + i
        if p < 0:
            continue
        first = max(0, p - window + 1) if window else 0
        for h in range(HQ):
            kk, vv = k[first:p + 1, h // R], v[first:p + 1, h // R]
            s = (kk @ q[i, h].astype(np.float64)) * scale
            top[i, h] = (np.abs(kk) @ np.abs(q[i, h].astype(np.float64))).max() * abs(scale)
            w = np.exp(s - s.max())
            w /= w.sum()
            o[i, h], mag[i, h] = w @ vv, w @ np.abs(vv)
    return o, mag, top


class Batch:
    """A batch of sequences over a paged cache: lengths, rows per sequence, a page table with the
    pages of all sequences in random order, and spare pages."""

    def __init__(self, rng, lens, rows, P, spare=2, extra_width=1):
        need = [-(-max(0, n) // P) for n in lens]
        self.P, self.lens, self.rows = P, list(lens), list(rows)
        self.pages = sum(need) + spare
        self.width = max(need + [0]) + extra_width
        order = rng.permutation(self.pages)
        self.table = np.full((len(lens), self.width), 2 ** 31 - 1, np.int32)   # unused entries: far outside
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.total = int(self.starts[-1])

    def arrays(self):
        return self.table, np.array(self.lens, np.int32), self.starts
