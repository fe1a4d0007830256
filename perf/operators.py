"""The operators around the quantized linear layer that a decoder's attention block needs, on
the shapes they meet in serving: what is computed in plain torch, what the library's calls
compute, and what each case has to move.

  norm   h = residual + x; codes and per-row scales of rms_norm(h) * gamma, int8 or fp8 (E4M3)
  kv     new K and V rows quantized into pages of a 4-bit cache, and rows read back from it
  attn   causal attention of the last rows of each sequence over that cache

Sizes: 4096-wide rows with 32 heads of 128 are the Llama-7B layer that the benchmark's
workloads are drawn for; 11008 is its feed-forward width; the others are generic.
"""
import math

import torch

own = False

F16, F32 = torch.float16, torch.float32


def listed():
    return [
        # one token's rows before the first projection of a layer: latency only
        dict(name="norm_one_token", op="norm", M=1, K=4096, x="f16", res="f16", out="int8"),
        # a ragged batch on a width that is no power of two, fp8 codes, residual kept in fp32
        dict(name="norm_ragged_e4m3", op="norm", M=333, K=11008, x="f16", res="f32", out="e4m3"),
        # a prompt's rows, the benchmark's M2048 K4096 layer
        dict(name="norm_prompt", op="norm", M=2048, K=4096, x="f16", res="f16", out="int8"),
        # one new token for each of 32 sequences: the write that every decode step makes
        dict(name="kv_decode_step", op="kv", B=32, new=1, L=1500, Hkv=8, D=128, G=64, P=16, read="new", x="f16"),
        # ragged prompts written at once, one scale for each head's row
        dict(name="kv_prompts", op="kv", B=5, new=1777, L=1777, Hkv=32, D=128, G=128, P=64, read="new", x="f16"),
        # a step's write, then whole sequences read back in fp16 (moved to another cache)
        dict(name="kv_read_all", op="kv", B=8, new=1, L=4099, Hkv=8, D=128, G=32, P=32, read="all", x="f32"),
        # one short chat turn, 32 heads of their own K and V: latency
        dict(name="attn_one_short", op="attn", B=1, q=1, L=517, Hkv=32, R=1, D=128, G=128, P=16, window=0),
        # a decode batch of mixed lengths with shared heads, its last slot idle (length 0)
        dict(name="attn_batch_ragged", op="attn", B=33, q=1, L=4100, Hkv=8, R=4, D=128, G=64, P=16, window=0),
        # one very long context: the split over the length has to fill the chip
        dict(name="attn_one_long", op="attn", B=1, q=1, L=131072, Hkv=8, R=4, D=128, G=64, P=64, window=0),
        # a full serving batch at long context: 600 MB of cache
        dict(name="attn_batch_long", op="attn", B=64, q=1, L=16384, Hkv=8, R=8, D=128, G=64, P=64, window=0),
        # a few drafted tokens a sequence, sliding window, small heads
        dict(name="attn_draft_window", op="attn", B=16, q=5, L=3001, Hkv=4, R=7, D=64, G=32, P=32, window=1024),
        # a prompt's chunk after a cached prefix
        dict(name="attn_prompt", op="attn", B=1, q=2048, L=4096, Hkv=8, R=4, D=128, G=64, P=64, window=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "kv", "kv", "attn", "attn", "attn"])
    if op == "norm":
        k = 64 * _log(rng, 4, 256)
        return dict(op="norm", M=_log(rng, 1, min(4096, 2 ** 25 // k)), K=k, x=rng.choice(["f16", "f32"]),
                    res=rng.choice(["none", "f16", "f32"]), out=rng.choice(["int8", "e4m3"]))
    d = rng.choice([64, 128, 128, 256])
    g = rng.choice([n for n in (32, 64, 128) if n <= d])
    c = dict(op=op, B=_log(rng, 1, 64), D=d, G=g, P=rng.choice([16, 32, 64, 128, 256]))
    if op == "kv":
        c["read"] = rng.choice(["new", "all"])
        c["Hkv"] = rng.choice([1, 2, 4, 8, 32])
        rows = max(1, 2 ** 25 // (c["B"] * c["Hkv"] * d))
        c["new"] = rng.choice([1, _log(rng, 1, min(rows, 4096))])
        c["L"] = max(c["new"], _log(rng, 1, min(rows, 8192)))
        c["x"] = rng.choice(["f16", "f32"])
        return c
    c["R"] = rng.choice([1, 2, 3, 4, 7, 8, 16])
    c["Hkv"] = rng.choice([1, 2, 4, 8])
    kind = rng.choice(["one", "few", "prompt"])
    if kind == "prompt":
        c["B"] = min(c["B"], 4)
        c["q"] = _log(rng, 17, 2048)
        rows = 2 ** 35 // (c["B"] * c["q"] * c["R"] * c["Hkv"] * d)
        c["L"] = max(c["q"], _log(rng, 17, max(17, min(8192, rows))))
        while c["B"] * c["q"] * c["L"] * c["R"] * c["Hkv"] * d > 2 ** 35:
            c["q"] = max(1, c["q"] // 2)
            c["L"] = max(c["q"], c["L"] // 2)
    else:
        c["q"] = 1 if kind == "one" else _log(rng, 2, 16)
        rows = 2 ** 28 // (c["B"] * c["q"] * c["Hkv"] * d)
        c["L"] = max(c["q"], _log(rng, 1, max(1, min(65536, rows))))
    c["window"] = rng.choice([0, 0, 0, _log(rng, 1, 2048)])
    return c


# ------------------------------------------------------------------ a case's row counts

def _lens(case):
    """(length, new rows) of each sequence: spread from L down, several of them with fewer new
    rows; the last of more than 32 sequences is an idle slot of length 0 with one row."""
    b, top, n = case["B"], case["L"], case["q"] if case["op"] == "attn" else case["new"]
    got = []
    for i in range(b):
        rows = max(1, n - (i * 5) % (n // 2 + 1))
        length = max(rows, top - (i * (top // 2)) // b - (i * 37) % 29 * (i > 0))
        got.append((0, 1) if b > 32 and i == b - 1 and case["op"] == "attn" else (length, rows))
    return got


def _page_bytes(case):
    return case["P"] * (case["D"] + 8 * (case["D"] // case["G"]))


# ------------------------------------------------------- the cache's bytes, in plain torch
#
# cache: uint8 [pages, kv heads, page bytes]; each page and head holds
#   K codes   [token][4][D / 32] words, word (kg, i) with d = 32 i + 8 kg + e, e = 0..7, element
#             e in bits 16 (e & 1) + 4 (e >> 1)
#   K scales  [D / G][scale, low][token] fp16
#   V codes   [token / 8][D / 4][8 tokens] 16-bit, quad n of 64-wide chunk c with d = 64 c + 2 n
#             + {0, 1, 32, 33} in bits 0, 4, 8, 12
#   V scales  as K's

def _codes(x, g):
    """x [..., D] -> codes, scale and low of each group of g: x ~ scale * code + low."""
    x = x.float().unflatten(-1, (-1, g))
    low = x.amin(-1).clamp(-65504.0, 65504.0).half()
    s = ((x.amax(-1) - low.float()) / torch.full((), 15.0, device=x.device)).clamp(0.0, 65504.0).half()
    s = torch.maximum(s, torch.full((), 2.0 ** -24, dtype=F16, device=x.device))
    c = torch.round((x - low.float()[..., None]) / s.float()[..., None]).clamp(0, 15)
    return c.to(torch.uint8).flatten(-2), s, low


def _k_bytes(c):
    """codes [..., D] -> K bytes [..., D / 2] in the order they are stored."""
    c = c.unflatten(-1, (-1, 4, 2, 2, 2))                      # i, kg, four, two, odd
    b = c[..., 0, :] | (c[..., 1, :] << 4)                     # i, kg, four, odd
    n = b.dim()
    return b.permute(*range(n - 4), n - 3, n - 4, n - 1, n - 2).reshape(*b.shape[:-4], -1)


def _v_bytes(c):
    """codes [..., D] -> V bytes [..., D / 4, 2]."""
    c = c.unflatten(-1, (-1, 2, 16, 2))                        # chunk, half, n, odd
    return (c[..., 0] | (c[..., 1] << 4)).transpose(-1, -2).flatten(-3, -2)


def _addresses(case, page, slot):
    """Byte addresses in the cache of rows at (page, slot) [T]: K bytes [T, H, D / 2], K's
    scales [T, H, D / G, 2], V bytes [T, H, D / 4, 2], V's scales."""
    h, d, g, p, dev = case["Hkv"], case["D"], case["G"], case["P"], page.device
    base = (page[:, None] * h + torch.arange(h, device=dev)) * _page_bytes(case)
    slot = slot[:, None]
    par = torch.arange(2 * (d // g), device=dev).view(-1, 2) * p * 2
    kb = (base + slot * (d // 2))[..., None] + torch.arange(d // 2, device=dev)
    kp = (base + p * d // 2 + slot * 2)[..., None, None] + par
    vb = base + p * d // 2 + p * (d // g) * 4 + (slot // 8) * (d * 4) + (slot % 8) * 2
    vb = (vb[..., None] + torch.arange(d // 4, device=dev) * 16)[..., None] + torch.arange(2, device=dev)
    vp = (base + p * d + p * (d // g) * 4 + slot * 2)[..., None, None] + par
    return kb, kp, vb, vp


def _write(case, cache, page, slot, k, v):
    """Quantizes rows k and v [T, H, D] into the cache at (page, slot) [T]."""
    kb, kp, vb, vp = _addresses(case, page, slot)
    flat, half = cache.view(-1), cache.view(F16).view(-1)
    for x, to, par, order in ((k, kb, kp, _k_bytes), (v, vb, vp, _v_bytes)):
        c, s, low = _codes(x, case["G"])
        flat[to] = order(c)
        half[par // 2] = torch.stack([s, low], -1)


def _nibbles(b):
    return torch.stack([b & 15, b >> 4], -1)


def _read(case, cache, page, slot):
    """Rows at (page, slot) [T] as fp32 k and v [T, H, D]."""
    d, g = case["D"], case["G"]
    kb, kp, vb, vp = _addresses(case, page, slot)
    flat, half = cache.view(-1), cache.view(F16).view(-1)
    k = _nibbles(flat[kb]).unflatten(-2, (4, d // 32, 2, 2))   # kg, i, odd, four, two
    k = k.permute(0, 1, 3, 2, 5, 6, 4).flatten(-5)
    v = _nibbles(flat[vb]).unflatten(2, (d // 64, 16)).transpose(3, 4).flatten(2)  # chunk, half, n, odd
    out = []
    for c, par in ((k, kp), (v, vp)):
        q = half[par // 2].float()
        out.append((c.float().unflatten(-1, (-1, g)) * q[..., :1] + q[..., 1:]).flatten(-2))
    return out


def _pages(case, cache, table):
    """All pages of `table` [B, n] as fp32 k and v [B, H, n * P, D]."""
    p, d, g, h = case["P"], case["D"], case["G"], case["Hkv"]
    blk = cache[table.long()]                                  # B, n, H, bytes
    ends = [p * d // 2, p * (d // g) * 4, p * d // 2, p * (d // g) * 4]
    kc, kp, vc, vp = (t.contiguous() for t in blk.split(ends, -1))
    lead = blk.shape[:3]
    k = _nibbles(kc.view(*lead, p, 4, d // 32, 2, 2)).permute(0, 1, 2, 3, 5, 4, 7, 8, 6).reshape(*lead, p, d)
    v = _nibbles(vc.view(*lead, p // 8, d // 64, 16, 8, 2)).permute(0, 1, 2, 3, 6, 4, 7, 5, 8).reshape(*lead, p, d)
    out = []
    for c, par in ((k, kp), (v, vp)):
        q = par.view(F16).view(*lead, d // g, 2, p).float().permute(0, 1, 2, 5, 3, 4)
        x = (c.float().unflatten(-1, (-1, g)) * q[..., :1] + q[..., 1:]).flatten(-2)
        out.append(x.permute(0, 2, 1, 3, 4).reshape(lead[0], h, -1, d))
    return out


# ---------------------------------------------------------------------------- inputs

def _rows(gen, shape, dev, gain):
    """Normal rows with a few channels larger than the others, as K projections have."""
    x = torch.randn(shape, generator=gen, device=dev)
    x[..., 3::29] *= gain
    return x


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "norm":
        m, k = case["M"], case["K"]
        x = torch.randn((m, k), generator=gen, device=dev)
        x[:, 5::997] *= 30.0
        s["x"] = x.to(F16 if case["x"] == "f16" else F32)
        s["res"] = None
        if case["res"] != "none":
            s["res"] = (4.0 * torch.randn((m, k), generator=gen, device=dev)).to(F16 if case["res"] == "f16" else F32)
        s["gamma"] = 1.0 + 0.3 * torch.randn(k, generator=gen, device=dev)
        s["eps"] = 1e-6
        return s
    b, h, d, g, p = (case[n] for n in ("B", "Hkv", "D", "G", "P"))
    rows = _lens(case)
    need = [-(-n // p) for n, _ in rows]
    width = max(need)
    count = sum(need) + 3
    order = torch.randperm(count, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros((b, width), dtype=torch.int32)
    at = 0
    where = []
    for n in need:
        where.append((at, n))
        at += n
    for i, (a, n) in enumerate(where):
        table[i, :n] = torch.arange(a, a + n, dtype=torch.int32)
    s["table"] = order[table.to(dev).long()].contiguous()
    s["lens"] = torch.tensor([n for n, _ in rows], dtype=torch.int32, device=dev)
    n_new = [n for _, n in rows]
    starts = [0]
    for n in n_new:
        starts.append(starts[-1] + n)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    t = starts[-1]
    # every page of the cache filled by quantizing normal rows, some pages at a time
    cache = torch.empty((count, h, _page_bytes(case)), dtype=torch.uint8, device=dev)
    ends = [p * d // 2, p * (d // g) * 4, p * d // 2, p * (d // g) * 4]
    step = max(1, 2 ** 25 // (h * p * d))
    for a in range(0, count, step):
        n = min(step, count - a)
        parts = cache[a:a + n].split(ends, -1)
        for j, gain in ((0, 3.0), (2, 1.0)):
            c, sc, low = _codes(_rows(gen, (n, h, p, d), dev, gain), g)
            if j == 0:
                parts[0].copy_(_k_bytes(c).flatten(-2))
            else:
                parts[2].copy_(_v_bytes(c).unflatten(2, (p // 8, 8)).transpose(3, 4).flatten(2))
            parts[j + 1].copy_(torch.stack([sc, low], -1).permute(0, 1, 3, 4, 2).reshape(n, h, -1).view(torch.uint8))
    s["cache"] = cache
    if case["op"] == "kv":
        kind = F16 if case["x"] == "f16" else F32
        s["k"] = _rows(gen, (t, h, d), dev, 3.0).to(kind)
        s["v"] = _rows(gen, (t, h, d), dev, 1.0).to(kind)
        s["read_starts"] = s["starts"]
        s["read_rows"] = t
        if case["read"] == "all":
            s["read_starts"] = torch.tensor([0] + [n for n, _ in rows], dtype=torch.int64, device=dev).cumsum(0).to(torch.int32)
            s["read_rows"] = sum(n for n, _ in rows)
    else:
        s["q"] = (1.5 * torch.randn((t, h * case["R"], d), generator=gen, device=dev)).half()
        s["max_q"] = max(n_new)
        s["max_len"] = max(n for n, _ in rows)
    return s


# ---------------------------------------------------------------------- the plain forms

def _places(s, starts, rows):
    """(sequence, position, page, slot) of each of `rows` rows, the last rows of each sequence."""
    row = torch.arange(rows, device=starts.device)
    seq = torch.searchsorted(starts, row.to(torch.int32), right=True) - 1
    pos = s["lens"].long()[seq] - starts.long()[seq + 1] + row
    at = pos.clamp(min=0)
    p = s["case"]["P"]
    return seq, pos, s["table"].long()[seq, at // p], at % p


def _plain_norm(s):
    case, x = s["case"], s["x"].float()
    h = x if s["res"] is None else x + s["res"].float()
    t = h * s["gamma"]
    most = torch.full((), 127.0 if case["out"] == "int8" else 448.0, device=x.device)
    step = t.abs().amax(-1, keepdim=True).clamp(min=1e-10) / most
    q = t / step
    if case["out"] == "int8":
        q = torch.round(q).clamp(-127, 127)
    else:
        q = q.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    scale = step * torch.rsqrt(h.square().mean(-1, keepdim=True) + s["eps"])
    out = dict(y=(q * scale).half(), scale=scale[:, 0])
    if s["res"] is not None:
        out["residual"] = h.to(s["res"].dtype)
    return out


def _plain_kv(s):
    case = s["case"]
    _, _, page, slot = _places(s, s["starts"], s["k"].shape[0])
    _write(case, s["cache"], page, slot, s["k"], s["v"])
    _, _, page, slot = _places(s, s["read_starts"], s["read_rows"])
    k, v = _read(case, s["cache"], page, slot)
    return dict(k=k.half(), v=v.half())


def _plain_attn(s):
    case, q, starts, lens = s["case"], s["q"], s["starts"].long(), s["lens"].long()
    b, h, r, d, n = case["B"], case["Hkv"], case["R"], case["D"], s["max_q"]
    k, v = _pages(case, s["cache"], s["table"])
    rows = (starts[:-1, None] + torch.arange(n, device=q.device)).clamp(max=q.shape[0] - 1)
    qs = q[rows].float().view(b, n, h, r, d).permute(0, 2, 3, 1, 4).reshape(b, h, r * n, d)
    pos = lens[:, None] - (starts[1:] - starts[:-1])[:, None] + torch.arange(n, device=q.device)
    at = torch.arange(k.shape[2], device=q.device)
    see = at <= pos[..., None]                                 # B, n, L
    if case["window"]:
        see = see & (at > pos[..., None] - case["window"])
    see = see[:, None, None]
    a = torch.matmul(qs, k.transpose(-1, -2).contiguous()).mul_(1.0 / math.sqrt(d)).view(b, h, r, n, -1)
    a = a.masked_fill_(~see, -math.inf)
    top = a.amax(-1, keepdim=True)
    a = a.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = a.sum(-1, keepdim=True)
    v = v.masked_fill((at >= lens[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(a.view(b, h, r * n, -1), v).view(b, h, r, n, d)
    o = (o / total.masked_fill(total == 0, 1.0)).permute(0, 3, 1, 2, 4).reshape(b, n, h * r, d)
    seq, pos, _, _ = _places(s, s["starts"], q.shape[0])
    return o[seq, torch.arange(q.shape[0], device=q.device) - starts[seq]].half()


# ---------------------------------------------------------------------- the library's calls

def _own_norm(s):
    import int8_quantized_linear_amd as ql

    case = s["case"]
    call = ql.rms_norm_quantize_int8 if case["out"] == "int8" else ql.rms_norm_quantize_e4m3
    xq, scale, *res = call(s["x"], s["gamma"], s["res"], eps=s["eps"])
    codes = xq if case["out"] == "int8" else xq.to(F16)
    y = torch.empty(xq.shape, dtype=F16, device=xq.device)
    out = dict(y=torch.mul(codes, scale[:, None], out=y), scale=scale)
    if s["res"] is not None:
        out["residual"] = res[0]
    return out


def _own_kv(s):
    import int8_quantized_linear_amd as ql

    case = s["case"]
    ql.kv4_append(s["k"], s["v"], s["cache"], s["table"], s["lens"], s["starts"], page_size=case["P"], group=case["G"])
    k, v = ql.kv4_read(s["cache"], s["table"], s["lens"], s["read_starts"], s["read_rows"], head_dim=case["D"],
                       page_size=case["P"], group=case["G"])
    return dict(k=k, v=v)


def _own_attn(s):
    import int8_quantized_linear_amd as ql

    case = s["case"]
    return ql.attention_kv4(s["q"], s["cache"], s["table"], s["lens"], s["starts"], page_size=case["P"], group=case["G"],
                            max_q=s["max_q"], max_len=s["max_len"], window=case["window"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "kv": _own_kv, "attn": _own_attn}[op](state)
    return {"norm": _plain_norm, "kv": _plain_kv, "attn": _plain_attn}[op](state)


# ---------------------------------------------------------------------- work and exact

def work(case):
    if case["op"] == "norm":
        m, k = case["M"], case["K"]
        size = {"none": 0, "f16": 2, "f32": 4}
        return dict(bytes=m * k * (size[case["x"]] + 2 * size[case["res"]] + 1) + 4 * k + 4 * m, flops=8 * m * k)
    rows = _lens(case)
    row = case["Hkv"] * (case["D"] + 8 * (case["D"] // case["G"]))   # K and V of one token
    d = case["D"]
    if case["op"] == "kv":
        new = sum(n for _, n in rows)
        back = new if case["read"] == "new" else sum(n for n, _ in rows)
        size = 2 if case["x"] == "f16" else 4
        plain = 2 * case["Hkv"] * d
        return dict(bytes=new * (plain * size + row) + back * (row + plain * 2), flops=new * plain * 6 + back * plain * 2)
    seen = reach = 0
    for length, n in rows:
        first = length - n                                           # position of the first row
        w = case["window"] or length + 1
        seen += sum(min(first + i + 1, w) for i in range(n) if first + i >= 0)
        reach += length - max(0, first + 1 - w) if length else 0
    t = sum(n for _, n in rows)
    heads = case["Hkv"] * case["R"]
    return dict(bytes=reach * row + 2 * t * heads * d * 2, flops=4 * seen * heads * d)


def _exact_rows(case, cache, pages, n):
    """k and v [H, n, D] in 64 bits of the first n tokens in `pages`: every element's word and
    bit worked out by itself."""
    p, d, g, dev = case["P"], case["D"], case["G"], cache.device
    t = torch.arange(n, device=dev)
    blk = cache[pages.long()[t // p]]                          # n, H, bytes: each token's page
    e = torch.arange(d, device=dev)
    slot = (t % p)[:, None]
    i, kg, el = e // 32, e % 32 // 8, e % 8
    kbit = slot * d * 4 + (kg * (d // 32) + i) * 32 + 16 * (el % 2) + 4 * (el // 2)
    c, j = e // 64, e % 64
    quad, part = c * 16 + j % 32 // 2, 2 * (j // 32) + j % 2
    vbit = (slot // 8) * d * 32 + quad * 128 + (slot % 8) * 16 + 4 * part
    out = []
    for off, bit in ((0, kbit), (p * d // 2 + p * (d // g) * 4, vbit)):
        at = (off + bit // 8)[:, None].expand(-1, blk.shape[1], -1)
        code = (torch.gather(blk, 2, at).long() >> (bit % 8)[:, None]) & 15
        par = off + p * d // 2 + (e // g) * 4 * p + 2 * slot
        word = [torch.gather(blk, 2, (par + z)[:, None].expand_as(at)).to(torch.int32) for z in (0, 1, 2 * p, 2 * p + 1)]
        sc, low = ((word[z] | word[z + 1] << 8).to(torch.int16).view(F16).double() for z in (0, 2))
        out.append((code.double() * sc + low).transpose(0, 1))
    return out


def _exact_quantized(x, g):
    x = x.double()
    y = x.reshape(*x.shape[:-1], -1, g)
    low = y.min(-1, keepdim=True).values.half().double()
    sc = ((y.max(-1, keepdim=True).values - low) / 15).half().double().clamp(min=2.0 ** -24)
    return (low + sc * torch.round((y - low) / sc).clamp(0, 15)).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double() + (0 if s["res"] is None else s["res"].double())
        y = h * s["gamma"].double()
        a = y.abs().max(1, keepdim=True).values
        if case["out"] == "int8":
            q = torch.round(127 * y / a)
            sc = a / 127
        else:
            q = 448 * y / a
            unit = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
            q = torch.round(q / unit) * unit
            sc = a / 448
        sc = sc / torch.sqrt((h * h).mean(1, keepdim=True) + s["eps"])
        out = dict(y=q * sc, scale=sc[:, 0])
        if s["res"] is not None:
            out["residual"] = h
        return out
    rows = _lens(case)
    if case["op"] == "kv":
        kn, vn = (_exact_quantized(s[n], case["G"]) for n in ("k", "v"))
        if case["read"] == "new":
            return dict(k=kn, v=vn)
        ks, vs, at = [], [], 0
        for b, (length, n) in enumerate(rows):
            k, v = _exact_rows(case, s["cache"], s["table"][b], length)
            k, v = k.transpose(0, 1).contiguous(), v.transpose(0, 1).contiguous()
            k[length - n:], v[length - n:] = kn[at:at + n], vn[at:at + n]
            ks.append(k)
            vs.append(v)
            at += n
        return dict(k=torch.cat(ks), v=torch.cat(vs))
    h, r, d = case["Hkv"], case["R"], case["D"]
    out, at = [], 0
    for b, (length, n) in enumerate(rows):
        q = s["q"][at:at + n].double().view(n, h, r, d)
        at += n
        o = torch.zeros((n, h, r, d), dtype=torch.float64, device=q.device)
        if length:
            k, v = _exact_rows(case, s["cache"], s["table"][b], length)
            pos = torch.arange(length - n, length, device=q.device)[:, None]
            j = torch.arange(length, device=q.device)
            hide = (j > pos) | ((j <= pos - case["window"]) if case["window"] else False)
            for x in range(h):
                for y in range(r):
                    w = (q[:, x, y] @ k[x].T) / math.sqrt(d)
                    w = torch.softmax(w.masked_fill(hide, -math.inf), -1)
                    o[:, x, y] = torch.nan_to_num(w @ v[x])
        out.append(o.reshape(n, h * r, d))
    return torch.cat(out)
