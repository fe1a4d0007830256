"""The attention half of a decoder layer in low precision, as a serving program would run it:

    RMS norm with the residual's addition -> int8 codes -> W8A8 projection of q, k and v
    -> K and V into a paged 4-bit cache -> causal attention over that cache
    -> int8 codes per row -> W8A8 output projection

for ragged prompts at first and then for single tokens, every step on the same cache. (Position
embeddings are left out: they belong between the projection and the cache.)

    python examples/quantized_attention_block.py

runs it on random weights and prints how far its output is from the same layer in fp32 with
unquantized weights, activations and cache.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import int8_quantized_linear_amd as ql  # noqa: E402


class Weights:
    """Random projections of a layer: fp32 for the reference, int8 per output channel for the layer."""

    def __init__(self, hidden, heads, kv_heads, head_dim, device, gen):
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        width = (heads + 2 * kv_heads) * head_dim
        self.gamma = 1.0 + 0.1 * torch.randn(hidden, generator=gen, device=device)
        self.qkv = torch.randn((width, hidden), generator=gen, device=device) * hidden ** -0.5
        self.out = torch.randn((hidden, heads * head_dim), generator=gen, device=device) * (heads * head_dim) ** -0.5
        self.qkv_codes, self.qkv_scale = ql.quantize_weight_per_channel(self.qkv)
        self.out_codes, self.out_scale = ql.quantize_weight_per_channel(self.out)


class Cache:
    """A paged 4-bit cache and the page table of its sequences; pages are handed out as they fill."""

    def __init__(self, batch, max_len, w, device, page_size=16, group=64):
        self.page_size, self.group = page_size, group
        self.width = -(-max_len // page_size)
        self.data = torch.empty((batch * self.width, w.kv_heads, ql.kv4_page_bytes(page_size, w.head_dim, group)),
                                dtype=torch.uint8, device=device)
        self.free = list(range(batch * self.width))[::-1]
        self.pages = [[] for _ in range(batch)]
        self.lens = [0] * batch

    def grow(self, rows):
        """Room for rows[b] more tokens of each sequence: the batch's arrays for the calls below."""
        for b, n in enumerate(rows):
            self.lens[b] += n
            while len(self.pages[b]) * self.page_size < self.lens[b]:
                self.pages[b].append(self.free.pop())
        dev = self.data.device
        table = torch.tensor([p + [0] * (self.width - len(p)) for p in self.pages], dtype=torch.int32, device=dev)
        lens = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        starts = torch.tensor([0] + list(rows), device=dev).cumsum(0).to(torch.int32)
        return dict(block_table=table, seq_lens=lens, starts=starts, page_size=self.page_size, group=self.group)


def attention_block(x, residual, w, cache, rows):
    """x [rows, hidden], the sublayer output before (fp16), residual of the same shape: the block's
    output (fp16) and the new residual. rows[b] of the rows are the next tokens of sequence b."""
    batch = cache.grow(rows)
    codes, scale, residual = ql.rms_norm_quantize_int8(x, w.gamma, residual, eps=1e-6)
    qkv = ql.gemm_w8a8_per_channel(codes, scale, w.qkv_codes, w.qkv_scale)
    qkv = qkv.view(x.shape[0], w.heads + 2 * w.kv_heads, w.head_dim)
    q, k, v = qkv.split([w.heads, w.kv_heads, w.kv_heads], dim=1)      # views: rows lie apart
    ql.kv4_append(k, v, cache.data, **batch)
    o = ql.attention_kv4(q, cache.data, **batch, max_q=max(rows), max_len=max(cache.lens))
    return ql.linear_w8a8(o.view(x.shape[0], -1), w.out_codes, w.out_scale), residual


def reference_block(x, residual, w, past, rows):
    """The same in fp32 with nothing quantized; past[b] is a list of sequence b's (k, v) so far."""
    h = x.float() + residual.float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * w.gamma
    qkv = (y @ w.qkv.T).view(x.shape[0], -1, w.head_dim)
    q, k, v = qkv.split([w.heads, w.kv_heads, w.kv_heads], dim=1)
    out, at, group = [], 0, w.heads // w.kv_heads
    for b, n in enumerate(rows):
        past[b].append((k[at:at + n], v[at:at + n]))
        kk, vv = (torch.cat(t).repeat_interleave(group, 1).transpose(0, 1).contiguous() for t in zip(*past[b]))
        qq = q[at:at + n].transpose(0, 1).contiguous()
        s = torch.matmul(qq, kk.transpose(1, 2).contiguous()) * w.head_dim ** -0.5
        total = kk.shape[1]
        hide = torch.arange(total, device=x.device) > torch.arange(total - n, total, device=x.device)[:, None]
        o = torch.matmul(torch.softmax(s.masked_fill(hide, float("-inf")), -1), vv)
        out.append(o.transpose(0, 1).reshape(n, -1))
        at += n
    return torch.cat(out) @ w.out.T, h


def run(hidden=1024, heads=8, kv_heads=2, head_dim=128, prompts=(70, 33, 128), steps=4, seed=0):
    """Relative errors of the block's output, over the prompts and over each later token."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    w = Weights(hidden, heads, kv_heads, head_dim, dev, gen)
    cache = Cache(len(prompts), max(prompts) + steps, w, dev)
    past = [[] for _ in prompts]
    errors = []
    for step in range(1 + steps):
        rows = list(prompts) if step == 0 else [1] * len(prompts)
        x, residual = (torch.randn((sum(rows), hidden), generator=gen, device=dev).half() for _ in range(2))
        got, new = attention_block(x, residual, w, cache, rows)
        want, h = reference_block(x, residual, w, past, rows)
        errors.append(float((got.float() - want).norm() / want.norm()))
        assert torch.equal(new, h.half())
    return errors


if __name__ == "__main__":
    for i, e in enumerate(run()):
        print("%-8s relative error against the unquantized layer %.3f" % ("prompts" if i == 0 else "token %d" % i, e))
