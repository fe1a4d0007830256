"""The norm, the 4-bit cache and the attention together with the W8A8 layers around them, as
examples/quantized_attention_block.py runs them, and each of the three on two streams and in a
replayed graph."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_util import dev, host

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ql():
    import int8_quantized_linear_amd as ql

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return ql


def test_example(ql):
    """Prompts and then single tokens through the example's block. The bound: 4-bit codes of a
    group of 64 normal values (a range of about 5 standard deviations in 15 steps) are off by
    5 / 15 / sqrt(12) = 0.1 of the values, V's by that in the output, K's through the scores by
    about as much, the int8 codes by less than 0.02: below 0.25 in all."""
    spec = importlib.util.spec_from_file_location("block", os.path.join(ROOT, "examples", "quantized_attention_block.py"))
    block = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(block)
    errors = block.run()
    assert len(errors) == 5 and max(errors) < 0.25, errors


class Path:
    """One stream's step: norm, append of two sequences' rows, read-back, decode and prompt attention."""

    def __init__(self, seed):
        rng = np.random.default_rng(seed)
        self.P, self.H, self.D, self.G = 32, 2, 128, 64
        self.b = ref.Batch(rng, [700, 41], [1, 33], self.P)
        self.one = ref.Batch(rng, [700, 41], [1, 1], self.P)
        self.meta = [dev(a) for a in self.b.arrays()]
        self.last = [self.meta[0], self.meta[1], dev(self.one.starts)]
        self.cache = dev(np.zeros((self.b.pages, self.H, ref.page_bytes(self.P, self.D, self.G)), np.uint8))
        self.fill(rng)

    def fill(self, rng):
        n = self.b.total
        new = dict(x=rng.standard_normal((n, 512)), r=rng.standard_normal((n, 512)), k=rng.standard_normal((n, self.H, self.D)),
                   v=rng.standard_normal((n, self.H, self.D)), q=rng.standard_normal((n, 4 * self.H, self.D)),
                   q1=rng.standard_normal((2, 4 * self.H, self.D)))
        for name, a in new.items():
            a = dev(a.astype(np.float16))
            if hasattr(self, name):
                getattr(self, name).copy_(a)
            else:
                setattr(self, name, a)
        self.gamma = dev(np.ones(512, np.float32)) if not hasattr(self, "gamma") else self.gamma

    def run(self, ql):
        kw = dict(page_size=self.P, group=self.G)
        out = list(ql.rms_norm_quantize_int8(self.x, self.gamma, self.r))
        out += [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
                for t in ql.rms_norm_quantize_e4m3(self.x, self.gamma, self.r)]
        ql.kv4_append(self.k, self.v, self.cache, *self.meta, **kw)
        out += ql.kv4_read(self.cache, *self.meta, self.b.total, self.D, **kw)
        out.append(ql.attention_kv4(self.q, self.cache, *self.meta, **kw, max_q=33, max_len=700))
        out.append(ql.attention_kv4(self.q1, self.cache, *self.last, **kw, max_q=1, max_len=700))
        return out


def test_two_streams(ql):
    """Two streams' steps issued in turn give, bit for bit, what each gives alone."""
    paths = [Path(1), Path(2)]
    torch.cuda.synchronize()
    alone = [[host(t) for t in p.run(ql)] for p in paths]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [None, None]
    for _ in range(4):
        for i, (s, p) in enumerate(zip(streams, paths)):
            with torch.cuda.stream(s):
                outs[i] = p.run(ql)
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        for w, t in zip(a, o):
            assert np.array_equal(host(t).view(np.uint8), w.view(np.uint8))


def test_replayed_in_a_graph(ql):
    """The step captured once and replayed over new inputs against eager runs of them, with eager
    work between the replays."""
    p = Path(3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p.run(ql)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = p.run(ql)
    torch.cuda.synchronize()
    for rep in range(3):
        p.fill(np.random.default_rng(50 + rep))
        want = [host(t).copy() for t in p.run(ql)]
        cache = host(p.cache).copy()
        p.cache.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (t, w) in enumerate(zip(outs, want)):
            if i < len(outs) - 2:   # the attention of the whole cache: only what this step wrote is there
                assert np.array_equal(host(t).view(np.uint8), w.view(np.uint8)), (rep, i)
        # with the cache as it was, the attention too
        p.cache.copy_(dev(cache))
        g.replay()
        torch.cuda.synchronize()
        for i, (t, w) in enumerate(zip(outs, want)):
            assert np.array_equal(host(t).view(np.uint8), w.view(np.uint8)), (rep, i)
