"""The block-scaled fp8 operators together, as a layer of a mixture-of-experts model calls them: each
step against 64 bits on the inputs it was given, then captured and replayed, on two streams at once, on
a workspace of any contents, with tokens that hold NaN, and at random sizes."""
import contextlib
import ctypes

import numpy as np
import pytest
import torch

import block_ref as ref
from gpu_util import DEV, Guarded, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    import int8_quantized_linear_amd as ql

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return ql


class Layer:
    """A projection, a router, experts and a projection back."""

    def __init__(self, ql, seed, K=448, H=704, E=9, I=320, top_k=3):
        rng = np.random.default_rng(seed)
        self.ql, self.K, self.top_k = ql, K, top_k
        w = lambda *s: dev(rng.standard_normal(s, dtype=np.float32) / np.float32(np.sqrt(s[-1])))  # noqa: E731
        self.w_in, self.s_in = ql.quantize_weight_block_e4m3(w(H, K))
        self.w_out, self.s_out = ql.quantize_weight_block_e4m3(w(K, H))
        self.w_router = (w(E, H) * 2).half()
        self.w13, self.s13 = ql.quantize_weight_block_e4m3(w(E, 2 * I, H))
        self.w2, self.s2 = ql.quantize_weight_block_e4m3(w(E, H, I))
        self.bias = dev(rng.standard_normal(H).astype(np.float32) * np.float32(0.1))

    def __call__(self, x, renorm=True, dt=torch.float16):
        """Every step's results, in order."""
        ql = self.ql
        xq, xs = ql.quantize_per_row_block_e4m3(x)
        h = ql.gemm_e4m3_block(xq, xs, self.w_in, self.s_in, self.bias, "silu")
        logits = ql.moe_router(h, self.w_router)
        m = ql.moe_e4m3_block(h, logits, self.w13, self.s13, self.w2, self.s2, self.top_k, renorm, dt)
        mq, ms = ql.quantize_per_row_block_e4m3(m)
        return xq, xs, h, logits, m, mq, ms, ql.gemm_e4m3_block(mq, ms, self.w_out, self.s_out, out_dtype=dt)


def _x(seed, T, K):
    return np.random.default_rng(seed).standard_normal((T, K)).astype(np.float16)


def _codes(t):
    return host(t.view(torch.uint8))


def _gemm_ok(xq, xs, wq, ws, bias, act, y, f16):
    wq = _codes(wq)
    pre, err = ref.gemm64(_codes(xq), host(xs), wq, np.repeat(host(ws), ref.B, 0)[:wq.shape[0]])
    want, tol = ref.gemm_tolerance(pre, err, bias, act, f16)
    assert (np.abs(host(y).astype(np.float64) - want) <= tol).all()


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("T", [1, 8, 40, 70, 200])
def test_every_step(ql, T, f16):
    lay = Layer(ql, T)
    x = _x(T, T, lay.K)
    xq, xs, h, logits, m, mq, ms, y = lay(dev(x), f16, torch.float16 if f16 else torch.float32)
    q, s = ref.quant_rows(x)
    assert np.array_equal(_codes(xq), q) and np.array_equal(host(xs), s)
    _gemm_ok(xq, xs, lay.w_in, lay.s_in, host(lay.bias), "silu", h, True)
    hh, w = host(h).astype(np.float64), host(lay.w_router).astype(np.float64)
    K = hh.shape[1]
    assert (np.abs(host(logits) - hh @ w.T) <= (K + 16) * 2.0 ** -23 * (np.abs(hh) @ np.abs(w).T)).all()
    want, err = ref.moe64(host(h), host(logits), _codes(lay.w13), host(lay.s13), _codes(lay.w2), host(lay.s2),
                          lay.top_k, f16)
    half, least = (2.0 ** -11, 2.0 ** -25) if f16 else (2.0 ** -24, 1e-37)
    assert (np.abs(host(m).astype(np.float64) - want) <= err * (1 + half) + half * np.abs(want) + least).all()
    q, s = ref.quant_rows(host(m))
    assert np.array_equal(_codes(mq), q) and np.array_equal(host(ms), s)
    _gemm_ok(mq, ms, lay.w_out, lay.s_out, None, "none", y, f16)


def _bits(outs):
    return [host(t.contiguous().view(torch.uint8)).copy() for t in outs]


def _same(got, want, what):
    for i, (a, b) in enumerate(zip(got, want)):
        assert np.array_equal(a, b), (what, i)


@pytest.mark.parametrize("T", [1, 17, 64, 150])
def test_replayed_in_a_graph(ql, T):
    lay = Layer(ql, 1)
    x = dev(_x(0, T, lay.K))
    w = dev(np.random.default_rng(3).standard_normal((3, 300, 256), dtype=np.float32))

    def run():
        return (*lay(x), *lay(x, False, torch.float32), *ql.quantize_weight_block_e4m3(w))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run()
    torch.cuda.synchronize()
    for rep in range(4):
        x.copy_(dev(_x(100 + rep, T, lay.K)))
        w.mul_(1.25)
        want = _bits(run())
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _same(_bits(outs), want, rep)


def test_two_graphs_of_one_pool(ql):
    """Captured into the same pool, their workspaces may be the same memory: replayed in turn."""
    lay = Layer(ql, 4)
    xs = [dev(_x(1, 5, lay.K)), dev(_x(2, 90, lay.K))]
    want = [_bits(lay(x)) for x in xs]
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=graphs[0].pool() if graphs else None):
            outs.append(lay(x))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        _same(_bits(outs[1]), want[1], 1)
        graphs[0].replay()
        torch.cuda.synchronize()
        _same(_bits(outs[0]), want[0], 0)


def test_two_streams_at_once(ql):
    lays = [Layer(ql, 5), Layer(ql, 6, K=1024, H=1344, E=20, I=192, top_k=6)]
    xs = [[dev(_x(n, T, lay.K)) for n, T in enumerate((1, 60, 130))] for lay in lays]
    want = [[_bits(lay(x)) for x in xl] for lay, xl in zip(lays, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [[], []]
    for rep in range(4):
        for n in range(3):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    outs[i].append(lays[i](xs[i][n]))
    torch.cuda.synchronize()
    for i in range(2):
        for j, out in enumerate(outs[i]):
            _same(_bits(out), want[i][j % 3], (i, j))


def test_workspace_of_any_contents(ql):
    """Exactly the documented size, any contents, left by a call of other sizes; nothing beside it written."""
    rng = np.random.default_rng(7)
    biggest = 0
    shapes = [(1, 5, 2, 192, 128), (64, 30, 4, 448, 704), (70, 3, 3, 64, 64), (9, 512, 16, 128, 192), (2, 8, 1, 1984, 64)]
    need = ctypes.c_int64(0)
    for T, E, k, K, I in shapes:
        assert ql.lib.moe_e4m3_block_workspace_bytes(T, k, K, I, ctypes.byref(need)) == 0
        biggest = max(biggest, need.value)
    pool = torch.full((biggest + 8192,), 255, dtype=torch.uint8, device=DEV)
    for T, E, k, K, I in shapes:
        q = lambda *s: ql.quantize_weight_block_e4m3(dev(rng.standard_normal(s, dtype=np.float32)))  # noqa: E731
        (w13, s13), (w2, s2) = q(E, 2 * I, K), q(E, K, I)
        x, lg = dev(_x(T, T, K)), dev(rng.standard_normal((T, E)).astype(np.float32))
        want = ql.moe_e4m3_block(x, lg, w13, s13, w2, s2, k, out_dtype=torch.float32)
        assert ql.lib.moe_e4m3_block_workspace_bytes(T, k, K, I, ctypes.byref(need)) == 0
        for fill in (None, 255, 0, 127):
            if fill is not None:
                pool.fill_(fill)
            tail = pool[4096 + need.value:].clone()
            head = pool[:4096].clone()
            out = Guarded((T, K), torch.float32)
            st = ql.lib.moe_e4m3_block(x.data_ptr(), lg.data_ptr(), w13.data_ptr(), s13.data_ptr(), w2.data_ptr(), s2.data_ptr(),
                                       out.view.data_ptr(), ql.QL_F32, T, E, k, K, I, 1, pool[4096:].data_ptr(), need.value,
                                       torch.cuda.current_stream().cuda_stream)
            assert st == 0
            assert torch.equal(out.view, want)
            out.check()
            assert torch.equal(pool[:4096], head) and torch.equal(pool[4096 + need.value:], tail)


def test_nan_stays_in_its_row(ql):
    """A padded batch may hold anything in its padding: a row's NaN and infinities reach no other row."""
    lay = Layer(ql, 8)
    for T in (6, 40, 130):
        x = _x(T, T, lay.K)
        clean = lay(dev(x))
        x[1], x[T - 2, 5], x[3, ::7] = np.nan, np.inf, -np.inf
        x[T // 2] = np.float16(65504)
        keep = [t for t in range(T) if t not in (1, 3, T - 2, T // 2)]
        for i, (a, b) in enumerate(zip(lay(dev(x)), clean)):
            a, b = (a[:, keep], b[:, keep]) if i in (1, 6) else (a[keep], b[keep])   # scales are [blocks, T]
            assert np.array_equal(host(a.contiguous().view(torch.uint8)), host(b.contiguous().view(torch.uint8))), (T, i)


def test_experts_that_none_takes_are_not_read(ql):
    lay = Layer(ql, 9, E=6)
    x = dev(_x(0, 20, lay.K))
    _, _, h, logits, m, *_ = lay(x)
    logits[:, 2] = float("-inf")
    logits[:, 5] = float("nan")
    want = ql.moe_e4m3_block(h, logits, lay.w13, lay.s13, lay.w2, lay.s2, 3)
    w13, s13, w2, s2 = (t.clone() for t in (lay.w13.view(torch.uint8), lay.s13, lay.w2.view(torch.uint8), lay.s2))
    for e in (2, 5):
        w13[e], w2[e], s13[e], s2[e] = 127, 255, float("nan"), float("inf")
    assert torch.equal(ql.moe_e4m3_block(h, logits, w13, s13, w2, s2, 3), want)


def test_random_sizes(ql):
    rng = np.random.default_rng(1234)
    for _ in range(40):
        M, N, K = int(rng.integers(1, 400)), int(rng.integers(1, 700)), 64 * int(rng.integers(1, 14))
        x = rng.standard_normal((M, K)).astype(np.float16)
        w = rng.standard_normal((N, K), dtype=np.float32) / np.float32(np.sqrt(K))
        wq, ws = ql.quantize_weight_block_e4m3(dev(w))
        xq, xs = ql.quantize_per_row_block_e4m3(dev(x))
        f16 = bool(rng.integers(2))
        dt = torch.float16 if f16 else torch.float32
        y = Guarded((M, N), dt)
        ql.gemm_e4m3_block(xq, xs, wq, ws, None, "none", dt, y.view)
        y.check()
        _gemm_ok(xq, xs, wq, ws, None, "none", y.view, f16)
    for _ in range(40):
        T, E = int(rng.integers(1, 100)), int(rng.integers(1, 40))
        k = int(rng.integers(1, min(E, 16) + 1))
        K, I = 64 * int(rng.integers(1, 9)), 64 * int(rng.integers(1, 9))
        f16, renorm = bool(rng.integers(2)), bool(rng.integers(2))
        dt = torch.float16 if f16 else torch.float32
        x = rng.standard_normal((T, K)).astype(np.float16)
        lg = rng.standard_normal((T, E)).astype(np.float32)
        lg[rng.random((T, E)) < 0.2] = -np.inf
        q = lambda *s: ql.quantize_weight_block_e4m3(dev(rng.standard_normal(s, dtype=np.float32) / np.float32(np.sqrt(s[-1]))))  # noqa: E731,E501
        (w13, s13), (w2, s2) = q(E, 2 * I, K), q(E, K, I)
        out = Guarded((T, K), dt)
        ql.moe_e4m3_block(dev(x), dev(lg), w13, s13, w2, s2, k, renorm, dt, out.view)
        out.check()
        want, err = ref.moe64(x, lg, _codes(w13), host(s13), _codes(w2), host(s2), k, renorm)
        half, least = (2.0 ** -11, 2.0 ** -25) if f16 else (2.0 ** -24, 1e-37)
        assert (np.abs(host(out.view).astype(np.float64) - want) <= err * (1 + half) + half * np.abs(want) + least).all(), \
            (T, E, k, K, I, f16, renorm)


def test_tensors_of_another_device(ql, monkeypatch):
    """With another device current, the call is made with the tensors' own."""
    lay = Layer(ql, 10)
    x = dev(_x(0, 3, lay.K))
    want = _bits(lay(x))
    entered = []

    @contextlib.contextmanager
    def device(index):
        entered.append(index)
        yield

    monkeypatch.setattr(ql, "_current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "device", device)
    _same(_bits(lay(x)), want, "")
    assert entered == [0] * 6
