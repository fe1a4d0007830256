"""The quantizers with a scale for each block of 128 (bit for bit against the definition) and
gemm_e4m3_block (against 64 bits, within what the matrix cores' sums and fp32 allow)."""
import numpy as np
import pytest
import torch

import block_ref as ref
from block_shapes import LARGE, SHAPES
from gpu_util import Guarded, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    import int8_quantized_linear_amd as ql

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return ql


def _values(rng, shape):
    """Normal values with outliers, zeros of both signs, whole blocks of zeros, tiny and large blocks."""
    x = rng.standard_normal(shape, dtype=np.float32)
    x[..., 3::41] *= 40
    x[..., ::7] *= np.float32(2.0 ** -9)
    x[..., 5::19] = 0
    x[..., 6::19] = -0.0
    if shape[-1] > 256:
        x[..., 128:256] = 0
    if shape[-1] > 512:
        x[..., 256:384] *= np.float32(2.0 ** -14)
        x[..., 384:512] *= 300
    return x


@pytest.mark.parametrize("xt", [np.float16, np.float32])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 4096), (3, 144), (16, 640), (17, 2112), (50, 11008), (333, 1072)])
def test_quantize_rows(ql, M, K, xt):
    x = _values(np.random.default_rng(M + K), (M, K)).astype(xt)
    xq, xs = Guarded((M, K), torch.uint8), Guarded((ref.blocks(K), M), torch.float32)
    got = ql.quantize_per_row_block_e4m3(dev(x), xq.view, xs.view)
    q, s = ref.quant_rows(x)
    assert np.array_equal(host(got[1]), s)
    assert np.array_equal(host(got[0]), q)
    xq.check()
    xs.check()


def test_quantize_rows_every_fp16(ql):
    """Every finite fp16 number as the second value of a block, beside maxima on both sides of a
    power of two."""
    v = np.arange(65536, dtype=np.uint16).view(np.float16)
    v = v[np.isfinite(v)]
    for top in (1.0, 447.0, 449.0, 65504.0):
        x = np.zeros((v.size, 16), np.float16)
        x[:, 0], x[:, 1] = top, v
        got = ql.quantize_per_row_block_e4m3(dev(x))
        q, s = ref.quant_rows(x)
        assert np.array_equal(host(got[1]), s)
        assert np.array_equal(host(got[0].view(torch.uint8)), q)


@pytest.mark.parametrize("shape", [(1, 16), (128, 128), (130, 272), (3, 1000, 1088), (2, 257, 144), (4096, 320)])
def test_quantize_weight(ql, shape):
    w = _values(np.random.default_rng(sum(shape)), shape)
    wq, ws = ql.quantize_weight_block_e4m3(dev(w))
    q, s = ref.quant_weight(w.reshape((-1, *shape[-2:])))
    assert wq.shape == shape and ws.shape == (*shape[:-2], ref.blocks(shape[-2]), ref.blocks(shape[-1]))
    assert np.array_equal(host(ws), s.reshape(ws.shape))
    assert np.array_equal(host(wq.view(torch.uint8)), q.reshape(shape))


def _operands(seed, M, N, K, gain=0.05):
    """Operands whose products pass fp16's range here and there; with a gain of 2^-16 they do not."""
    rng = np.random.default_rng(seed)
    xq, xs = ref.quant_rows(_values(rng, (M, K)))
    wq, ws = ref.quant_weight(_values(rng, (1, N, K)) * np.float32(gain))
    return xq, xs, wq[0], ws[0], rng.standard_normal(N).astype(np.float32)


def _check(ql, ops, act, f16, with_bias, sample=None):
    xq, xs, wq, ws, bias = ops
    M, N = xq.shape[0], wq.shape[0]
    bias = bias if with_bias else None
    dt = torch.float16 if f16 else torch.float32
    y = Guarded((M, N), dt)
    got = ql.gemm_e4m3_block(dev(xq), dev(xs), dev(wq), dev(ws), None if bias is None else dev(bias), act, dt, y.view)
    y.check()
    got = host(got).astype(np.float64)
    if f16:   # infinite from 65520 on: taken as 65536, half a step from the largest that is not
        got = np.clip(got, -65536, 65536)
    rows, cols = (np.arange(M), np.arange(N)) if sample is None else sample
    pre, err = ref.gemm64(xq[rows], xs[:, rows], wq[cols], np.repeat(ws, ref.B, 0)[cols])
    want, tol = ref.gemm_tolerance(pre, err, None if bias is None else bias[cols], act, f16)
    want = np.clip(want, -65536, 65536) if f16 else want
    diff = np.abs(got[np.ix_(rows, cols)] - want)
    assert (diff <= tol).all(), "%d outside, worst %g of its tolerance" % ((diff > tol).sum(), (diff / tol).max())


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(ql, M, N, K, f16):
    _check(ql, _operands(M * N + K, M, N, K), "none", f16, (M + N) % 2 == 0)
    _check(ql, _operands(M * N + K, M, N, K, 2.0 ** -16), "none", f16, (M + N) % 2 == 0)


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("M,N,K", [(3, 200, 256), (40, 132, 192), (150, 196, 320)])
def test_gemm_activation(ql, M, N, K, act, f16):
    _check(ql, _operands(7, M, N, K, 2.0 ** -16), act, f16, True)


@pytest.mark.parametrize("M,N,K", LARGE)
def test_gemm_sampled(ql, M, N, K):
    """Large products on a sample of rows and columns, the edges of every tile size among them."""
    rng = np.random.default_rng(M)
    pick = lambda n: np.unique(np.concatenate([rng.integers(0, n, 24), [0, n - 1, n // 2], np.arange(63, n, 64)[:3],  # noqa: E731
                                               np.arange(max(0, n - 2), n)]))
    _check(ql, _operands(N, M, N, K, 2.0 ** -16), "none", True, True, (pick(M), pick(N)))


def test_longest_k(ql):
    _check(ql, _operands(1, 2, 20, 131008), "none", False, False)
    _check(ql, _operands(2, 70, 20, 131008), "none", False, False, (np.arange(0, 70, 23), np.arange(20)))


def test_scales_apart(ql):
    """Scales of neighbouring blocks that differ by up to 2^120, and of zero."""
    for M in (3, 150):
        xq, xs, wq, ws, _ = _operands(M, M, 200, 640)
        rng = np.random.default_rng(0)
        xs = np.exp2(rng.integers(-60, 30, xs.shape)).astype(np.float32)
        ws = np.exp2(rng.integers(-60, 30, ws.shape)).astype(np.float32)
        xs[1, ::5] = 0
        _check(ql, (xq, xs, wq, ws, None), "none", False, False)


def test_all_codes(ql):
    """Every finite code against every one, subnormals and both zeros included."""
    codes = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    xq = np.zeros((254, 64), np.uint8)
    xq[:, 9] = codes
    wq = np.zeros((254, 64), np.uint8)
    wq[:, 9] = codes
    for rows in (254, 4):
        y = ql.gemm_e4m3_block(dev(xq[:rows]), dev(np.ones((1, rows), np.float32)), dev(wq),
                               dev(np.ones((2, 1), np.float32)), out_dtype=torch.float32)
        assert np.array_equal(host(y), (ref.TABLE[codes][:rows, None] * ref.TABLE[codes][None]).astype(np.float32))


def test_empty_and_refusals(ql):
    xq, xs, wq, ws, bias = map(dev, _operands(3, 4, 200, 256))
    assert ql.gemm_e4m3_block(xq[:0], xs[:, :0].contiguous(), wq, ws).shape == (0, 200)
    assert ql.gemm_e4m3_block(xq, xs, wq[:0], ws[:0]).shape == (4, 0)
    assert ql.quantize_per_row_block_e4m3(torch.empty((0, 64), device="cuda"))[0].shape == (0, 64)
    assert ql.quantize_weight_block_e4m3(torch.empty((0, 64), device="cuda"))[1].shape == (0, 1)
    for bad in (lambda: ql.gemm_e4m3_block(xq, xs.t().contiguous(), wq, ws), lambda: ql.gemm_e4m3_block(xq, xs, wq, ws[:1]),
                lambda: ql.gemm_e4m3_block(xq, xs, wq[:, :128].contiguous(), ws), lambda: ql.gemm_e4m3_block(xq, xs, wq, ws, bias[:9]),
                lambda: ql.gemm_e4m3_block(xq, xs, wq.t(), ws), lambda: ql.gemm_e4m3_block(xq, xs, wq, ws, act="relu"),
                lambda: ql.gemm_e4m3_block(xq.cpu(), xs, wq, ws)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ql.gemm_e4m3_block(xq.half(), xs, wq, ws), lambda: ql.gemm_e4m3_block(xq, xs.half(), wq, ws),
                lambda: ql.gemm_e4m3_block(xq, xs, wq, ws, out_dtype=torch.bfloat16),
                lambda: ql.quantize_per_row_block_e4m3(xq), lambda: ql.quantize_weight_block_e4m3(xs.half())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(ql.QLError):
        ql.quantize_per_row_block_e4m3(torch.zeros((2, 24), device="cuda"))
    with pytest.raises(ql.QLError):
        ql.gemm_e4m3_block(xq[:, :32].contiguous(), xs[:1], wq[:, :32].contiguous(), ws[:, :1].contiguous())


def test_linear_and_repeat(ql):
    """The whole layer on fp16 and fp32 rows, and the same bits from every repeat."""
    rng = np.random.default_rng(5)
    for M in (1, 40, 600):
        x = dev(_values(rng, (M, 1024)))
        wq, ws = ql.quantize_weight_block_e4m3(dev(_values(rng, (700, 1024))))
        y = ql.linear_e4m3_block(x, wq, ws)
        assert y.dtype == torch.float32
        xq, xs = ql.quantize_per_row_block_e4m3(x)
        for _ in range(10):
            assert torch.equal(ql.gemm_e4m3_block(xq, xs, wq, ws, out_dtype=torch.float32), y)
        assert ql.linear_e4m3_block(x.half(), wq, ws).dtype == torch.float16
