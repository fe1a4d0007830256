"""The block-scaled operators at the ends of the sizes they accept, samples of the outputs against 64 bits."""
import numpy as np
import pytest
import torch

import block_ref as ref
from gpu_util import Guarded, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    import int8_quantized_linear_amd as ql

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return ql


def _normal(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("T,E,k,K,I", [(3, 2, 1, 131008, 64), (64, 3, 2, 131008, 64), (3, 2, 2, 64, 131008),
                                       (64, 16, 16, 64, 131008), (8, 512, 16, 64, 64), (1, 1, 1, 131008, 128)])
def test_experts(ql, T, E, k, K, I, f16):
    (w13, s13), (w2, s2) = (ql.quantize_weight_block_e4m3(_normal(n, *s) / s[-1] ** 0.5)
                            for n, s in enumerate(((E, 2 * I, K), (E, K, I))))
    x, lg = _normal(2, T, K).half(), _normal(3, T, E)
    dt = torch.float16 if f16 else torch.float32
    out = Guarded((T, K), dt)
    ql.moe_e4m3_block(x, lg, w13, s13, w2, s2, k, True, dt, out.view)
    out.check()
    some = sorted({0, T // 2, T - 1})
    codes = [host(a.view(torch.uint8)) if a.dtype is not torch.float32 else host(a) for a in (w13, s13, w2, s2)]
    want, err = ref.moe64(host(x)[some], host(lg)[some], *codes, k, True, h_error=2.0 ** -17 if f16 else 2.0 ** -25)
    half, least = (2.0 ** -11, 2.0 ** -25) if f16 else (2.0 ** -24, 1e-37)
    diff = np.abs(host(out.view)[some].astype(np.float64) - want)
    assert (diff <= err * (1 + half) + half * np.abs(want) + least).all()


@pytest.mark.parametrize("M,N,K", [(1, 1 << 23, 64), (40, (1 << 21) + 5, 64), ((1 << 20) + 3, 17, 64), (140000, 3, 896)])
def test_product(ql, M, N, K):
    wq, ws = ql.quantize_weight_block_e4m3(_normal(0, N, K) / K ** 0.5)
    xq, xs = ql.quantize_per_row_block_e4m3(_normal(1, M, K).half())
    rng = np.random.default_rng(M)
    pick = lambda n: np.unique(np.concatenate([rng.integers(0, n, 20), [0, n // 2, n - 1]]))  # noqa: E731
    r, c = pick(M), pick(N)
    rows, cols = dev(r), dev(c)
    ops = [host(a) for a in (xq.view(torch.uint8)[rows], xs[:, rows], wq.view(torch.uint8)[cols], ws[cols // ref.B])]
    pre, err = ref.gemm64(*ops)
    for f16 in (True, False):
        out = Guarded((M, N), torch.float16 if f16 else torch.float32)
        ql.gemm_e4m3_block(xq, xs, wq, ws, None, "none", out.view.dtype, out.view)
        out.check()
        want, tol = ref.gemm_tolerance(pre, err, None, "none", f16)
        assert (np.abs(host(out.view[rows][:, cols]).astype(np.float64) - want) <= tol).all()


@pytest.mark.parametrize("M,K", [(3, 1 << 20), ((1 << 20) + 1, 16), (1, 131008)])
def test_rows(ql, M, K):
    x = _normal(4, M, K).half()
    xq, xs = ql.quantize_per_row_block_e4m3(x)
    some = np.unique(np.concatenate([np.random.default_rng(K).integers(0, M, 50), [0, M - 1]]))
    q, s = ref.quant_rows(host(x)[some])
    assert np.array_equal(host(xq.view(torch.uint8))[some], q) and np.array_equal(host(xs)[:, some], s)
