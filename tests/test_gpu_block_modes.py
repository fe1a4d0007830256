"""gemm_e4m3_block in every output mode (fp32 and fp16, without and with a bias, no activation, GELU, SiLU) by each
of its kernels. Plain fp32 outputs are held to 64 bits, all of them within a bound on what the matrix cores drop and a
sample within the closer bound of gemm64; every other mode, on every output, to what it makes of the plain ones."""
import numpy as np
import pytest
import torch

import block_ref as ref
from block_modes import MODES
from gpu_util import Guarded, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    import int8_quantized_linear_amd as ql

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return ql


def _operands(M, N, K):
    """Products of about 1.5, with zeros, and where K has them a block of zeros and a block of small values."""
    rng = np.random.default_rng(M + N + K)
    x = rng.standard_normal((M, K), dtype=np.float32)
    x[..., 5::19] = 0
    x[..., 3::67] *= 4
    if K > 256:
        x[..., 128:192] = 0
    if K > 1024:
        x[..., 256:384] *= np.float32(2.0 ** -14)
    w = rng.standard_normal((1, N, K), dtype=np.float32) * np.float32(1.5 / np.sqrt(K))
    xq, xs = ref.quant_rows(x)
    wq, ws = ref.quant_weight(w)
    return xq, xs, wq[0], ws[0], rng.standard_normal(N).astype(np.float32)


def _values(codes, scales, floor=False):
    """What E4M3 codes [n, K] with scales [n, blocks] stand for, in 64 bits; floor: magnitudes, those that are not 0 at
    least that of code 2^-6 (the exponent that the matrix cores take a subnormal code with)."""
    v = codes.view(torch.float8_e4m3fn).float().double()
    if floor:
        v = torch.where(v == 0, v, v.abs().clamp(min=2.0 ** -6))
    return v * scales.double().repeat_interleave(ref.B, 1)[:, :codes.shape[1]]


def _check_plain(xq, xs, wq, ws, y):
    """A product loses less than 2^(E - 13), E the largest sum of exponents in its group of 8: less than 2^-13 of the group's
    largest product of floored magnitudes, so a group's 8 less than 2^-10 of its sum. Then 16 groups a block, the
    scales' two roundings, blocks and up to 8 partial sums in fp32."""
    rows = ws.repeat_interleave(ref.B, 0)[:wq.shape[0]]
    want = _values(xq, xs.t()) @ _values(wq, rows).t()
    size = _values(xq, xs.t(), True) @ _values(wq, rows, True).t()
    bound = size * (2.0 ** -10 + (16 + 3 + xs.shape[0] + 8) * 2.0 ** -24)
    bad = (y.double() - want).abs() > bound
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


def _sample(n):
    rng = np.random.default_rng(n)
    return np.unique(np.concatenate([rng.integers(0, n, 12), [0, n - 1, n // 2], np.arange(max(0, n - 2), n)]))


def _activated(v, act):
    if act == "gelu":
        return v * 0.5 * torch.special.erfc(-v / 2 ** 0.5)
    return v / (1 + torch.exp(-v)) if act == "silu" else v


@pytest.mark.parametrize("M,N,K", MODES)
def test_every_mode(ql, M, N, K):
    ops = _operands(M, N, K)
    xq, xs, wq, ws, bias = map(dev, ops)

    def run(act="none", dt=torch.float32, with_bias=False):
        out = Guarded((M, N), dt)
        ql.gemm_e4m3_block(xq, xs, wq, ws, bias if with_bias else None, act, dt, out.view)
        out.check()
        return out.view

    plain = run()
    _check_plain(xq, xs, wq, ws, plain)
    r, c = _sample(M), _sample(N)
    pre, err = ref.gemm64(ops[0][r], ops[1][:, r], ops[2][c], np.repeat(ops[3], ref.B, 0)[c])
    want, tol = ref.gemm_tolerance(pre, err, None, "none", False)
    assert (np.abs(host(plain)[np.ix_(r, c)].astype(np.float64) - want) <= tol).all()

    for with_bias in (False, True):
        v = plain + bias if with_bias else plain
        assert torch.equal(run(with_bias=with_bias), v)
        assert torch.equal(run(dt=torch.float16, with_bias=with_bias), v.half())
        for act in ("gelu", "silu"):
            want = _activated(v.double(), act)
            for dt in (torch.float32, torch.float16):
                got = run(act, dt, with_bias).double()
                # as gemm_tolerance, from inputs without an error of their own
                if act == "gelu":
                    tol = (1.5e-5 if dt is torch.float16 else 2e-7) * v.double().abs()
                else:
                    tol = (v.double().abs() + 4) * 2.0 ** -23 * want.abs() + 1e-30
                half, least = (2.0 ** -11, 2.0 ** -25) if dt is torch.float16 else (2.0 ** -24, 1e-37)
                bad = (got - want).abs() > tol * (1 + half) + half * want.abs() + least
                assert not bad.any(), (act, dt, with_bias, int(bad.sum()), bad.nonzero()[:4].tolist())
