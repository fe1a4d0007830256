"""rms_norm_quantize_int8 and rms_norm_quantize_e4m3 against the definition: codes, the residual
written back, and s bit for bit (each is decided by operations rounded on their own), the row's
scale within what fp32 summation of its squares allows."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_util import Guarded, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    import int8_quantized_linear_amd as ql

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return ql


def _inputs(seed, M, K, xt, rt):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K), dtype=np.float32)
    x[:, ::97] *= 30
    res = None if rt is None else (4 * rng.standard_normal((M, K), dtype=np.float32)).astype(rt)
    gamma = (1 + 0.3 * rng.standard_normal(K)).astype(np.float32)
    return x.astype(xt), res, gamma


def _check(ql, x, res, gamma, eps, e4m3, in_place=False):
    M, K = x.shape
    call = ql.rms_norm_quantize_e4m3 if e4m3 else ql.rms_norm_quantize_int8
    dr = None if res is None else dev(res)
    got = call(dev(x), dev(gamma), dr, eps=eps, res_out=dr if in_place else None)
    h, t, s = ref.norm_codes(x, res, gamma, 448 if e4m3 else 127)
    if e4m3:
        want = torch.from_numpy(np.clip(t, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(host(got[0].view(torch.uint8)), want)
    else:
        assert np.array_equal(host(got[0]), np.clip(np.rint(t), -127, 127).astype(np.int8))
    want = ref.norm_scale64(h, s, eps)
    # K positive terms in chains of K / 256 and then 10 additions deep, halved by the root; mean,
    # eps, root, reciprocal and the product round once each
    tol = ((K / 256 + 10) / 2 + 5) * 2.0 ** -24
    assert np.abs(host(got[1]).astype(np.float64) / want - 1).max() <= tol
    if res is None:
        assert len(got) == 2
    else:
        out = host(got[2])
        assert out.dtype == res.dtype
        assert np.array_equal(out, h.astype(res.dtype))
        assert (got[2].data_ptr() == dr.data_ptr()) == in_place


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rt", [None, np.float16, np.float32])
@pytest.mark.parametrize("xt", [np.float16, np.float32])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 2064), (7, 4096), (2, 11008), (5, 16400)])
def test_against_definition(ql, M, K, xt, rt, e4m3):
    _check(ql, *_inputs(M + K, M, K, xt, rt), 1e-6, e4m3)


@pytest.mark.parametrize("rt", [np.float16, np.float32])
@pytest.mark.parametrize("K", [512, 4096, 20480])
def test_in_place(ql, K, rt):
    """res_out is the residual itself, for rows kept in registers and rows read twice."""
    _check(ql, *_inputs(K, 9, K, np.float16, rt), 1e-5, False, in_place=True)


@pytest.mark.parametrize("M,K", [(2047, 4096), (70000, 64)])
def test_many_rows(ql, M, K):
    _check(ql, *_inputs(5, M, K, np.float16, np.float16), 1e-6, False)


@pytest.mark.parametrize("e4m3", [False, True])
def test_zero_rows_and_gains(ql, e4m3):
    """Rows of zeros (absmax floored at 1e-10, scale finite), gains of zero and of both signs, and
    h of the smallest fp16 numbers."""
    x, res, gamma = _inputs(3, 6, 256, np.float16, np.float16)
    x[1], res[1] = 0, 0
    x[2], res[2] = np.float16(6e-8), 0
    res[3] = -x[3]
    gamma[::3] *= -1
    gamma[5] = 0
    _check(ql, x, res, gamma, 1e-6, e4m3)
    x, _, gamma = _inputs(4, 2, 64, np.float16, None)
    _check(ql, x, None, np.zeros_like(gamma), 1e-6, e4m3)


def test_writes_only_its_outputs(ql):
    x, res, gamma = _inputs(8, 5, 1040, np.float16, np.float32)
    q, s, r = Guarded((5, 1040), torch.int8), Guarded((5,), torch.float32), Guarded((5, 1040), torch.float32)
    dx, dr, dg = dev(x), dev(res), dev(gamma)
    ql.prepare("rms_norm_quantize_int8", dx, 1, dr, 0, dg, 1e-6, 5, 1040, r.view, q.view, s.view)()
    torch.cuda.synchronize()
    for b in (q, s, r):
        b.check()


def test_feeds_the_layer(ql):
    """The codes and scales are what gemm_w8a8_per_channel takes: the layer on the norm's output
    against fp64 from the codes, within R12's bound for fp32 outputs."""
    rng = np.random.default_rng(11)
    x, res, gamma = _inputs(12, 33, 512, np.float16, np.float16)
    wq, ws = ql.quantize_weight_per_channel(dev((rng.standard_normal((96, 512)) * 0.05).astype(np.float32)))
    xq, xs, _ = ql.rms_norm_quantize_int8(dev(x), dev(gamma), dev(res))
    y = host(ql.gemm_w8a8_per_channel(xq, xs, wq, ws, None, torch.float32)).astype(np.float64)
    y64 = host(xq).astype(np.float64) @ host(wq).astype(np.float64).T
    y64 = y64 * host(xs).astype(np.float64)[:, None] * host(ws).astype(np.float64)[None]
    assert np.all(np.abs(y - y64) <= 1e-5 * np.abs(y64) + 1e-12)


def test_refusals(ql):
    x, res, gamma = (dev(a) for a in _inputs(1, 4, 64, np.float16, np.float16))
    f = ql.rms_norm_quantize_int8
    with pytest.raises(ValueError):
        f(x[0], gamma)
    with pytest.raises(ValueError):
        f(x, gamma[:32])
    with pytest.raises(TypeError):
        f(x, gamma.half())
    with pytest.raises(TypeError):
        f(x.bfloat16(), gamma)
    with pytest.raises(ValueError):
        f(x, gamma, res[:2])
    with pytest.raises(ValueError):
        f(x, gamma, None, res_out=res)
    with pytest.raises(TypeError):
        f(x, gamma, res, res_out=res.float())
    with pytest.raises(ValueError):
        f(x.t(), gamma)
    with pytest.raises(ValueError):
        f(x.cpu(), gamma.cpu())
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(ql.QLError):
            f(x, gamma, eps=eps)
    with pytest.raises(ql.QLError):
        f(dev(np.zeros((2, 24), np.float16)), dev(np.zeros(24, np.float32)))
    xq, xs = f(x[:0], gamma)
    assert xq.shape == (0, 64) and xs.shape == (0,)


def test_more_rows_than_a_launch(ql):
    """2^22 rows make one launch; the rows of the second are its own."""
    M, K = (1 << 22) + 3, 16
    x = torch.randn((M, K), device="cuda:0", dtype=torch.float16)
    res = torch.randn((M, K), device="cuda:0", dtype=torch.float32)
    gamma = torch.ones(K, device="cuda:0")
    xq, xs, h = ql.rms_norm_quantize_int8(x, gamma, res)
    pick = [0, 1, (1 << 22) - 1, 1 << 22, M - 1]
    hw, t, s = ref.norm_codes(host(x[pick]), host(res[pick]), host(gamma), 127)
    assert np.array_equal(host(xq[pick]), np.clip(np.rint(t), -127, 127).astype(np.int8))
    assert np.array_equal(host(h[pick]), hw)
    want = ref.norm_scale64(hw, s, 1e-6)
    assert np.abs(host(xs[pick]).astype(np.float64) / want - 1).max() <= ((K / 256 + 10) / 2 + 5) * 2.0 ** -24
