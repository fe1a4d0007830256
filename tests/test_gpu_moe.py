"""moe_router and moe_e4m3_block against a plain implementation in 64 bits."""
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


def _weights(rng, E, N, K):
    """Codes and scales of normal weights, with a block of zeros and blocks of other sizes."""
    w = rng.standard_normal((E, N, K), dtype=np.float32) / np.float32(np.sqrt(K))
    w[..., :64] *= 3
    w[:, N // 2:] *= 0.5
    w[E // 2, :16] = 0
    return ref.quant_weight(w)


def _inputs(seed, T, E, K, I):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, K), dtype=np.float32)
    x[:, 3::131] *= 12
    logits = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
    return (x.astype(np.float16), logits, *_weights(rng, E, 2 * I, K), *_weights(rng, E, K, I))


def _run(ql, inp, k, renorm=True, dt=torch.float16, out=None):
    return ql.moe_e4m3_block(*map(dev, inp), top_k=k, renormalize=renorm, out_dtype=dt, out=out)


def _check(ql, inp, k, renorm, f16, bound=None):
    T, K = inp[0].shape
    dt = torch.float16 if f16 else torch.float32
    out = Guarded((T, K), dt)
    got = host(_run(ql, inp, k, renorm, dt, out.view)).astype(np.float64)
    out.check()
    want, err = ref.moe64(*inp, k, renorm) if bound is None else bound
    half = 2.0 ** -11 if f16 else 2.0 ** -24
    tol = err * (1 + half) + half * np.abs(want) + (2.0 ** -25 if f16 else 1e-37)
    diff = np.abs(got - want)
    assert (diff <= tol).all(), "%d outside, worst %g of its tolerance" % ((diff > tol).sum(), (diff / tol).max())
    return got, want


@pytest.mark.parametrize("T,E,K", [(1, 1, 64), (1, 64, 2048), (5, 7, 192), (16, 60, 1984), (17, 128, 4096), (64, 8, 320),
                                   (130, 100, 704), (3, 513, 64), (2, 16, 131008)])
def test_router(ql, T, E, K):
    rng = np.random.default_rng(T * E + K)
    x, w = rng.standard_normal((T, K)).astype(np.float16), (0.1 * rng.standard_normal((E, K))).astype(np.float16)
    out = Guarded((T, E), torch.float32)
    got = host(ql.moe_router(dev(x), dev(w), out.view))
    out.check()
    x, w = x.astype(np.float64), w.astype(np.float64)
    # a sum of K exact products in any order, a step of at most one unit an addition
    assert (np.abs(got - x @ w.T) <= (K + 16) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)).all()
    assert np.sqrt(((got - x @ w.T) ** 2).sum() / ((x @ w.T) ** 2).sum()) < 2e-6


SHAPES = [(1, 1, 1, 64, 64), (1, 8, 2, 256, 128), (1, 64, 8, 512, 192), (2, 3, 3, 64, 320), (3, 60, 4, 192, 1344),
          (7, 16, 1, 1984, 64), (16, 4, 4, 448, 448), (17, 8, 2, 320, 256), (19, 130, 6, 128, 192), (31, 3, 1, 256, 704),
          (33, 9, 3, 576, 128), (64, 2, 2, 128, 64), (64, 40, 16, 192, 128), (65, 5, 2, 128, 192), (150, 12, 3, 64, 64),
          (4, 512, 16, 64, 64), (9, 257, 5, 128, 64)]


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,K,I", SHAPES)
def test_experts(ql, T, E, k, K, I, renorm, f16):
    _check(ql, _inputs(T + E + K + I, T, E, K, I), k, renorm, f16)


def test_longer_sums(ql):
    _check(ql, _inputs(3, 3, 4, 4096, 2112), 2, True, False)
    _check(ql, _inputs(4, 40, 3, 2048, 1408), 2, False, True)


def test_ties_go_to_the_lower_expert(ql):
    T, E, k = 6, 70, 5
    inp = list(_inputs(1, T, E, 128, 128))
    lg = np.zeros((T, E), np.float32)
    lg[1] = -1
    lg[1, 60:] = 2                       # ten equal ones, the first five taken
    lg[2, 69], lg[2, 3] = 1, 1
    lg[3] = np.arange(E) // 7            # groups of equals, best last
    lg[4, ::2] = 0.0
    lg[4, 1::2] = -0.0                   # equal
    inp[1] = lg
    for renorm in (True, False):
        _check(ql, inp, k, renorm, False)


def test_masked_experts(ql):
    """-inf masks; a token may have fewer than top_k experts, or none; NaN is never chosen."""
    for T in (5, 20, 64):
        E, k = 24, 4
        inp = list(_inputs(T, T, E, 192, 128))
        lg = inp[1]
        lg[0] = -np.inf
        lg[1, :] = -np.inf
        lg[1, 17] = -3
        lg[2, ::2] = -np.inf
        lg[3, 5:] = -np.inf
        lg[4, 7] = np.nan
        lg[-1] = -np.inf
        if T == 64:
            lg[20:40] = np.nan
        for renorm in (True, False):
            got, _ = _check(ql, inp, k, renorm, False)
            assert (got[0] == 0).all() and (got[-1] == 0).all()
    lg[:] = -np.inf
    assert not host(_run(ql, inp, k)).any()


def test_large_and_small_logits(ql):
    inp = list(_inputs(2, 8, 30, 128, 128))
    inp[1] = (inp[1] * 40).astype(np.float32)
    inp[1][0] = np.float32(3e38) * np.linspace(-1, 1, 30).astype(np.float32)
    inp[1][1] = np.float32(1e-40) * np.arange(30)
    _check(ql, inp, 3, False, False)
    _check(ql, inp, 3, True, True)


def test_values_far_apart(ql):
    """h past fp16's range and far below it, at block scales from 2^-30 to 2^20."""
    rng = np.random.default_rng(0)
    inp = list(_inputs(9, 10, 6, 320, 192))
    inp[3] = (inp[3] * np.exp2(rng.integers(-10, 20, inp[3].shape))).astype(np.float32)
    inp[5] = (inp[5] * np.exp2(rng.integers(-30, 10, inp[5].shape))).astype(np.float32)
    _check(ql, inp, 2, True, False)
    inp[0] = (inp[0].astype(np.float32) * 2.0 ** -14).astype(np.float16)     # subnormal fp16 among them
    _check(ql, inp, 2, True, False)


def test_a_token_does_not_depend_on_the_others(ql):
    T, E, k = 64, 20, 4
    inp = _inputs(6, T, E, 448, 704)
    whole = _run(ql, inp, k, dt=torch.float32)
    for rows in ([0], [5, 63], list(range(15)), list(range(20, 50)), list(range(63, -1, -1))):
        part = _run(ql, (inp[0][rows], inp[1][rows], *inp[2:]), k, dt=torch.float32)
        assert torch.equal(part, whole[rows])
    for _ in range(10):
        assert torch.equal(_run(ql, inp, k, dt=torch.float32), whole)


def test_every_token_takes_one_expert(ql):
    inp = list(_inputs(8, 64, 5, 192, 128))
    inp[1][:] = np.array([0, 1, 9, 2, 3], np.float32)
    _check(ql, inp, 1, True, True)
    _check(ql, inp, 3, False, False)


def test_refusals(ql):
    inp = [dev(a) for a in _inputs(1, 3, 6, 128, 64)]
    ql.moe_e4m3_block(*inp, top_k=2)
    assert ql.moe_e4m3_block(inp[0][:0], inp[1][:0], *inp[2:], top_k=2).shape == (0, 128)
    x, lg, w13, s13, w2, s2 = inp
    for bad in ((x[:2], lg, w13, s13, w2, s2), (x, lg[:, :5], w13, s13, w2, s2), (x, lg, w13[:, :100].contiguous(), s13, w2, s2),
                (x, lg, w13, s13, w2[:5], s2), (x, lg, w13, s13[:, :, :0], w2, s2), (x, lg, w13, s13, w2, s2[:5]),
                (x, lg.cpu(), w13, s13, w2, s2), (x, lg, w13.transpose(1, 2), s13, w2, s2), (x[0], lg, w13, s13, w2, s2)):
        with pytest.raises(ValueError):
            ql.moe_e4m3_block(*bad, top_k=2)
    for bad in ((x.float(), lg, w13, s13, w2, s2), (x, lg.half(), w13, s13, w2, s2), (x, lg, w13.float(), s13, w2, s2)):
        with pytest.raises(TypeError):
            ql.moe_e4m3_block(*bad, top_k=2)
    for k in (0, 7, -1):
        with pytest.raises(ql.QLError):
            ql.moe_e4m3_block(*inp, top_k=k)
    with pytest.raises(TypeError):
        ql.moe_e4m3_block(*inp, top_k=2, out_dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ql.moe_router(x, x[:, :64].contiguous())
    with pytest.raises(TypeError):
        ql.moe_router(x, x.float())
    assert ql.moe_router(x[:0], x).shape == (0, 3)


# many tokens an expert and enough codes: the kernels whose eight waves share the tokens' operand
@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("T,E,k,K,I", [(33, 3, 2, 2048, 8256), (64, 6, 2, 1984, 4160), (70, 7, 7, 1600, 4096),
                                       (20, 2, 1, 4096, 12352), (64, 65, 16, 2112, 512)])
def test_experts_with_many_tokens(ql, T, E, k, K, I, f16):
    """Against 64 bits, with experts that all tokens, few and none take; every token as in a call of its own."""
    assert T * k >= 8 * E and E * K * I >= 40 << 20 and E * -(-I // 128) >= 192
    rng = np.random.default_rng(T + K)
    q = lambda *s: ql.quantize_weight_block_e4m3(dev(rng.standard_normal(s, dtype=np.float32) / np.float32(np.sqrt(s[-1]))))  # noqa: E731,E501
    (w13, s13), (w2, s2) = q(E, 2 * I, K), q(E, K, I)
    x = rng.standard_normal((T, K)).astype(np.float16)
    lg = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    lg[:, 0] += 4
    lg[:, E - 1] -= 5
    lg[T // 3] = -np.inf
    dt = torch.float16 if f16 else torch.float32
    out = Guarded((T, K), dt)
    args = (w13, s13, w2, s2, k, f16, dt)
    ql.moe_e4m3_block(dev(x), dev(lg), *args, out.view)
    out.check()
    some = [0, 1, T // 3, T // 2, T - 1]
    for t in some:
        assert torch.equal(ql.moe_e4m3_block(dev(x[t:t + 1]), dev(lg[t:t + 1]), *args), out.view[t:t + 1])
    inp = (x[some], lg[some], *(host(a.view(torch.uint8)) if a.dtype is not torch.float32 else host(a) for a in (w13, s13, w2, s2)))
    want, err = ref.moe64(*inp, k, f16)
    half, least = (2.0 ** -11, 2.0 ** -25) if f16 else (2.0 ** -24, 1e-37)
    diff = np.abs(host(out.view)[some].astype(np.float64) - want)
    assert (diff <= err * (1 + half) + half * np.abs(want) + least).all()


def test_many_tokens_and_no_expert(ql):
    """The wide kernels where every logit masks its expert, and where one token has one."""
    T, E, K, I = 32, 4, 2048, 6144
    q = lambda *s: ql.quantize_weight_block_e4m3(torch.randn(s, device="cuda") / s[-1] ** 0.5)  # noqa: E731
    (w13, s13), (w2, s2) = q(E, 2 * I, K), q(E, K, I)
    x, lg = torch.randn(T, K, device="cuda").half(), torch.full((T, E), float("-inf"), device="cuda")
    assert not host(ql.moe_e4m3_block(x, lg, w13, s13, w2, s2, 2)).any()
    lg[9, 3] = -2
    out = ql.moe_e4m3_block(x, lg, w13, s13, w2, s2, 2)
    assert torch.equal(out[9:10], ql.moe_e4m3_block(x[9:10], lg[9:10], w13, s13, w2, s2, 2)) and host(out[9]).any()
    assert not host(out[:9]).any() and not host(out[10:]).any()
