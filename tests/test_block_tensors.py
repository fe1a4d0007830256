"""The binding of the block-scaled operators refuses tensors that are not on the GPU before any call of the
library: a kernel would read their addresses (the library is replaced here, no kernel runs)."""
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def ql(monkeypatch):
    if not os.path.exists(os.path.join(ROOT, "int8_quantized_linear_amd", "libql.so")):
        pytest.skip("libql.so not built")
    import int8_quantized_linear_amd as ql

    class Library:
        def __getattr__(self, name):
            pytest.fail("lib.%s was reached" % name)

    monkeypatch.setattr(ql, "lib", Library())
    monkeypatch.setattr(ql, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(ql, "_current_device", lambda: 0)
    return ql


def _half(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def _codes(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def test_router(ql):
    x, w = _half(3, 64), _half(4, 64)
    for args in ((x, w), (x, w, torch.zeros(3, 4)), (x[:0], w), (x, w[:0])):
        with pytest.raises(ValueError, match="GPU"):
            ql.moe_router(*args)
    for bad in (None, [[1.0] * 64], 3):
        with pytest.raises(TypeError):
            ql.moe_router(bad, w)


def test_the_others(ql):
    f = torch.zeros
    for call in (lambda: ql.quantize_per_row_block_e4m3(_half(3, 64)),
                 lambda: ql.quantize_weight_block_e4m3(f(3, 64)),
                 lambda: ql.gemm_e4m3_block(_codes(3, 64), f(1, 3), _codes(5, 64), f(1, 1)),
                 lambda: ql.linear_e4m3_block(_half(3, 64), _codes(5, 64), f(1, 1)),
                 lambda: ql.moe_e4m3_block(_half(3, 64), f(3, 4), _codes(4, 128, 64), f(4, 1, 1), _codes(4, 64, 64), f(4, 1, 1), 2)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_codes_of_another_shape(ql, monkeypatch):
    """The output for the codes has x's shape, also where one of the two holds nothing (its pointer is null). CPU
    tensors stand for the GPU's here."""
    monkeypatch.setattr(ql, "_check", lambda t, *args: t)
    monkeypatch.setattr(ql, "_current_device", lambda: -1)
    for x, xq in ((_half(0, 64), _codes(0, 32)), (_half(5, 64), _codes(0, 64)), (_half(5, 64), _codes(4, 64)),
                  (_half(0, 64), _codes(5, 64))):
        with pytest.raises(ValueError, match="xq has shape"):
            ql.quantize_per_row_block_e4m3(x, xq)
