"""Python binding of libql.so, the MI355X quantized linear layer.

Every function here has the name of a C entry point in ``include/ql.h`` and does
argument marshalling only: it checks torch tensors (device, dtype, contiguity,
shape), allocates outputs the caller did not pass, and hands raw device pointers and
the current HIP stream to the library. Every step of the computation runs in the
library's HIP kernels; there is no other code path. If the library has not been built
the import fails with an ImportError.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Tuple

import torch

__all__ = [
    "QLError", "lib", "library_path", "quantize_per_row_int8", "quantize_weight_per_channel",
    "gemm_w8a8_per_channel", "gemm_w8a8_int32", "gemm_w8a16", "gemm_w4a16_grouped",
    "quantize_weight_block_asym_u8", "quantize_weight_int4_grouped", "linear_w8a8", "prepare",
    "gemm_w8a8_per_channel_act", "gemm_w4a16_grouped_act", "ACTIVATIONS",
    "quantize_per_row_int8_asym", "weight_column_sums_i8", "gemm_w8a8_asym", "linear_w8a8_asym",
    "quantize_per_row_e4m3", "quantize_weight_per_channel_e4m3", "gemm_e4m3_per_channel",
    "linear_e4m3", "quantize_per_tensor_int8", "gemm_w8a8_requant",
    "rms_norm_quantize_int8", "rms_norm_quantize_e4m3", "kv4_page_bytes", "kv4_append", "kv4_read",
    "attention_kv4",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libql.so")

if not os.path.exists(library_path):
    raise ImportError(
        "libql.so is not built at %s; build it with `python -m int8_quantized_linear_amd.build`"
        % library_path)

lib = ctypes.CDLL(library_path)

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int
_F = ctypes.c_float

QL_F32, QL_F16 = 0, 1
# ql_activation: applied by the epilogue after the scales and the bias
ACTIVATIONS = {"none": 0, "gelu": 1, "silu": 2}
STATUS = {0: "QL_OK", 1: "QL_ERR_NULL", 2: "QL_ERR_SHAPE", 3: "QL_ERR_ALIGN", 4: "QL_ERR_DTYPE",
          5: "QL_ERR_DEVICE"}

_SIGS = {
    "quantize_per_row_int8": [_P, _I, _I64, _I64, _P, _P, _P],
    "quantize_weight_per_channel": [_P, _I64, _I64, _P, _P, _P],
    "gemm_w8a8_per_channel": [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _P],
    "gemm_w8a8_int32": [_P, _P, _P, _I64, _I64, _I64, _P],
    "gemm_w8a16": [_P, _P, _P, _P, _I64, _P, _P, _I64, _I64, _I64, _P],
    "gemm_w4a16_grouped": [_P, _P, _P, _I64, _P, _P, _I64, _I64, _I64, _P],
    "gemm_w8a8_per_channel_act": [_P, _P, _P, _P, _P, _I, _P, _I, _I64, _I64, _I64, _P],
    "gemm_w4a16_grouped_act": [_P, _P, _P, _I64, _P, _I, _P, _I64, _I64, _I64, _P],
    "quantize_per_row_int8_asym": [_P, _I, _I64, _I64, _P, _P, _P, _P],
    "weight_column_sums_i8": [_P, _I64, _I64, _P, _P],
    "gemm_w8a8_asym": [_P, _P, _P, _P, _P, _P, _P, _I, _P, _I, _I64, _I64, _I64, _P],
    "quantize_per_row_e4m3": [_P, _I, _I64, _I64, _P, _P, _P],
    "quantize_per_tensor_int8": [_P, _I, _I64, _P, _P, _P],
    "gemm_w8a8_requant": [_P, _P, _P, _P, _P, _I, _P, _I64, _P, _I64, _I64, _I64, _P],
    "quantize_weight_per_channel_e4m3": [_P, _I64, _I64, _P, _P, _P],
    "gemm_e4m3_per_channel": [_P, _P, _P, _P, _P, _I, _P, _I, _I64, _I64, _I64, _P],
    "quantize_weight_block_asym_u8": [_P, _I64, _I64, _I64, _P, _P, _P, _P],
    "quantize_weight_int4_grouped": [_P, _I64, _I64, _I64, _P, _P, _P],
    "rms_norm_quantize_int8": [_P, _I, _P, _I, _P, _F, _I64, _I64, _P, _P, _P, _P],
    "rms_norm_quantize_e4m3": [_P, _I, _P, _I, _P, _F, _I64, _I64, _P, _P, _P, _P],
    "kv4_append": [_P, _P, _I, _I64, _I64, _I64, _P, _I64, _I64, _I64, _I64, _I64, _P, _I64, _P, _P, _I64, _P],
    "kv4_read": [_P, _I64, _I64, _I64, _I64, _I64, _P, _I64, _P, _P, _I64, _I64, _I, _P, _P, _P],
    "attention_kv4": [_P, _I64, _P, _I64, _I64, _P, _I64, _I64, _I64, _I64, _I64, _P, _I64, _P, _P, _I64, _I64,
                      _I64, _F, _I64, _P, _I64, _P],
    "attention_kv4_workspace_bytes": [_I64, _I64, _I64, _I64, _I64, _I64, _I64, _I64, ctypes.POINTER(_I64)],
}
for _name, _args in _SIGS.items():
    _f = getattr(lib, _name)
    _f.argtypes = _args
    _f.restype = _I
lib.ql_status_str.argtypes = [_I]
lib.ql_status_str.restype = ctypes.c_char_p


class QLError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__("%s: %s" % (fn, lib.ql_status_str(status).decode()))


def _call(fn: str, *args):
    st = getattr(lib, fn)(*args)
    if st != 0:
        raise QLError(fn, st)


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t: torch.Tensor, name: str, dtypes, shape=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device.type != "cuda":
        raise ValueError("%s must be a GPU tensor, got %s" % (name, t.device))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.dtype not in dtypes:
        raise TypeError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous (row-major)" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    return t


def _out(t, name, shape, dtype, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _check(t, name, (dtype,), shape, device)


# ---------------------------------------------------------------- quantizers

def quantize_per_row_int8(x: torch.Tensor, xq: Optional[torch.Tensor] = None,
                          x_scale: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Per-row symmetric int8 of x [M, K] (fp16 or fp32): returns (xq int8 [M, K], x_scale fp32 [M])."""
    _check(x, "x", (torch.float16, torch.float32))
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    M, K = x.shape
    xq = _out(xq, "xq", (M, K), torch.int8, x.device)
    x_scale = _out(x_scale, "x_scale", (M,), torch.float32, x.device)
    _call("quantize_per_row_int8", _ptr(x), QL_F16 if x.dtype == torch.float16 else QL_F32, M, K,
          _ptr(xq), _ptr(x_scale), _stream(x))
    return xq, x_scale


def quantize_per_tensor_int8(x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Per-tensor symmetric int8 of x (fp16 or fp32, any shape, contiguous): (xq int8 of x's
    shape, x_scale fp32 [1])."""
    _check(x, "x", (torch.float16, torch.float32))
    xq = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    xs = torch.empty((1,), dtype=torch.float32, device=x.device)
    _call("quantize_per_tensor_int8", _ptr(x), QL_F16 if x.dtype == torch.float16 else QL_F32,
          x.numel(), _ptr(xq), _ptr(xs), _stream(x))
    return xq, xs


def quantize_per_row_int8_asym(x: torch.Tensor):
    """Asymmetric int8 per row of x [M, K] (fp16 or fp32): (xq int8 [M, K], x_scale fp32
    [M], x_zero fp32 [M]) with x ~ x_scale * (xq - x_zero)."""
    _check(x, "x", (torch.float16, torch.float32))
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    M, K = x.shape
    xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
    xs = torch.empty((M,), dtype=torch.float32, device=x.device)
    xz = torch.empty((M,), dtype=torch.float32, device=x.device)
    _call("quantize_per_row_int8_asym", _ptr(x), QL_F16 if x.dtype == torch.float16 else QL_F32, M, K,
          _ptr(xq), _ptr(xs), _ptr(xz), _stream(x))
    return xq, xs, xz


def weight_column_sums_i8(wq: torch.Tensor) -> torch.Tensor:
    """int32 [N]: the code sum of each column of W, given as its [N, K] storage."""
    _check(wq, "wq", (torch.int8,))
    N, K = wq.shape
    out = torch.empty((N,), dtype=torch.int32, device=wq.device)
    _call("weight_column_sums_i8", _ptr(wq), K, N, _ptr(out), _stream(wq))
    return out


def quantize_weight_per_channel(w_nk: torch.Tensor, wq: Optional[torch.Tensor] = None,
                                w_scale: Optional[torch.Tensor] = None):
    """Per-output-channel symmetric int8 of W [K, N] column-major, given as its [N, K]
    row-major storage (e.g. ``linear.weight``). Returns (wq int8 [N, K], w_scale fp32 [N])."""
    _check(w_nk, "w", (torch.float32,))
    N, K = w_nk.shape
    wq = _out(wq, "wq", (N, K), torch.int8, w_nk.device)
    w_scale = _out(w_scale, "w_scale", (N,), torch.float32, w_nk.device)
    _call("quantize_weight_per_channel", _ptr(w_nk), K, N, _ptr(wq), _ptr(w_scale), _stream(w_nk))
    return wq, w_scale


# E4M3 codes travel as torch.float8_e4m3fn (the OCP format) or as their raw bytes (uint8).
_FP8 = (torch.float8_e4m3fn, torch.uint8)


def quantize_per_row_e4m3(x: torch.Tensor):
    """Per-row fp8 (E4M3) of x [M, K] (fp16 or fp32): (xq float8_e4m3fn [M, K], x_scale fp32 [M])."""
    _check(x, "x", (torch.float16, torch.float32))
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    M, K = x.shape
    xq = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=x.device)
    xs = torch.empty((M,), dtype=torch.float32, device=x.device)
    _call("quantize_per_row_e4m3", _ptr(x), QL_F16 if x.dtype == torch.float16 else QL_F32, M, K,
          _ptr(xq), _ptr(xs), _stream(x))
    return xq, xs


def quantize_weight_per_channel_e4m3(w_nk: torch.Tensor):
    """Per-output-channel fp8 (E4M3) of W ([N, K] storage, fp32): (wq float8_e4m3fn [N, K],
    w_scale fp32 [N])."""
    _check(w_nk, "w", (torch.float32,))
    N, K = w_nk.shape
    wq = torch.empty((N, K), dtype=torch.float8_e4m3fn, device=w_nk.device)
    ws = torch.empty((N,), dtype=torch.float32, device=w_nk.device)
    _call("quantize_weight_per_channel_e4m3", _ptr(w_nk), K, N, _ptr(wq), _ptr(ws), _stream(w_nk))
    return wq, ws


def quantize_weight_block_asym_u8(w_nk: torch.Tensor, block: int = 64):
    """Block-asymmetric uint8 of W ([N, K] storage): (q uint8 [N, K], scale fp32 [N, K/block],
    zero_point uint8 [N, K/block])."""
    _check(w_nk, "w", (torch.float32,))
    N, K = w_nk.shape
    if block <= 0 or K % block:
        raise ValueError("block must divide K")
    dev = w_nk.device
    q = torch.empty((N, K), dtype=torch.uint8, device=dev)
    s = torch.empty((N, K // block), dtype=torch.float32, device=dev)
    z = torch.empty((N, K // block), dtype=torch.uint8, device=dev)
    _call("quantize_weight_block_asym_u8", _ptr(w_nk), K, N, block, _ptr(q), _ptr(s), _ptr(z),
          _stream(w_nk))
    return q, s, z


def quantize_weight_int4_grouped(w_nk: torch.Tensor, group: int = 128):
    """Per-group int4 of W ([N, K] storage): (packed int32 [N, K/8], scales fp16 [N, K/group])."""
    _check(w_nk, "w", (torch.float32,))
    N, K = w_nk.shape
    if group <= 0 or K % group:
        raise ValueError("group must divide K")
    dev = w_nk.device
    p = torch.empty((N, K // 8), dtype=torch.int32, device=dev)
    s = torch.empty((N, K // group), dtype=torch.float16, device=dev)
    _call("quantize_weight_int4_grouped", _ptr(w_nk), K, N, group, _ptr(p), _ptr(s), _stream(w_nk))
    return p, s


# ------------------------------------------------- norm, and the 4-bit K/V cache

def rms_norm_quantize_int8(x, gamma, residual=None, eps: float = 1e-6, res_out=None):
    """Root-mean-square norm of residual + x as int8 codes per row: x [M, K] (fp16 or fp32), gamma
    fp32 [K], residual [M, K] (fp16 or fp32) or None. Returns (xq int8 [M, K], x_scale fp32 [M])
    with x_scale * xq ~ h / sqrt(mean(h^2) + eps) * gamma, and with a residual also h = residual +
    x in the residual's dtype, written to res_out (which may be the residual, or x if that has its
    dtype) or a new tensor."""
    return _rms_norm(x, gamma, residual, eps, res_out, "rms_norm_quantize_int8", torch.int8)


def rms_norm_quantize_e4m3(x, gamma, residual=None, eps: float = 1e-6, res_out=None):
    """rms_norm_quantize_int8 with fp8 (E4M3) codes: xq is float8_e4m3fn [M, K]."""
    return _rms_norm(x, gamma, residual, eps, res_out, "rms_norm_quantize_e4m3", torch.float8_e4m3fn)


_FLOATS = (torch.float16, torch.float32)
# The stream's handle without a Stream object around it: a decode step makes these calls once a
# layer, and building the object is a sixth of a call's host time.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _same(t, name, dtype, shape, index):
    """_check for one dtype, an exact shape and a device index, quick where all is as it should be."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.shape == shape
            and t.is_contiguous()):
        _check(t, name, (dtype,), shape, torch.device("cuda", index))
    return t.data_ptr()


def _float_matrix(t, name):
    """fp16 or fp32, contiguous, on the GPU: its dtype code and pointer."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in _FLOATS and t.is_contiguous()):
        _check(t, name, _FLOATS)
    return QL_F16 if t.dtype is torch.float16 else QL_F32, t.data_ptr()


def _status(fn, st):
    if st != 0:
        raise QLError(fn, st)


def _rms_norm(x, gamma, residual, eps, res_out, fn, code_dtype):
    xdt, xp = _float_matrix(x, "x")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must be 2-D [M, K]")
    M, K = shape
    index = x.get_device()
    gp = _same(gamma, "gamma", torch.float32, (K,), index)
    rdt, rp, op = QL_F32, None, None
    if residual is not None:
        rdt, rp = _float_matrix(residual, "residual")
        rt = residual.dtype
        _same(residual, "residual", rt, shape, index)
        if res_out is None:
            res_out = torch.empty_like(residual)
        op = rp if res_out is residual else _same(res_out, "res_out", rt, shape, index)
    elif res_out is not None:
        raise ValueError("res_out needs a residual")
    xq = torch.empty_like(x, dtype=code_dtype)
    xs = gamma.new_empty((M,))
    _status(fn, getattr(lib, fn)(xp, xdt, rp, rdt, gp, eps, M, K,
                                 op, xq.data_ptr(), xs.data_ptr(), _raw_stream(index)))
    return (xq, xs) if residual is None else (xq, xs, res_out)


def kv4_page_bytes(page_size: int, head_dim: int, group: int) -> int:
    """Bytes of one page and kv head of the 4-bit K/V cache, which is a uint8 tensor
    [num_pages, kv_heads, kv4_page_bytes(...)]. Its contents need not be set before use."""
    return page_size * (head_dim + 8 * (head_dim // group))


def _check_kv4(cache, block_table, seq_lens, starts, head_dim, page_size, group):
    """Device index, batch and the pointers of the cache and of the batch's arrays."""
    _check(cache, "cache", (torch.uint8,))
    if group <= 0 or head_dim % group:
        raise ValueError("group must divide the head size")
    if cache.dim() != 3 or cache.shape[2] != kv4_page_bytes(page_size, head_dim, group):
        raise ValueError("cache has shape %s, expected [num_pages, kv_heads, %d]"
                         % (tuple(cache.shape), kv4_page_bytes(page_size, head_dim, group)))
    index = cache.get_device()
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be a 2-D tensor [batch, pages of a sequence]")
    shape = block_table.shape
    batch = shape[0]
    return (index, batch, cache.data_ptr(), _same(block_table, "block_table", torch.int32, shape, index),
            _same(seq_lens, "seq_lens", torch.int32, (batch,), index),
            _same(starts, "starts", torch.int32, (batch + 1,), index))


def _rows3(t, name, dtypes, heads, head_dim, index):
    """The row stride of a [rows, heads, head_dim] tensor, whose rows may lie apart (a slice of a
    wider projection)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.get_device() != index:
        raise ValueError("%s is on %s, expected cuda:%d" % (name, t.device, index))
    if t.dtype not in dtypes:
        raise TypeError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[2] != head_dim or (heads is not None and shape[1] != heads):
        raise ValueError("%s has shape %s, expected [rows, %s, %d]"
                         % (name, tuple(shape), "heads" if heads is None else heads, head_dim))
    if (stride[2] != 1 or (shape[1] > 1 and stride[1] != head_dim)) and t.numel():
        raise ValueError("%s must have contiguous rows" % name)
    return stride[0] if shape[0] > 1 else shape[1] * head_dim


def kv4_append(k, v, cache, block_table, seq_lens, starts, page_size: int, group: int = 64):
    """Quantizes rows of k and v [rows, kv_heads, head_dim] (fp16 or fp32; rows may lie apart) into
    the 4-bit cache. Sequence b owns rows starts[b] to starts[b + 1], its last positions;
    seq_lens (int32 [batch]) are the lengths with these rows, block_table (int32 [batch, n]) each
    sequence's pages."""
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be 3-D [rows, kv_heads, head_dim]")
    T, H, D = k.shape
    index, batch, cp, tp, lp, sp = _check_kv4(cache, block_table, seq_lens, starts, D, page_size, group)
    ks = _rows3(k, "k", _FLOATS, cache.shape[1], D, index)
    vs = _rows3(v, "v", (k.dtype,), H, D, index)
    if v.shape[0] != T:
        raise ValueError("k and v have different numbers of rows")
    _status("kv4_append", lib.kv4_append(
        k.data_ptr(), v.data_ptr(), QL_F16 if k.dtype is torch.float16 else QL_F32, ks, vs, T, cp, cache.shape[0],
        page_size, H, D, group, tp, block_table.shape[1], lp, sp, batch, _raw_stream(index)))


def kv4_read(cache, block_table, seq_lens, starts, rows: int, head_dim: int, page_size: int, group: int = 64,
             dtype=torch.float16):
    """The last starts[b + 1] - starts[b] positions of each sequence, `rows` in all, as k and v
    [rows, kv_heads, head_dim] in dtype (fp16 or fp32)."""
    index, batch, cp, tp, lp, sp = _check_kv4(cache, block_table, seq_lens, starts, head_dim, page_size, group)
    if dtype not in _FLOATS:
        raise TypeError("dtype must be float16 or float32")
    k = cache.new_empty((rows, cache.shape[1], head_dim), dtype=dtype)
    v = torch.empty_like(k)
    _status("kv4_read", lib.kv4_read(
        cp, cache.shape[0], page_size, cache.shape[1], head_dim, group, tp, block_table.shape[1], lp, sp, batch, rows,
        QL_F16 if dtype is torch.float16 else QL_F32, k.data_ptr(), v.data_ptr(), _raw_stream(index)))
    return k, v


@functools.lru_cache(maxsize=1024)
def _attention_workspace(*sizes):
    need = _I64(0)
    _call("attention_kv4_workspace_bytes", *sizes, ctypes.byref(need))
    return need.value


def attention_kv4(q, cache, block_table, seq_lens, starts, page_size: int, group: int = 64,
                  max_q: Optional[int] = None, max_len: Optional[int] = None, scale: Optional[float] = None,
                  window: int = 0, out=None):
    """Causal attention of q [rows, q_heads, head_dim] (fp16; rows may lie apart) over the 4-bit
    cache, which already holds the rows' own keys: fp16 [rows, q_heads, head_dim]. Rows, lengths
    and pages as for kv4_append; q_heads is a multiple of the cache's heads. scale defaults to
    head_dim ** -0.5; window > 0 keeps the last `window` positions of each row. max_q and max_len,
    the most rows of a sequence and the longest length, shape the launch; they default to what the
    tensors' sizes allow. Prompts and single tokens are faster in a call each than in one."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be 3-D [rows, q_heads, head_dim]")
    T, HQ, D = q.shape
    index, batch, cp, tp, lp, sp = _check_kv4(cache, block_table, seq_lens, starts, D, page_size, group)
    pages, H, _ = cache.shape
    qs = _rows3(q, "q", (torch.float16,), None, D, index)
    if H == 0 or HQ == 0 or HQ % H:
        raise ValueError("q has %d heads, not a multiple of the cache's %d" % (HQ, H))
    width = block_table.shape[1]
    if max_q is None:
        max_q = max(1, T - batch + 1)
    if max_len is None:
        max_len = max(1, width * page_size)
    if scale is None:
        scale = D ** -0.5
    if out is None:
        out = q.new_empty((T, HQ, D))
        op = out.data_ptr()
    else:
        op = _same(out, "out", torch.float16, (T, HQ, D), index)
    need = _attention_workspace(T, HQ, H, D, batch, max_q, max_len, window)
    ws = cache.new_empty((need,)) if need else None   # of the current stream, as the kernels are
    _status("attention_kv4", lib.attention_kv4(
        q.data_ptr(), qs, op, T, HQ, cp, pages, page_size, H, D, group, tp, width, lp, sp, batch, max_q, max_len,
        scale, window, None if ws is None else ws.data_ptr(), need, _raw_stream(index)))
    return out


# --------------------------------------------------------------------- GEMMs

def _act_code(act: str) -> int:
    if act not in ACTIVATIONS:
        raise ValueError("act must be one of %s" % sorted(ACTIVATIONS))
    return ACTIVATIONS[act]


def gemm_w8a8_per_channel(xq, x_scale, wq, w_scale, bias=None, out_dtype=torch.float16, y=None):
    """y [M, N] = float(xq @ wq^T) * x_scale[:, None] * w_scale[None, :] + bias."""
    return _gemm_w8a8(xq, x_scale, wq, w_scale, bias, None, out_dtype, y)


def gemm_w8a8_per_channel_act(xq, x_scale, wq, w_scale, bias=None, act: str = "gelu",
                              out_dtype=torch.float16, y=None):
    """y [M, N] = act(float(xq @ wq^T) * x_scale[:, None] * w_scale[None, :] + bias),
    act in ACTIVATIONS, applied in the GEMM's epilogue."""
    return _gemm_w8a8(xq, x_scale, wq, w_scale, bias, _act_code(act), out_dtype, y)


def _gemm_w8a8(xq, x_scale, wq, w_scale, bias, act, out_dtype, y):
    _check(xq, "xq", (torch.int8,))
    M, K = xq.shape
    dev = xq.device
    _check(wq, "wq", (torch.int8,), None, dev)
    N = wq.shape[0]
    _check(wq, "wq", (torch.int8,), (N, K), dev)
    _check(x_scale, "x_scale", (torch.float32,), (M,), dev)
    _check(w_scale, "w_scale", (torch.float32,), (N,), dev)
    if bias is not None:
        _check(bias, "bias", (torch.float32,), (N,), dev)
    if out_dtype not in (torch.float16, torch.float32):
        raise TypeError("out_dtype must be float16 or float32")
    y = _out(y, "y", (M, N), out_dtype, dev)
    ydt = QL_F16 if out_dtype == torch.float16 else QL_F32
    if act is None:
        _call("gemm_w8a8_per_channel", _ptr(xq), _ptr(x_scale), _ptr(wq), _ptr(w_scale), _ptr(bias),
              _ptr(y), ydt, M, N, K, _stream(xq))
    else:
        _call("gemm_w8a8_per_channel_act", _ptr(xq), _ptr(x_scale), _ptr(wq), _ptr(w_scale), _ptr(bias),
              act, _ptr(y), ydt, M, N, K, _stream(xq))
    return y


def gemm_w8a8_requant(xq, x_scale, wq, w_scale, out_scale, bias=None, act: str = "none", yq=None):
    """int8 [M, N]: clamp(rne(act(((acc * x_scale[m]) * w_scale[n]) + bias[n]) / out_scale), +-127)
    with out_scale fp32 of 1 (per tensor) or N (per output column) entries."""
    _check(xq, "xq", (torch.int8,))
    M, K = xq.shape
    dev = xq.device
    N = wq.shape[0]
    _check(wq, "wq", (torch.int8,), (N, K), dev)
    _check(x_scale, "x_scale", (torch.float32,), (M,), dev)
    _check(w_scale, "w_scale", (torch.float32,), (N,), dev)
    _check(out_scale, "out_scale", (torch.float32,), None, dev)
    if out_scale.dim() != 1 or out_scale.numel() not in (1, N):
        raise ValueError("out_scale must have 1 or N entries")
    if bias is not None:
        _check(bias, "bias", (torch.float32,), (N,), dev)
    yq = _out(yq, "yq", (M, N), torch.int8, dev)
    _call("gemm_w8a8_requant", _ptr(xq), _ptr(x_scale), _ptr(wq), _ptr(w_scale), _ptr(bias), _act_code(act),
          _ptr(out_scale), out_scale.numel(), _ptr(yq), M, N, K, _stream(xq))
    return yq


def gemm_w8a8_int32(xq, wq, acc=None):
    """int32 accumulators xq @ wq^T, [M, N]."""
    _check(xq, "xq", (torch.int8,))
    M, K = xq.shape
    N = wq.shape[0]
    _check(wq, "wq", (torch.int8,), (N, K), xq.device)
    acc = _out(acc, "acc", (M, N), torch.int32, xq.device)
    _call("gemm_w8a8_int32", _ptr(xq), _ptr(wq), _ptr(acc), M, N, K, _stream(xq))
    return acc


def gemm_w8a16(x, wq, w_scale, zero_point=None, group_size: int = 0, bias=None, y=None):
    """Weight-only 8-bit GEMM: x fp16 [M, K]; wq [N, K] int8 (symmetric) or uint8 (with
    zero_point); w_scale fp32 [N] (group_size 0) or [N, K/group_size]."""
    _check(x, "x", (torch.float16,))
    M, K = x.shape
    dev = x.device
    N = wq.shape[0]
    _check(wq, "wq", (torch.uint8,) if zero_point is not None else (torch.int8,), (N, K), dev)
    sshape = (N,) if group_size == 0 else (N, K // group_size)
    _check(w_scale, "w_scale", (torch.float32,), sshape, dev)
    if zero_point is not None:
        _check(zero_point, "zero_point", (torch.uint8,), sshape, dev)
    if bias is not None:
        _check(bias, "bias", (torch.float32,), (N,), dev)
    y = _out(y, "y", (M, N), torch.float16, dev)
    _call("gemm_w8a16", _ptr(x), _ptr(wq), _ptr(w_scale), _ptr(zero_point), group_size, _ptr(bias),
          _ptr(y), M, N, K, _stream(x))
    return y


def gemm_w4a16_grouped(x, wq_packed, scales, group_size: int, bias=None, y=None):
    """W4A16: x fp16 [M, K]; wq_packed int32 [N, K/8]; scales fp16 [N, K/group_size]."""
    return _gemm_w4a16(x, wq_packed, scales, group_size, bias, None, y)


def gemm_w4a16_grouped_act(x, wq_packed, scales, group_size: int, bias=None, act: str = "gelu", y=None):
    """gemm_w4a16_grouped with act (in ACTIVATIONS) fused into the epilogue."""
    return _gemm_w4a16(x, wq_packed, scales, group_size, bias, _act_code(act), y)


def _gemm_w4a16(x, wq_packed, scales, group_size, bias, act, y):
    _check(x, "x", (torch.float16,))
    M, K = x.shape
    dev = x.device
    N = wq_packed.shape[0]
    _check(wq_packed, "wq_packed", (torch.int32,), (N, K // 8), dev)
    _check(scales, "scales", (torch.float16,), (N, K // group_size) if group_size > 0 else None, dev)
    if bias is not None:
        _check(bias, "bias", (torch.float32,), (N,), dev)
    y = _out(y, "y", (M, N), torch.float16, dev)
    if act is None:
        _call("gemm_w4a16_grouped", _ptr(x), _ptr(wq_packed), _ptr(scales), group_size, _ptr(bias),
              _ptr(y), M, N, K, _stream(x))
    else:
        _call("gemm_w4a16_grouped_act", _ptr(x), _ptr(wq_packed), _ptr(scales), group_size, _ptr(bias),
              act, _ptr(y), M, N, K, _stream(x))
    return y


def gemm_w8a8_asym(xq, x_scale, x_zero, wq, w_scale, w_colsum, bias=None, act: str = "none",
                   out_dtype=torch.float16, y=None):
    """y = act(x_scale[m] w_scale[n] (xq @ wq^T - x_zero[m] w_colsum[n]) + bias[n])."""
    _check(xq, "xq", (torch.int8,))
    M, K = xq.shape
    dev = xq.device
    N = wq.shape[0]
    _check(wq, "wq", (torch.int8,), (N, K), dev)
    _check(x_scale, "x_scale", (torch.float32,), (M,), dev)
    _check(x_zero, "x_zero", (torch.float32,), (M,), dev)
    _check(w_scale, "w_scale", (torch.float32,), (N,), dev)
    _check(w_colsum, "w_colsum", (torch.int32,), (N,), dev)
    if bias is not None:
        _check(bias, "bias", (torch.float32,), (N,), dev)
    if out_dtype not in (torch.float16, torch.float32):
        raise TypeError("out_dtype must be float16 or float32")
    y = _out(y, "y", (M, N), out_dtype, dev)
    _call("gemm_w8a8_asym", _ptr(xq), _ptr(x_scale), _ptr(x_zero), _ptr(wq), _ptr(w_scale), _ptr(w_colsum),
          _ptr(bias), _act_code(act), _ptr(y), QL_F16 if out_dtype == torch.float16 else QL_F32, M, N, K,
          _stream(xq))
    return y


def gemm_e4m3_per_channel(xq, x_scale, wq, w_scale, bias=None, act: str = "none",
                          out_dtype=torch.float16, y=None):
    """y = act(x_scale[m] w_scale[n] sum_k xq[m,k] wq[n,k] + bias[n]) with E4M3 codes
    (float8_e4m3fn or uint8 tensors), fp32 accumulation."""
    _check(xq, "xq", _FP8)
    M, K = xq.shape
    dev = xq.device
    N = wq.shape[0]
    _check(wq, "wq", _FP8, (N, K), dev)
    _check(x_scale, "x_scale", (torch.float32,), (M,), dev)
    _check(w_scale, "w_scale", (torch.float32,), (N,), dev)
    if bias is not None:
        _check(bias, "bias", (torch.float32,), (N,), dev)
    if out_dtype not in (torch.float16, torch.float32):
        raise TypeError("out_dtype must be float16 or float32")
    y = _out(y, "y", (M, N), out_dtype, dev)
    _call("gemm_e4m3_per_channel", _ptr(xq), _ptr(x_scale), _ptr(wq), _ptr(w_scale), _ptr(bias),
          _act_code(act), _ptr(y), QL_F16 if out_dtype == torch.float16 else QL_F32, M, N, K,
          _stream(xq))
    return y


def linear_e4m3(x, wq, w_scale, bias=None, act: str = "none", out_dtype=None):
    """The fp8 layer: per-row E4M3 quantization of x, then the fused GEMM."""
    xq, xs = quantize_per_row_e4m3(x)
    od = out_dtype or (torch.float32 if x.dtype == torch.float32 else torch.float16)
    return gemm_e4m3_per_channel(xq, xs, wq, w_scale, bias, act, od)


def linear_w8a8_asym(x, wq, w_scale, w_colsum, bias=None, act: str = "none", out_dtype=None):
    """The layer with asymmetric per-row activations: quantize x, then the GEMM."""
    xq, xs, xz = quantize_per_row_int8_asym(x)
    od = out_dtype or (torch.float32 if x.dtype == torch.float32 else torch.float16)
    return gemm_w8a8_asym(xq, xs, xz, wq, w_scale, w_colsum, bias, act, od)


def linear_w8a8(x, wq, w_scale, bias=None, out_dtype=None):
    """The whole W8A8 layer: per-row quantization of x, then the fused GEMM."""
    xq, xs = quantize_per_row_int8(x)
    od = out_dtype or (torch.float32 if x.dtype == torch.float32 else torch.float16)
    return gemm_w8a8_per_channel(xq, xs, wq, w_scale, bias, od)


def prepare(fn: str, *args):
    """Pre-marshals one library call for repeated launches (benchmark loops): tensors
    become raw device pointers, Python ints stay sizes, and the current stream of the
    first tensor's device is captured. Returns a zero-argument callable that launches
    and raises QLError on a non-OK status. The caller keeps the tensors alive."""
    f = getattr(lib, fn)
    conv = []
    device = None
    for a in args:
        if isinstance(a, torch.Tensor):
            if a.device.type != "cuda":
                raise ValueError("prepare: tensors must be on the GPU")
            device = device or a.device
            conv.append(ctypes.c_void_p(a.data_ptr()))
        elif a is None:
            conv.append(None)
        else:
            conv.append(a)
    conv.append(ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream))

    def launch():
        st = f(*conv)
        if st != 0:
            raise QLError(fn, st)

    return launch
