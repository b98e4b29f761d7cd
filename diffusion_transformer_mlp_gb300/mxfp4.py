"""MXFP4 (microscaled 4-bit floating point) operators: quantisation, the
block-scaled product, a paged KV cache held in 4 bits and attention over it.

    w = mxfp4_quantize(w_bf16)                               # once per weight
    y = mxfp4_linear(x, w)                                   # quantise the rows of x, then the product
    cache = empty_mxfp4_cache(pages, page_size, kv_heads, dim)
    mxfp4_cache_write(cache, k, v, slots)                    # quantise new tokens into their slots
    o = mxfp4_cache_attention(q, cache, table, lens)         # one query a sequence, or q_starts for more
    k, v = mxfp4_cache_read(cache, table, starts, total)     # whole sequences back

Each function forwards to the C entry point of the same name (mxfp4.h has the
format, the layouts and the masks); PyTorch provides device memory and the
current stream.  Calls are asynchronous on that stream, or on ``stream``.
Workspaces come from PyTorch's caching allocator; tensors used on another
stream than the one they were allocated on need ``record_stream``, as any
PyTorch tensor does.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import load

__all__ = ["MXFP4Tensor", "MXFP4Cache", "empty_mxfp4", "empty_mxfp4_cache", "mxfp4_padded_cols", "mxfp4_scale_bytes",
           "mxfp4_scale_offset", "mxfp4_quantize", "mxfp4_dequantize", "mxfp4_gemm", "mxfp4_linear",
           "mxfp4_cache_write", "mxfp4_cache_read", "mxfp4_cache_attention"]

_CODES = {torch.bfloat16: _lib.MXFP4_BF16, torch.float16: _lib.MXFP4_FP16, torch.float32: _lib.MXFP4_FP32}


def mxfp4_padded_cols(cols: int) -> int:
    return -(-cols // 128) * 128 if cols > 0 else 0


def mxfp4_scale_bytes(rows: int, cols: int) -> int:
    return -(-rows // 128) * 128 * (mxfp4_padded_cols(cols) // 32) if rows > 0 else 0


def mxfp4_scale_offset(r: int, c: int, cols: int) -> int:
    return int(load().mxfp4_scale_offset(r, c, cols))


@dataclass
class MXFP4Tensor:
    """Device MXFP4 matrix [rows, cols]: QDATA [rows, padded_cols / 2] uint8
    (further rows are ignored) and the tiled E8M0 scales."""
    qdata: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int

    @property
    def device(self) -> torch.device:
        return self.qdata.device


@dataclass
class MXFP4Cache:
    """Paged KV cache: codes [pages, kv_heads, page_size, dim / 2] and E8M0
    scales [pages, kv_heads, page_size, dim / 32] of keys and values, uint8."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor

    @property
    def device(self) -> torch.device:
        return self.k_codes.device

    @property
    def page_size(self) -> int:
        return self.k_codes.shape[2]


def empty_mxfp4(rows: int, cols: int, device="cuda") -> MXFP4Tensor:
    return MXFP4Tensor(torch.empty(rows, mxfp4_padded_cols(cols) // 2, dtype=torch.uint8, device=device),
                       torch.empty(mxfp4_scale_bytes(rows, cols), dtype=torch.uint8, device=device), rows, cols)


def empty_mxfp4_cache(pages: int, page_size: int, kv_heads: int, dim: int, device="cuda") -> MXFP4Cache:
    codes, scales = (pages, kv_heads, page_size, dim // 2), (pages, kv_heads, page_size, dim // 32)
    k, ks, v, vs = (torch.empty(s, dtype=torch.uint8, device=device) for s in (codes, scales, codes, scales))
    return MXFP4Cache(k, ks, v, vs)


def _enter(dev: torch.device, stream):
    """The raw handle of `stream` (the device's current one if None)."""
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    return (torch.cuda.current_stream(dev) if stream is None else stream).cuda_stream


def _call(dev: torch.device, name: str, *args) -> None:
    """The C entry point `name`, with `dev` current (launches go there)."""
    f = getattr(load(), name)
    if torch.cuda.current_device() == dev.index:
        st = f(*args)
    else:
        with torch.cuda.device(dev):
            st = f(*args)
    if st:
        _lib.check(st, name)


def _same_device(dev: torch.device, *ts: torch.Tensor) -> None:
    for t in ts:
        if t.device != dev:
            raise ValueError("tensors must be on one CUDA device")


def _code(dtype: torch.dtype, name: str, fp32: bool = True) -> int:
    c = _CODES.get(dtype)
    if c is None or (c == _lib.MXFP4_FP32 and not fp32):
        raise ValueError(f"{name} must be bfloat16{', float16 or float32' if fp32 else ' or float16'}")
    return c


def _matrix(x: torch.Tensor, name: str) -> int:
    c = _code(x.dtype, name)
    if x.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    if x.stride(1) != 1 and x.shape[1] > 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    return c


def _check_mxfp4(t: MXFP4Tensor, name: str) -> MXFP4Tensor:
    q, s = t.qdata, t.scales
    if q.dtype != torch.uint8 or s.dtype != torch.uint8 or not q.is_contiguous() or not s.is_contiguous():
        raise ValueError(f"{name}.qdata and {name}.scales must be contiguous uint8 tensors")
    if t.rows < 1 or t.cols < 1:
        raise ValueError(f"{name} must have rows and columns")
    if q.numel() < t.rows * (mxfp4_padded_cols(t.cols) // 2) or s.numel() < mxfp4_scale_bytes(t.rows, t.cols):
        raise ValueError(f"{name}'s buffers are too small for [{t.rows}, {t.cols}]")
    if s.device != q.device:
        raise ValueError("tensors must be on one CUDA device")
    return t


def _row_stride(x: torch.Tensor) -> int:
    return x.stride(0) if x.shape[0] > 1 else max(x.stride(0), x.shape[1])


def mxfp4_quantize(x: torch.Tensor, out: MXFP4Tensor | None = None, stream=None) -> MXFP4Tensor:
    """MXFP4 of a bfloat16, float16 or float32 matrix, one pass."""
    code = _matrix(x, "x")
    rows, cols = x.shape
    s = _enter(x.device, stream)
    if out is None:
        out = empty_mxfp4(rows, cols, x.device)
    elif out.rows != rows or out.cols != cols:
        raise ValueError(f"out holds a [{out.rows}, {out.cols}] MXFP4 tensor, [{rows}, {cols}] is needed")
    else:
        _same_device(x.device, _check_mxfp4(out, "out").qdata)
    if rows == 0 or cols == 0:
        return out
    _call(x.device, "mxfp4_quantize", x.data_ptr(), code, rows, cols, _row_stride(x), out.qdata.data_ptr(),
          out.scales.data_ptr(), s)
    return out


def _out_matrix(out, rows: int, cols: int, dtype, dev) -> torch.Tensor:
    if out is None:
        return torch.empty(rows, cols, dtype=dtype, device=dev)
    if out.shape != (rows, cols):
        raise ValueError(f"out must be [{rows}, {cols}]")
    _same_device(dev, out)
    return out


def mxfp4_dequantize(t: MXFP4Tensor, dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """The values of an MXFP4 matrix (of type out.dtype if `out` is given)."""
    if t.rows == 0 or t.cols == 0:
        return _out_matrix(out, t.rows, t.cols, dtype, t.device)
    _check_mxfp4(t, "t")
    s = _enter(t.device, stream)
    out = _out_matrix(out, t.rows, t.cols, dtype, t.device)
    code = _matrix(out, "out")
    _call(t.device, "mxfp4_dequantize", t.qdata.data_ptr(), t.scales.data_ptr(), t.rows, t.cols, out.data_ptr(), code,
          _row_stride(out), s)
    return out


def mxfp4_gemm(a: MXFP4Tensor, w: MXFP4Tensor, out: torch.Tensor | None = None, dtype: torch.dtype = torch.bfloat16,
               status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """a [m, k] times w [n, k] transposed: block-scaled FP4 tensor-core
    product, FP32 accumulation, rounded once to `dtype` (or out.dtype)."""
    if a.cols != w.cols:
        raise ValueError("activation and weight K differ")
    _check_mxfp4(a, "a")
    _check_mxfp4(w, "w")
    dev = a.device
    s = _enter(dev, stream)
    _same_device(dev, w.qdata)
    out = _out_matrix(out, a.rows, w.rows, dtype, dev)
    code = _matrix(out, "out")
    _call(dev, "mxfp4_gemm", a.qdata.data_ptr(), a.scales.data_ptr(), w.qdata.data_ptr(), w.scales.data_ptr(), a.rows,
          w.rows, a.cols, out.data_ptr(), code, _row_stride(out), None if status is None else status.data_ptr(), s)
    return out


def mxfp4_linear(x: torch.Tensor, w: MXFP4Tensor, out: torch.Tensor | None = None, dtype: torch.dtype | None = None,
                 status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """mxfp4_gemm(mxfp4_quantize(x), w) in one call; the result has x's type
    unless `out` or `dtype` says otherwise."""
    xc = _matrix(x, "x")
    m, k = x.shape
    if k != w.cols:
        raise ValueError("activation and weight K differ")
    _check_mxfp4(w, "w")
    dev = x.device
    s = _enter(dev, stream)
    _same_device(dev, w.qdata)
    out = _out_matrix(out, m, w.rows, x.dtype if dtype is None else dtype, dev)
    code = _matrix(out, "out")
    if m == 0:
        return out
    need = -(-m * mxfp4_padded_cols(k) // 512) * 256 + mxfp4_scale_bytes(m, k)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    _call(dev, "mxfp4_linear", x.data_ptr(), xc, m, _row_stride(x), w.qdata.data_ptr(), w.scales.data_ptr(), w.rows, k,
          out.data_ptr(), code, _row_stride(out), ws.data_ptr(), need, None if status is None else status.data_ptr(), s)
    return out


def _cache_struct(c: MXFP4Cache) -> _lib.CacheStruct:
    k, ks, v, vs = c.k_codes, c.k_scales, c.v_codes, c.v_scales
    shape = k.shape
    if len(shape) != 4:
        raise ValueError("cache codes must be [pages, kv_heads, page_size, dim / 2]")
    sshape = (shape[0], shape[1], shape[2], shape[3] // 16)
    if v.shape != shape or ks.shape != sshape or vs.shape != sshape:
        raise ValueError("the cache's codes and scales do not fit together")
    dev = k.device
    for t in (k, ks, v, vs):
        if t.dtype != torch.uint8 or not t.is_contiguous():
            raise ValueError("the cache's buffers must be contiguous uint8 tensors")
        if t.device != dev:
            raise ValueError("tensors must be on one CUDA device")
    return _lib.CacheStruct(k.data_ptr(), ks.data_ptr(), v.data_ptr(), vs.data_ptr(), shape[0], shape[2], shape[1],
                            shape[3] * 2, 0)


def _int_tensor(t: torch.Tensor, dtype: torch.dtype, dims: int, name: str, dev) -> None:
    if t.dtype != dtype or t.dim() != dims or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dims}-D {str(dtype).replace('torch.', '')} tensor")
    if t.device != dev:
        raise ValueError("tensors must be on one CUDA device")


def _heads(x: torch.Tensor, heads: int, dim: int, name: str) -> None:
    if x.dim() != 3 or x.shape[1] != heads or x.shape[2] != dim:
        raise ValueError(f"{name} must be [tokens, {heads}, {dim}]")
    if x.stride(2) != 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")


def mxfp4_cache_write(cache: MXFP4Cache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
    """Quantises k and v [tokens, kv_heads, dim] into slots [tokens] (int64,
    page * page_size + offset; negative slots are skipped)."""
    c = _cache_struct(cache)
    dev = cache.device
    s = _enter(dev, stream)
    _heads(k, c.kv_heads, c.dim, "k")
    _heads(v, c.kv_heads, c.dim, "v")
    if k.dtype != v.dtype or k.shape[0] != v.shape[0]:
        raise ValueError("k and v must have one type and one number of tokens")
    code = _code(k.dtype, "k")
    _int_tensor(slots, torch.int64, 1, "slots", dev)
    if slots.shape[0] != k.shape[0]:
        raise ValueError("slots must have an entry for each token")
    _same_device(dev, k, v)
    _call(dev, "mxfp4_cache_write", ctypes.addressof(c), k.data_ptr(), v.data_ptr(), code, k.shape[0], k.stride(0),
          k.stride(1), v.stride(0), v.stride(1), slots.data_ptr(), s)


def mxfp4_cache_read(cache: MXFP4Cache, table: torch.Tensor, starts: torch.Tensor, total: int,
                     dtype: torch.dtype = torch.bfloat16, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Keys and values [total, kv_heads, dim] of whole sequences: table
    [seqs, n] int32 block table, starts [seqs + 1] int32 first rows, `total`
    the last of them."""
    c = _cache_struct(cache)
    dev = cache.device
    s = _enter(dev, stream)
    code = _code(dtype, "dtype")
    _int_tensor(table, torch.int32, 2, "table", dev)
    _int_tensor(starts, torch.int32, 1, "starts", dev)
    if starts.shape[0] != table.shape[0] + 1:
        raise ValueError("starts must have an entry for each sequence and one more")
    if total < 0:
        raise ValueError("total must not be negative")
    k = torch.empty(total, c.kv_heads, c.dim, dtype=dtype, device=dev)
    v = torch.empty_like(k)
    _call(dev, "mxfp4_cache_read", ctypes.addressof(c), table.data_ptr(), table.shape[1], table.shape[0],
          starts.data_ptr(), total, k.data_ptr(), v.data_ptr(), code, s)
    return k, v


_attn_ws: dict = {}


def _attention_workspace(heads: int, q_heads: int, dim: int, max_queries: int, dev) -> int:
    key = (heads, q_heads, dim, max_queries, dev.index)
    n = _attn_ws.get(key)
    if n is None:
        n = _attn_ws[key] = int(load().mxfp4_attention_workspace_bytes(heads, q_heads, dim, max_queries))
    return n


def mxfp4_cache_attention(q: torch.Tensor, cache: MXFP4Cache, table: torch.Tensor, lens: torch.Tensor,
                          q_starts: torch.Tensor | None = None, max_queries: int | None = None,
                          scale: float | None = None, causal: bool = True, window: int = 0, sinks: int = 0,
                          out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                          status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """softmax(scale q k^T + mask) v over the cache.

    q [total, q_heads, dim] bfloat16 or float16; table [seqs, n] int32; lens
    [seqs] int32: tokens of each sequence in the cache, the new ones among
    them; q_starts [seqs + 1] int32: first query row of each sequence (None:
    one query each) with max_queries an upper bound of their number.  `scale`
    defaults to dim ** -0.5.  With window > 0 a query sees its last `window`
    keys (itself among them) and the first `sinks`.  Rows that see no key give
    zeros, and -inf in `lse` (float32 [total, q_heads], filled if given)."""
    c = _cache_struct(cache)
    dev = cache.device
    s = _enter(dev, stream)
    if q.dim() != 3 or q.shape[2] != c.dim or q.shape[1] % c.kv_heads or q.shape[1] == 0:
        raise ValueError(f"q must be [total, multiple of {c.kv_heads}, {c.dim}]")
    if q.stride(2) != 1:
        raise ValueError("q must have unit stride along its last dimension")
    code = _code(q.dtype, "q", fp32=False)
    total, heads, dim = q.shape
    _int_tensor(table, torch.int32, 2, "table", dev)
    _int_tensor(lens, torch.int32, 1, "lens", dev)
    seqs = lens.shape[0]
    if table.shape[0] != seqs:
        raise ValueError("table must have a row for each sequence")
    if q_starts is None:
        if total != seqs or max_queries not in (None, 1):
            raise ValueError("without q_starts every sequence has one query")
        max_queries = 1
    else:
        _int_tensor(q_starts, torch.int32, 1, "q_starts", dev)
        if q_starts.shape[0] != seqs + 1:
            raise ValueError("q_starts must have an entry for each sequence and one more")
        if max_queries is None:
            max_queries = total
    if max_queries < 0 or window < 0 or sinks < 0:
        raise ValueError("max_queries, window and sinks must not be negative")
    if out is None:
        out = torch.empty(total, heads, dim, dtype=q.dtype, device=dev)
    elif out.shape != q.shape or out.dtype != q.dtype or out.stride(2) != 1:
        raise ValueError("out must have q's shape and type and unit stride along its last dimension")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (total, heads) or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [total, q_heads] tensor")
    _same_device(dev, q, out)
    if total == 0 or seqs == 0 or max_queries == 0:
        return out
    max_queries = min(max_queries, total)
    need = _attention_workspace(c.kv_heads, heads, dim, max_queries, dev)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    args = _lib.AttentionStruct(q.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(),
                                table.data_ptr(), lens.data_ptr(), None if q_starts is None else q_starts.data_ptr(),
                                ws.data_ptr(), None if status is None else status.data_ptr(), q.stride(0), q.stride(1),
                                out.stride(0), out.stride(1), table.shape[1], need, seqs, total, max_queries, heads,
                                code, int(causal), min(window, 0x7FFFFFFF), min(sinks, 0x7FFFFFFF),
                                dim ** -0.5 if scale is None else scale, 0)
    _call(dev, "mxfp4_cache_attention", ctypes.addressof(c), ctypes.addressof(args), s)
    return out
