"""MXFP4 (microscaled 4-bit floating point) operators: quantisation, the
block-scaled product, a paged KV cache held in 4 bits and attention over it.

    w = mxfp4_quantize(w_bf16)                               # once per weight
    y = mxfp4_linear(x, w)                                   # quantise the rows of x, then the product
    cache = empty_mxfp4_cache(pages, page_size, kv_heads, dim)
    mxfp4_cache_write(cache, k, v, slots)                    # quantise new tokens into their slots
    o = mxfp4_cache_attention(q, cache, table, lens)         # one query a sequence, or q_starts for more
    k, v = mxfp4_cache_read(cache, table, starts, total)     # whole sequences back

Each function forwards to the C entry point of the same name (mxfp4.h has the
format, the layouts and the masks) through the compiled module _mxfp4, which
checks the arguments; PyTorch provides device memory and the current stream.
Calls are asynchronous on that stream, or on ``stream``.  Workspaces and new
outputs come from PyTorch's caching allocator and belong to the stream of the
call; outputs are recorded on the current stream as well.  The caller orders
the two streams, and calls ``record_stream`` for inputs that were allocated on
another stream than the call's, as for any PyTorch tensor.  There is no backward
pass: mxfp4_linear and mxfp4_cache_attention refuse inputs that require one.
"""
from __future__ import annotations

import ctypes
import importlib.util
import threading
from dataclasses import dataclass

import torch

from . import _lib, build

__all__ = ["MXFP4Tensor", "MXFP4Cache", "empty_mxfp4", "empty_mxfp4_cache", "mxfp4_padded_cols", "mxfp4_scale_bytes",
           "mxfp4_scale_offset", "mxfp4_quantize", "mxfp4_dequantize", "mxfp4_gemm", "mxfp4_linear",
           "mxfp4_cache_write", "mxfp4_cache_read", "mxfp4_cache_attention"]

_FUNCTIONS = ("mxfp4_quantize", "mxfp4_dequantize", "mxfp4_gemm", "mxfp4_linear_workspace_bytes", "mxfp4_linear",
              "mxfp4_cache_write", "mxfp4_cache_read", "mxfp4_attention_workspace_bytes", "mxfp4_cache_attention")
_lock = threading.Lock()


class _Unloaded:
    """Stands for the compiled module until a function of it is first used:
    loads the library and the module, which then takes its place."""

    def __getattr__(self, name: str):
        global _ext
        with _lock:
            if isinstance(_ext, _Unloaded):
                L = _lib.load()
                if not build.binding_is_current():
                    build.build()
                spec = importlib.util.spec_from_file_location("_mxfp4", build.BINDING)
                module = importlib.util.module_from_spec(spec)
                spec.loader.exec_module(module)
                module.bind(_lib.check, *(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in _FUNCTIONS))
                _ext = module
        return getattr(_ext, name)


_ext = _Unloaded()


def mxfp4_padded_cols(cols: int) -> int:
    return -(-cols // 128) * 128 if cols > 0 else 0


def mxfp4_scale_bytes(rows: int, cols: int) -> int:
    return -(-rows // 128) * 128 * (mxfp4_padded_cols(cols) // 32) if rows > 0 else 0


def mxfp4_scale_offset(r: int, c: int, cols: int) -> int:
    return int(_lib.load().mxfp4_scale_offset(r, c, cols))


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


def mxfp4_quantize(x: torch.Tensor, out: MXFP4Tensor | None = None, stream=None) -> MXFP4Tensor:
    """MXFP4 of a bfloat16, float16 or float32 matrix, one pass."""
    if out is None:
        return MXFP4Tensor(*_ext.quantize(x, None, None, stream))
    if x.shape != (out.rows, out.cols):
        raise ValueError(f"out holds a [{out.rows}, {out.cols}] MXFP4 tensor, {list(x.shape)} is needed")
    _ext.quantize(x, out.qdata, out.scales, stream)
    return out


def mxfp4_dequantize(t: MXFP4Tensor, dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """The values of an MXFP4 matrix (of type out.dtype if `out` is given)."""
    return _ext.dequantize(t.qdata, t.scales, t.rows, t.cols, dtype, out, stream)


def mxfp4_gemm(a: MXFP4Tensor, w: MXFP4Tensor, out: torch.Tensor | None = None, dtype: torch.dtype = torch.bfloat16,
               status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """a [m, k] times w [n, k] transposed: block-scaled FP4 tensor-core
    product, FP32 accumulation, rounded once to `dtype` (or out.dtype)."""
    return _ext.gemm(a.qdata, a.scales, a.rows, a.cols, w.qdata, w.scales, w.rows, w.cols, dtype, out, status, stream)


def mxfp4_linear(x: torch.Tensor, w: MXFP4Tensor, out: torch.Tensor | None = None, dtype: torch.dtype | None = None,
                 status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """mxfp4_gemm(mxfp4_quantize(x), w) in one call; the result has x's type
    unless `out` or `dtype` says otherwise."""
    return _ext.linear(x, w.qdata, w.scales, w.rows, w.cols, dtype, out, status, stream)


def mxfp4_cache_write(cache: MXFP4Cache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
    """Quantises k and v [tokens, kv_heads, dim] into slots [tokens] (int64,
    page * page_size + offset; negative slots are skipped, the others have to differ)."""
    _ext.cache_write(cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, k, v, slots, stream)


def mxfp4_cache_read(cache: MXFP4Cache, table: torch.Tensor, starts: torch.Tensor, total: int,
                     dtype: torch.dtype = torch.bfloat16, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Keys and values [total, kv_heads, dim] of whole sequences: table
    [seqs, n] int32 block table, starts [seqs + 1] int32 first rows, `total`
    the last of them."""
    return _ext.cache_read(cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, table, starts, total, dtype,
                           stream)


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
    return _ext.cache_attention(q, cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, table, lens, q_starts,
                                max_queries, scale, causal, window, sinks, out, lse, status, stream)
