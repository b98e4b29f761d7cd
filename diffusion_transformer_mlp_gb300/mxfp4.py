"""MXFP4 (microscaled 4-bit floating point) operators: quantisation, the
block-scaled product, a paged KV cache held in 4 bits and attention over it;
the norm and rotary positions of heads on their way there, and the cache's pages.

    w = mxfp4_quantize(w_bf16)                               # once per weight
    y = mxfp4_linear(x, w)                                   # quantise the rows of x, then the product
    cache = empty_mxfp4_cache(pages, page_size, kv_heads, dim)
    mxfp4_cache_write(cache, k, v, slots)                    # quantise new tokens into their slots
    o = mxfp4_cache_attention(q, cache, table, lens)         # one query a sequence, or q_starts for more
    k, v = mxfp4_cache_read(cache, table, starts, total)     # whole sequences back
    q, k = head_norm_rotary(q, k, rotary, positions, wq, wk) # norm and rotation of heads
    q = mxfp4_cache_write_rotary(cache, q, k, v, slots, rotary, positions, wq, wk)  # and k, v into the cache
    pages = empty_mxfp4_pages(pages, page_size, rows, per_row)
    slots, copies, missing = mxfp4_pages_extend(pages, counts, total)  # pages for new tokens
    mxfp4_cache_copy(cache, copies)                          # of pages that others hold too
    mxfp4_pages_select(pages, sources)                       # fork, reorder and free rows
    o = mxfp4_cache_attention_shared(q, cache, table, lens, groups, shared)  # prefixes read once a group

Each function forwards to the C entry point of the same name (mxfp4.h has the
format, the layouts and the masks) through the compiled module _mxfp4, which
checks the arguments; PyTorch provides device memory and the current stream.
Calls are asynchronous on that stream, or on ``stream``.  Workspaces and new
outputs come from PyTorch's caching allocator and belong to the stream of the
call; outputs are recorded on the current stream as well.  The caller orders
the two streams, and calls ``record_stream`` for inputs that were allocated on
another stream than the call's, as for any PyTorch tensor.  There is no backward
pass: mxfp4_linear, the attention functions and those that rotate refuse inputs
that require one.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import threading
from dataclasses import dataclass

import torch

from . import _lib, build

__all__ = ["MXFP4Tensor", "MXFP4Cache", "empty_mxfp4", "empty_mxfp4_cache", "mxfp4_padded_cols", "mxfp4_scale_bytes",
           "mxfp4_scale_offset", "mxfp4_quantize", "mxfp4_dequantize", "mxfp4_gemm", "mxfp4_linear",
           "mxfp4_cache_write", "mxfp4_cache_read", "mxfp4_cache_attention", "mxfp4_cache_attention_shared",
           "HeadRotary", "head_rotary", "rotary_frequencies", "head_norm_rotary", "mxfp4_cache_write_rotary",
           "MXFP4Pages", "empty_mxfp4_pages", "mxfp4_pages_select", "mxfp4_pages_extend", "mxfp4_pages_compact",
           "mxfp4_cache_copy"]

_FUNCTIONS = ("mxfp4_quantize", "mxfp4_dequantize", "mxfp4_gemm", "mxfp4_linear_workspace_bytes", "mxfp4_linear",
              "mxfp4_cache_write", "mxfp4_cache_read", "mxfp4_attention_workspace_bytes", "mxfp4_cache_attention",
              "mxfp4_attention_shared_call_workspace_bytes", "mxfp4_cache_attention_shared", "head_norm_rotary",
              "mxfp4_cache_write_rotary", "mxfp4_pages_workspace_bytes", "mxfp4_pages_select", "mxfp4_pages_extend",
              "mxfp4_pages_compact", "mxfp4_cache_copy")
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


def mxfp4_cache_attention_shared(q: torch.Tensor, cache: MXFP4Cache, table: torch.Tensor, lens: torch.Tensor,
                                 groups: torch.Tensor, shared: torch.Tensor, q_starts: torch.Tensor | None = None,
                                 max_queries: int | None = None, max_group: int | None = None,
                                 scale: float | None = None, causal: bool = True, always: bool = False,
                                 out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                                 status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """mxfp4_cache_attention of sequences that share a prefix, which is read once
    for all queries of a group.

    groups [n + 1] int32: first sequence of each group; shared [n] int32: tokens
    that the sequences of a group have in common (their block tables name pages
    with the same bytes there, as after mxfp4_pages_select); max_group an upper
    bound of a group's queries (default: all of q; give it where most sequences are
    in no group).  Where reading the prefix by every sequence is estimated to be as
    fast (few sequences that share, small block tables), that is done, but with
    `always`; the estimate takes the tables for full, so for short prefixes in wide
    tables call mxfp4_cache_attention.  The other arguments are those of
    mxfp4_cache_attention; there is no window."""
    return _ext.cache_attention_shared(q, cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, table, lens,
                                       q_starts, max_queries, scale, causal, 0, 0, out, lse, status, stream, groups,
                                       shared, max_group, always)


@dataclass
class HeadRotary:
    """Which pairs of a head turn, by how much and with which axis' position:
    turns [pairs] int64, the frequency of each pair in units of 2^-64 turn a
    position; axis [pairs] int32 or None; interleaved: pairs are neighbours
    (2i, 2i + 1), else (i, i + pairs).  head_rotary makes one."""
    turns: torch.Tensor
    axis: torch.Tensor | None = None
    interleaved: bool = False


def rotary_frequencies(sizes, theta: float = 10000.0) -> tuple[torch.Tensor, torch.Tensor]:
    """Frequencies and axes of a head whose axes rotate sections of sizes[a]
    elements each, theta ** (-2 i / sizes[a]) for pair i of a section, in the
    order of the axes (float64 and int32, on the CPU)."""
    if any(n < 0 or n % 2 for n in sizes):
        raise ValueError("an axis rotates an even number of elements")
    freq = [float(theta) ** (-torch.arange(0, n, 2, dtype=torch.float64) / n) for n in sizes]
    axis = [torch.full((n // 2,), a, dtype=torch.int32) for a, n in enumerate(sizes)]
    return torch.cat(freq), torch.cat(axis)


def head_rotary(inv_freq: torch.Tensor, axis: torch.Tensor | None = None, interleaved: bool = False,
                device="cuda") -> HeadRotary:
    """The rotation of a head by position * inv_freq[i] radians for pair i
    (inv_freq [pairs] finite, pairs a multiple of 8), with column axis[i] of the
    positions."""
    f = inv_freq.detach().to("cpu", torch.float64)
    if f.dim() != 1 or f.numel() % 8 or not bool(torch.isfinite(f).all()):
        raise ValueError("inv_freq must be 1-D and finite, and its size a multiple of 8")
    if axis is not None and axis.shape != f.shape:
        raise ValueError("axis must have an entry for each of inv_freq")
    t = f / (2 * math.pi)
    t = (t - t.floor()) * 2.0 ** 32  # in 2^-32 turn; the second 32 bits apart
    turns = (t.floor().to(torch.int64) << 32) + ((t - t.floor()) * 2.0 ** 32).round().to(torch.int64)
    return HeadRotary(turns.to(device), None if axis is None else axis.to(device, torch.int32), interleaved)


def head_norm_rotary(q: torch.Tensor, k: torch.Tensor | None, rotary: HeadRotary, positions: torch.Tensor,
                     q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                     q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                     stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """Norm and rotation of heads, in one pass: x / sqrt(mean(x^2) + eps) *
    weight over each head (no norm without a weight), then `rotary` by positions
    [tokens, axes] (or [tokens]) int32.

    q and k [tokens, heads, dim] bfloat16, float16 or float32, any strides along
    tokens and heads; weights [dim] of the same type or float32.  The outputs may
    be q and k themselves (q_out is q, k_out is k), and share memory with nothing else."""
    return _ext.norm_rotary(q, k, rotary.turns, rotary.axis, rotary.interleaved, positions, q_weight, k_weight, eps,
                            q_out, k_out, stream)


def mxfp4_cache_write_rotary(cache: MXFP4Cache, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                             rotary: HeadRotary, positions: torch.Tensor, q_weight: torch.Tensor | None = None,
                             k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                             q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """head_norm_rotary and mxfp4_cache_write in one pass: returns the normed and
    rotated q; k goes normed, rotated and quantised (without a rounding between)
    and v quantised into slots [tokens].  bfloat16 or float16."""
    return _ext.cache_write_rotary(cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, q, k, v, slots,
                                   rotary.turns, rotary.axis, rotary.interleaved, positions, q_weight, k_weight, eps,
                                   q_out, stream)


@dataclass
class MXFP4Pages:
    """The pages of a cache, or of the caches of all layers: refs [pages] int32,
    how many rows hold each page (0: free); table [rows, n] int32; lens [rows]
    int32.  Row b of lens[b] tokens holds its first ceil(lens[b] / page_size)
    entries.  table and lens are those of the attention functions."""
    refs: torch.Tensor
    table: torch.Tensor
    lens: torch.Tensor
    page_size: int

    @property
    def device(self) -> torch.device:
        return self.refs.device


def empty_mxfp4_pages(pages: int, page_size: int, rows: int, per_row: int, device="cuda") -> MXFP4Pages:
    """A pool of free pages and `rows` empty rows of up to `per_row` pages."""
    return MXFP4Pages(torch.zeros(pages, dtype=torch.int32, device=device),
                      torch.zeros(rows, per_row, dtype=torch.int32, device=device),
                      torch.zeros(rows, dtype=torch.int32, device=device), page_size)


def mxfp4_pages_select(pages: MXFP4Pages, sources: torch.Tensor, stream=None) -> None:
    """Every row becomes what row sources[b] (int32 [rows]) was: sources[b] = b
    leaves it alone, another row forks or reorders (its pages are held by both),
    -1 frees it."""
    _ext.pages_select(pages.refs, pages.table, pages.lens, pages.page_size, sources, stream)


def mxfp4_pages_extend(pages: MXFP4Pages, counts: torch.Tensor, total: int,
                       stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Pages for counts[b] (int32 [rows]) more tokens of every row, `total` of
    them or fewer: (slots [total] int64 of the new tokens, row by row; copies
    [rows, 2] int32; missing [1] int32).  The lengths count the new tokens then.
    copies are the pages that a row goes on in although others hold them too: give
    them to mxfp4_cache_copy before the new tokens are written.  missing is 0, or
    the free pages that are lacking, or -1 where the table's rows or `total` are
    too short: nothing has changed then, and all slots are -1."""
    return _ext.pages_extend(pages.refs, pages.table, pages.lens, pages.page_size, counts, total, stream)


def mxfp4_pages_compact(pages: MXFP4Pages, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Moves the held pages to the ids 0 .. used - 1: (moves [pages // 2, 2]
    int32 for mxfp4_cache_copy, used [1] int32)."""
    return _ext.pages_compact(pages.refs, pages.table, pages.lens, pages.page_size, stream)


def mxfp4_cache_copy(cache: MXFP4Cache, pairs: torch.Tensor, source: MXFP4Cache | None = None, stream=None) -> None:
    """Copies page pairs[i, 0] of `source` (default: the cache itself) to page
    pairs[i, 1] of `cache`; pairs with a negative or too large id are skipped.  No
    page may be the target of two pairs, or target and source at once."""
    s = cache if source is None else source
    _ext.cache_copy(cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, s.k_codes, s.k_scales, s.v_codes,
                    s.v_scales, pairs, stream)
