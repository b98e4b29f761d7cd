"""The MXFP4 entry points without a GPU: sizes, and argument errors that come
back before any CUDA call (the pointers below are never dereferenced)."""
import ctypes
import math

import pytest

import diffusion_transformer_mlp_gb300 as fc2
from diffusion_transformer_mlp_gb300 import _lib

P16, P8, P1 = (ctypes.c_void_p(v) for v in (0x10000, 0x10008, 0x10001))
NUL = ctypes.c_void_p(0)
BF16, FP16, FP32 = 0, 1, 2
INVALID, UNSUPPORTED, ALIGN = _lib.NVFP4_EINVAL, _lib.NVFP4_EUNSUPPORTED, _lib.NVFP4_EALIGN


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (127, 128), (129, 129), (37810, 14336), (300, 14300)])
def test_sizes(rows, cols):
    L = _lib.load()
    pad = -(-cols // 128) * 128
    assert fc2.mxfp4_padded_cols(cols) == L.mxfp4_padded_cols(cols) == pad
    assert L.mxfp4_qdata_bytes(rows, cols) == rows * pad // 2
    assert fc2.mxfp4_scale_bytes(rows, cols) == L.mxfp4_scale_bytes(rows, cols) == -(-rows // 128) * 128 * pad // 32
    seen = set()
    for r in {0, rows - 1, rows // 2, min(rows - 1, 33)}:
        for c in {0, -(-cols // 32) - 1, cols // 64}:
            at = fc2.mxfp4_scale_offset(r, c, cols)
            assert 0 <= at < fc2.mxfp4_scale_bytes(rows, cols)
            seen.add((at, r, c))
    assert len({at for at, _, _ in seen}) == len(seen)


def test_empty_sizes():
    L = _lib.load()
    assert L.mxfp4_padded_cols(0) == 0 and L.mxfp4_qdata_bytes(0, 64) == 0 and L.mxfp4_scale_bytes(-3, 64) == 0
    assert L.mxfp4_linear_workspace_bytes(0, 64) == 0
    assert L.mxfp4_attention_workspace_bytes(0, 8, 64, 1) == 0 and L.mxfp4_attention_workspace_bytes(1, 8, 96, 1) == 0


def test_linear_workspace_holds_the_quantised_rows():
    L = _lib.load()
    for m, k in ((1, 100), (300, 14336), (37810, 14336)):
        need = L.mxfp4_qdata_bytes(m, k) + L.mxfp4_scale_bytes(m, k)
        assert L.mxfp4_linear_workspace_bytes(m, k) in range(need, need + 1024) or m <= 32


def test_quantise_and_dequantise():
    L = _lib.load()
    q = L.mxfp4_quantize
    assert q(NUL, BF16, 4, 64, 64, P16, P16, NUL) == INVALID
    assert q(P16, BF16, 4, 64, 64, NUL, P16, NUL) == INVALID
    assert q(P16, 3, 4, 64, 64, P16, P16, NUL) == INVALID            # element type
    assert q(P16, BF16, 0, 64, 64, P16, P16, NUL) == INVALID
    assert q(P16, BF16, 4, 0, 64, P16, P16, NUL) == INVALID
    assert q(P16, BF16, 4, 64, 63, P16, P16, NUL) == INVALID         # stride below a row
    assert q(P16, BF16, 4, (1 << 24) + 1, 1 << 25, P16, P16, NUL) == UNSUPPORTED
    assert q(P16, BF16, 1 << 40, 64, 64, P16, P16, NUL) == UNSUPPORTED
    assert q(P1, BF16, 4, 64, 64, P16, P16, NUL) == ALIGN
    assert q(P16, BF16, 4, 64, 64, P8, P16, NUL) == ALIGN
    assert "mxfp4_quantize" in _lib.last_error()
    d = L.mxfp4_dequantize
    assert d(P16, NUL, 4, 64, P16, BF16, 64, NUL) == INVALID
    assert d(P16, P16, 4, 64, P16, 7, 64, NUL) == INVALID
    assert d(P16, P16, 4, 64, P16, BF16, 60, NUL) == INVALID
    assert d(P16, P8, 4, 64, P16, BF16, 64, NUL) == ALIGN
    assert d(P16, P16, 4, 64, P1, FP32, 64, NUL) == ALIGN


def test_products():
    L = _lib.load()
    ok = [P16] * 4
    g = L.mxfp4_gemm
    assert g(NUL, *ok[1:], 4, 8, 64, P16, BF16, 8, NUL, NUL) == INVALID
    assert g(*ok, 0, 8, 64, P16, BF16, 8, NUL, NUL) == INVALID
    assert g(*ok, 4, 8, 64, P16, BF16, 7, NUL, NUL) == INVALID       # stride below a row
    assert g(*ok, 4, 8, 64, P16, 9, 8, NUL, NUL) == INVALID
    assert g(*ok, 4, 8, (1 << 24) + 1, P16, BF16, 8, NUL, NUL) == UNSUPPORTED
    assert g(P8, *ok[1:], 4, 8, 64, P16, BF16, 8, NUL, NUL) == ALIGN
    assert g(*ok, 4, 8, 64, P1, BF16, 8, NUL, NUL) == ALIGN
    lin = L.mxfp4_linear
    assert lin(NUL, BF16, 400, 64, P16, P16, 8, 64, P16, BF16, 8, P16, 1 << 30, NUL, NUL) == INVALID
    assert lin(P16, BF16, 400, 60, P16, P16, 8, 64, P16, BF16, 8, P16, 1 << 30, NUL, NUL) == INVALID
    assert lin(P16, 5, 400, 64, P16, P16, 8, 64, P16, BF16, 8, P16, 1 << 30, NUL, NUL) == INVALID
    assert lin(P16, BF16, 400, 64, P16, P16, 8, 64, P16, BF16, 8, P16, 16, NUL, NUL) == INVALID  # workspace too small
    assert lin(P16, BF16, 400, 64, P16, P16, 8, 64, P16, BF16, 8, P8, 1 << 30, NUL, NUL) == ALIGN


class Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "k_scales", "v_codes", "v_scales")] + \
        [("pages", ctypes.c_int64)] + [(n, ctypes.c_int32) for n in ("page_size", "kv_heads", "dim", "reserved")]


class Attention(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "out", "lse", "table", "lens", "q_starts", "workspace",
                                               "dev_status")] + \
        [(n, ctypes.c_int64) for n in ("q_st", "q_sh", "o_st", "o_sh", "table_ld", "workspace_bytes")] + \
        [(n, ctypes.c_int32) for n in ("seqs", "total_q", "max_queries", "q_heads", "dtype", "causal", "window",
                                       "sinks")] + [("scale", ctypes.c_float), ("reserved", ctypes.c_int32)]


def _cache(**kw):
    c = Cache()
    for f in ("k_codes", "k_scales", "v_codes", "v_scales"):
        setattr(c, f, 0x10000)
    c.pages, c.page_size, c.kv_heads, c.dim = 16, 16, 2, 64
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [(dict(k_codes=None), INVALID), (dict(v_scales=None), INVALID), (dict(pages=0), INVALID),
              (dict(kv_heads=0), INVALID), (dict(page_size=24), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
              (dict(page_size=512), UNSUPPORTED), (dict(dim=96), UNSUPPORTED), (dict(kv_heads=70000), UNSUPPORTED),
              (dict(pages=1 << 31), UNSUPPORTED), (dict(v_codes=0x10008), ALIGN)]


def test_cache_write_and_read():
    L = _lib.load()
    by = ctypes.byref
    w = lambda c, k=P16, v=P16, dt=BF16, n=3, slots=P16: L.mxfp4_cache_write(by(c), k, v, dt, n, 128, 64, 128, 64, slots,
                                                                             NUL)
    r = lambda c, table=P16, ld=4, seqs=2, starts=P16, total=9, k=P16, dt=BF16: L.mxfp4_cache_read(
        by(c), table, ld, seqs, starts, total, k, P16, dt, NUL)
    for kw, err in BAD_CACHES:
        assert w(_cache(**kw)) == err and r(_cache(**kw)) == err, kw
    c = _cache()
    assert w(c, dt=4) == INVALID and w(c, n=-1) == INVALID and w(c, k=NUL) == INVALID and w(c, slots=NUL) == INVALID
    assert w(c, k=P1) == ALIGN and w(c, slots=P1) == ALIGN and w(c, n=1 << 31) == UNSUPPORTED
    assert r(c, dt=4) == INVALID and r(c, total=-1) == INVALID and r(c, table=NUL) == INVALID and r(c, ld=0) == INVALID
    assert r(c, k=P8) == ALIGN and r(c, starts=P1) == ALIGN and r(c, total=1 << 31) == UNSUPPORTED
    # nothing to do is no error, whatever the other arguments are
    assert w(c, k=NUL, n=0) == _lib.NVFP4_OK and r(c, table=NUL, total=0) == _lib.NVFP4_OK


def _attention(**kw):
    a = Attention()
    for f in ("q", "out", "table", "lens", "q_starts", "workspace"):
        setattr(a, f, 0x10000)
    a.q_st, a.q_sh, a.o_st, a.o_sh = 256, 64, 256, 64
    a.table_ld, a.workspace_bytes, a.seqs, a.total_q, a.max_queries = 4, 1 << 40, 2, 5, 3
    a.q_heads, a.dtype, a.causal, a.scale = 4, BF16, 1, 0.125
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,err", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
    (dict(workspace=None), INVALID), (dict(workspace_bytes=16), INVALID), (dict(dtype=FP32), INVALID),
    (dict(q_heads=3), INVALID), (dict(q_heads=0), INVALID), (dict(seqs=-1), INVALID), (dict(table_ld=0), INVALID),
    (dict(max_queries=-1), INVALID), (dict(q_starts=None), INVALID),
    (dict(max_queries=1 << 24), UNSUPPORTED), (dict(table_ld=1 << 28), UNSUPPORTED), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(q=0x10001), ALIGN),
    (dict(workspace=0x10008), ALIGN), (dict(table=0x10001), ALIGN)])
def test_attention(kw, err):
    L = _lib.load()
    assert L.mxfp4_cache_attention(ctypes.byref(_cache()), ctypes.byref(_attention(**kw)), NUL) == err, _lib.last_error()


def test_attention_checks_the_cache():
    L = _lib.load()
    for kw, err in BAD_CACHES:
        assert L.mxfp4_cache_attention(ctypes.byref(_cache(**kw)), ctypes.byref(_attention()), NUL) == err, kw
    assert L.mxfp4_cache_attention(ctypes.byref(_cache()), None, NUL) == INVALID
