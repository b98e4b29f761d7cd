"""The entry points for rotary positions, pages and shared prefixes without a
GPU: sizes, and argument errors that come back before anything runs."""
import ctypes
import math

import pytest

from diffusion_transformer_mlp_gb300 import _lib
from test_mxfp4_abi import ALIGN, BAD_CACHES, BF16, FP16, FP32, INVALID, NUL, P1, P16, P8, UNSUPPORTED, _attention, _cache

by = ctypes.byref
OK = _lib.NVFP4_OK


class Heads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "out", "weight")] + \
        [(n, ctypes.c_int64) for n in ("st", "sh", "o_st", "o_sh")] + [(n, ctypes.c_int32) for n in ("heads", "reserved")]


class Rotary(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("turns", "axis", "positions")] + \
        [(n, ctypes.c_int32) for n in ("pairs", "axes", "interleaved", "reserved")]


class Pages(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("refs", "table", "lens")] + \
        [(n, ctypes.c_int64) for n in ("pages", "table_ld")] + [(n, ctypes.c_int32) for n in ("rows", "page_size")]


class SharedArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("groups", "shared")] + [(n, ctypes.c_int32) for n in ("count", "max_group", "always", "reserved")]


def made(cls, defaults, kw):
    s = cls()
    for k, v in {**defaults, **kw}.items():
        setattr(s, k, v)
    return s


def heads(**kw):
    return made(Heads, dict(x=0x10000, out=0x10000, st=256, sh=64, o_st=256, o_sh=64, heads=4), kw)


def rotary(**kw):
    return made(Rotary, dict(turns=0x10000, axis=0x10000, positions=0x10000, pairs=32, axes=2), kw)


def pages(**kw):
    return made(Pages, dict(refs=0x10000, table=0x10000, lens=0x10000, pages=64, table_ld=8, rows=4, page_size=16), kw)


ROTARY = [(dict(pairs=-8), UNSUPPORTED), (dict(pairs=12), UNSUPPORTED), (dict(pairs=40), UNSUPPORTED),
          (dict(axes=0), INVALID), (dict(axes=70000), INVALID), (dict(turns=None), INVALID),
          (dict(positions=None), INVALID), (dict(turns=0x10004), ALIGN), (dict(axis=0x10002), ALIGN),
          (dict(positions=0x10001), ALIGN)]


def test_rotary():
    L = _lib.load()

    def f(q=heads(), k=heads(heads=2), r=rotary(), dt=BF16, wdt=BF16, n=3, dim=64, eps=1e-6):
        ref = lambda s: None if s is None else by(s)
        return L.head_norm_rotary(ref(q), ref(k), ref(r), dt, wdt, n, dim, eps, NUL)
    for kw, err in ROTARY:
        assert f(r=rotary(**kw)) == err, kw
    assert f(q=None) == INVALID and f(r=None) == INVALID and f(q=heads(x=None)) == INVALID
    assert f(k=heads(out=None)) == INVALID and f(q=heads(heads=0)) == INVALID and f(k=heads(heads=70000)) == INVALID
    assert f(dt=5) == INVALID and f(dt=BF16, wdt=FP16) == INVALID and f(n=-1) == INVALID and f(n=1 << 31) == UNSUPPORTED
    assert f(dim=0) == UNSUPPORTED and f(dim=72) == UNSUPPORTED and f(dim=272) == UNSUPPORTED
    for eps in (0.0, -1.0, 1e-13, 1.5, math.nan, math.inf):
        assert f(eps=eps) == INVALID
    assert f(q=heads(x=0x10001)) == ALIGN and f(k=heads(out=0x10001)) == ALIGN and f(q=heads(weight=0x10001)) == ALIGN
    assert f(q=heads(weight=0x10002), wdt=FP32) == ALIGN
    assert f(n=0) == OK and f(q=heads(x=None), n=0) == OK and f(q=heads(heads=0), n=0) == INVALID


def test_cache_write_rotary():
    L = _lib.load()

    def f(c=_cache(), q=heads(), k=heads(heads=2), v=heads(heads=2), slots=P16, r=rotary(), dt=BF16, wdt=BF16, n=3, eps=1e-6):
        ref = lambda s: None if s is None else by(s)
        return L.mxfp4_cache_write_rotary(ref(c), ref(q), ref(k), ref(v), slots, ref(r), dt, wdt, n, eps, NUL)
    for kw, err in BAD_CACHES:
        assert f(c=_cache(**kw)) == err, kw
    for kw, err in ROTARY:
        assert f(r=rotary(**kw)) == err, kw
    assert f(c=None) == INVALID and f(q=None) == INVALID and f(k=None) == INVALID and f(v=None) == INVALID
    assert f(dt=FP32, wdt=FP32) == INVALID and f(k=heads(heads=3)) == INVALID and f(v=heads(heads=1)) == INVALID
    assert f(v=heads(heads=2, weight=0x10000)) == INVALID and f(slots=NUL) == INVALID and f(slots=P1) == ALIGN
    assert f(q=heads(out=None)) == INVALID and f(q=heads(heads=0)) == INVALID and f(k=heads(heads=2, x=0x10001)) == ALIGN
    assert f(slots=NUL, n=0) == OK


BAD_PAGES = [(dict(refs=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
             (dict(pages=0), INVALID), (dict(rows=0), INVALID), (dict(table_ld=0), INVALID), (dict(page_size=0), INVALID),
             (dict(page_size=24), UNSUPPORTED), (dict(page_size=512), UNSUPPORTED), (dict(pages=(1 << 30) + 1), UNSUPPORTED),
             (dict(rows=(1 << 20) + 1), UNSUPPORTED), (dict(table_ld=1 << 27), UNSUPPORTED),
             (dict(rows=1 << 20, table_ld=1 << 12), UNSUPPORTED), (dict(refs=0x10002), ALIGN), (dict(table=0x10001), ALIGN),
             (dict(lens=0x10001), ALIGN)]


def test_pages():
    L = _lib.load()
    big = 1 << 50
    sel = lambda g, src=P16, ws=P16, n=big: L.mxfp4_pages_select(g, src, ws, n, NUL)
    ext = lambda g, c=P16, total=5, slots=P16, copies=P16, missing=P16, ws=P16, n=big: L.mxfp4_pages_extend(
        g, c, total, slots, copies, missing, ws, n, NUL)
    com = lambda g, moves=P16, used=P16, ws=P16, n=big: L.mxfp4_pages_compact(g, moves, used, ws, n, NUL)
    for kw, err in BAD_PAGES:
        g = by(pages(**kw))
        assert sel(g) == err and ext(g) == err and com(g) == err, kw
    g = by(pages())
    for f in (sel, ext, com):
        assert f(None) == INVALID and f(g, ws=NUL) == INVALID and f(g, ws=P8) == ALIGN and f(g, n=64) == INVALID
    assert sel(g, src=NUL) == INVALID and sel(g, src=P1) == ALIGN
    assert ext(g, c=NUL) == INVALID and ext(g, slots=NUL) == INVALID and ext(g, copies=NUL) == INVALID
    assert ext(g, missing=NUL) == INVALID and ext(g, total=-1) == INVALID and ext(g, total=1 << 31) == UNSUPPORTED
    assert ext(g, slots=ctypes.c_void_p(0x10004)) == ALIGN and ext(g, copies=P1) == ALIGN
    assert com(g, moves=NUL) == INVALID and com(g, used=NUL) == INVALID and com(g, used=P1) == ALIGN
    small, large = (L.mxfp4_pages_workspace_bytes(by(pages(pages=n))) for n in (64, 10 ** 6))
    assert 0 < small < large and L.mxfp4_pages_workspace_bytes(None) == 0
    assert L.mxfp4_pages_workspace_bytes(by(pages(rows=1000, table_ld=5000))) >= 4 * 1000 * 5000


def test_cache_copy():
    L = _lib.load()
    f = lambda a=_cache(), b=_cache(), pairs=P16, n=3: L.mxfp4_cache_copy(by(a), by(b), pairs, n, NUL)
    for kw, err in BAD_CACHES:
        assert f(a=_cache(**kw)) == err and f(b=_cache(**kw)) == err, kw
    assert f(b=_cache(page_size=32)) == INVALID and f(b=_cache(kv_heads=1)) == INVALID and f(b=_cache(dim=128)) == INVALID
    assert f(pairs=NUL) == INVALID and f(pairs=P1) == ALIGN and f(n=-1) == INVALID and f(n=1 << 31) == UNSUPPORTED
    assert f(pairs=NUL, n=0) == OK


@pytest.mark.parametrize("kw,skw,err", [
    (dict(q=None), {}, INVALID), (dict(workspace_bytes=1 << 12), {}, INVALID), (dict(window=8), {}, UNSUPPORTED),
    (dict(dtype=FP32), {}, INVALID), (dict(q_heads=3), {}, INVALID), (dict(max_queries=1 << 24), {}, UNSUPPORTED),
    (dict(total_q=1 << 24), dict(max_group=1 << 24), UNSUPPORTED), (dict(scale=math.nan), {}, INVALID),
    ({}, dict(count=-1), INVALID), ({}, dict(max_group=-1), INVALID), ({}, dict(groups=None), INVALID),
    ({}, dict(shared=None), INVALID), ({}, dict(groups=0x10002), ALIGN), ({}, dict(shared=0x10001), ALIGN)])
def test_shared(kw, skw, err):
    L = _lib.load()
    s = made(SharedArgs, dict(groups=0x10000, shared=0x10000, count=1, max_group=5), skw)
    assert L.mxfp4_cache_attention_shared(by(_cache()), by(_attention(**kw)), by(s), NUL) == err, _lib.last_error()


def test_shared_checks_the_rest():
    L = _lib.load()
    s = made(SharedArgs, dict(groups=0x10000, shared=0x10000, count=1, max_group=5), {})
    for kw, err in BAD_CACHES:
        assert L.mxfp4_cache_attention_shared(by(_cache(**kw)), by(_attention()), by(s), NUL) == err, kw
    f = L.mxfp4_cache_attention_shared
    assert f(None, by(_attention()), by(s), NUL) == INVALID and f(by(_cache()), None, by(s), NUL) == INVALID
    assert f(by(_cache()), by(_attention()), None, NUL) == INVALID
    assert f(by(_cache()), by(_attention(seqs=0)), by(s), NUL) == OK


def test_shared_workspace():
    w = _lib.load().mxfp4_attention_shared_workspace_bytes
    own = _lib.load().mxfp4_attention_workspace_bytes
    assert w(8, 32, 128, 0, 1, 4, 16, 1, 4) == 0 and w(8, 32, 128, 4, 1, 0, 16, 1, 4) == 0
    assert w(8, 32, 128, 4, 1, 4, 16, 0, 0) == own(8, 32, 128, 1)
    assert w(8, 32, 128, 64, 1, 64, 1000, 2, 64) >= own(8, 32, 128, 64) + 64 * 32 * 128 * 8 + 66 * 4000
