"""The paged MXFP4 cache and the attention over it against their definitions
in binary64.

Cache bytes are exact.  Attention: the scores are exact products summed in
float32 (relative error below 2^-14 of sum |q k| scale over at most 256 terms,
and the sizes below keep that sum under 64 times ... the tolerance states it
per case through the weights: dp/p <= 2^-24 256 sum|q k| scale < 2^-11 for
sums up to 32), ex2 is good to 2^-22, weights are rounded to FP16 (2^-12, or
2^-22 for up to 8 rows), and the output once to its type (unit roundoff 2^-8 or 2^-11).
Bound: half an ulp of the output + 2^-10 sum p |v|."""
import math

import pytest
import torch

import diffusion_transformer_mlp_gb300 as fc2
import _mx as mx

pytestmark = pytest.mark.gpu

HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def make_cache(pages, page, heads, dim, seed):
    """A cache full of arbitrary bytes, NaN scales among them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = fc2.empty_mxfp4_cache(pages, page, heads, dim)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    return c


def make_table(lens, page, seed, extra=2):
    g = torch.Generator().manual_seed(seed)
    need = [max(1, -(-n // page)) for n in lens]
    pages = sum(need) + extra
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.randint(0, pages, (len(lens), max(need) + 1), generator=g, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table.cuda(), pages


def fill(cache, table, lens, page, k, v):
    """Writes token rows k, v [sum lens, heads, dim] of every sequence."""
    slots = torch.cat([table[b, torch.arange(n) // page].long() * page + torch.arange(n, device="cuda") % page
                       for b, n in enumerate(lens)] + [torch.empty(0, dtype=torch.int64, device="cuda")])
    fc2.mxfp4_cache_write(cache, k, v, slots)
    return slots


def cache_values(cache):
    return (mx.decode(mx.unpack(cache.k_codes), cache.k_scales), mx.decode(mx.unpack(cache.v_codes), cache.v_scales))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("dim,heads,page", [(64, 1, 16), (64, 3, 64), (128, 8, 32), (128, 2, 256), (256, 5, 16),
                                            (256, 1, 128)])
def test_cache_write_and_read(dim, heads, page, dtype):
    lens = [1, 17, 0, 130, 64]
    table, pages = make_table(lens, page, dim + heads)
    cache = make_cache(pages, page, heads, dim, 1)
    before = [t.clone() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
    total = sum(lens)
    g = torch.Generator(device="cuda").manual_seed(3)
    k = (torch.randn(total, heads, dim, generator=g, device="cuda") * 3).to(dtype)
    v = torch.randn(total, heads, dim, generator=g, device="cuda").to(dtype)
    slots = fill(cache, table, lens, page, k, v)
    # bytes of the written slots are the definition's, all others are untouched
    for x, codes, scales, c0, s0 in ((k, cache.k_codes, cache.k_scales, before[0], before[1]),
                                     (v, cache.v_codes, cache.v_scales, before[2], before[3])):
        code, e = mx.encode(x)
        at, off = slots // page, slots % page
        want_c, want_s = c0.clone(), s0.clone()
        want_c[at, :, off] = code[..., 0::2] | code[..., 1::2] << 4
        want_s[at, :, off] = e
        assert torch.equal(codes, want_c) and torch.equal(scales, want_s)
    starts = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    for out in (torch.float32, dtype):
        kr, vr = fc2.mxfp4_cache_read(cache, table, starts, total, out)
        assert torch.equal(kr.double(), mx.values(k)) and torch.equal(vr.double(), mx.values(v))


def test_cache_write_strided_skipped_and_empty():
    page, heads, dim = 16, 4, 128
    cache = make_cache(4, page, heads, dim, 5)
    qkv = torch.randn(10, 6 + 2 * heads, dim + 3, device="cuda", dtype=torch.bfloat16)[..., 1:dim + 1]
    k, v = qkv[:, 6:6 + heads], qkv[:, 6 + heads:]
    slots = torch.tensor([0, -1, 63, 17, 64, 18, -5, 1 << 40, 33, 2], device="cuda")
    ref = [t.clone() for t in (cache.k_codes, cache.v_codes)]
    fc2.mxfp4_cache_write(cache, k, v, slots)
    keep = (slots >= 0) & (slots < 64)
    s = slots[keep]
    for x, got, want in ((k, cache.k_codes, ref[0]), (v, cache.v_codes, ref[1])):
        code, _ = mx.encode(x[keep])
        want[s // page, :, s % page] = code[..., 0::2] | code[..., 1::2] << 4
        assert torch.equal(got, want)
    fc2.mxfp4_cache_write(cache, k[:0], v[:0], slots[:0])
    one = k[:1, :1].expand(10, heads, dim)  # one row for every head, strides of zero
    fc2.mxfp4_cache_write(cache, one, one, slots)
    code, _ = mx.encode(one[keep])
    assert torch.equal(cache.k_codes[s // page, :, s % page], code[..., 0::2] | code[..., 1::2] << 4)


def test_cache_read_nan_blocks():
    page, heads, dim = 16, 2, 64
    cache = make_cache(2, page, heads, dim, 6)
    k = torch.randn(20, heads, dim, device="cuda")
    k[3, 1, 40] = math.inf
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    fill(cache, table, [20], page, k, k)
    kr, _ = fc2.mxfp4_cache_read(cache, table, torch.tensor([0, 20], dtype=torch.int32, device="cuda"), 20)
    nan = torch.zeros(20, heads, dim, dtype=torch.bool, device="cuda")
    nan[3, 1, 32:] = True
    assert torch.equal(torch.isnan(kr), nan)


def run_attention(lens, nq, hq, hkv, dim, page, dtype, seed=0, mul_k=1.0, mul_v=1.0, scale=None, **kw):
    table, pages = make_table(lens, page, seed)
    cache = make_cache(pages, page, hkv, dim, seed + 1)
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    total = sum(max(0, n) for n in lens)
    k = (torch.randn(total, hkv, dim, generator=g, device="cuda") * mul_k).to(dtype)
    v = (torch.randn(total, hkv, dim, generator=g, device="cuda") * mul_v).to(dtype)
    fill(cache, table, [max(0, n) for n in lens], page, k, v)
    starts = [0]
    for n in nq:
        starts.append(starts[-1] + n)
    q = torch.randn(starts[-1], hq, dim, generator=g, device="cuda").to(dtype)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qs = None if all(n == 1 for n in nq) and not kw.pop("explicit", False) else torch.tensor(starts, dtype=torch.int32,
                                                                                            device="cuda")
    lse = torch.full((starts[-1], hq), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = fc2.mxfp4_cache_attention(q, cache, table, lens_t, q_starts=qs, max_queries=max(nq), scale=scale, lse=lse,
                                    status=status, **kw)
    assert int(status) == 0
    kc, vc = cache_values(cache)
    ref, ref_lse, mag = mx.attention(q.double(), kc, vc, table, lens, starts, page,
                                     dim ** -0.5 if scale is None else scale, **kw)
    return out, lse, ref, ref_lse, mag, (q, cache, table, lens_t, qs, max(nq))


def check(out, lse, ref, ref_lse, mag):
    assert torch.equal(torch.isnan(out), torch.isnan(ref))
    fine = ~torch.isnan(ref)
    bound = HALF_ULP[out.dtype] * 1.01 * ref.abs() + 2.0 ** -10 * mag + (2.0 ** -25 if out.dtype is torch.float16 else 0)
    worst = float((((out.double() - ref).abs() / bound.clamp(min=1e-300))[fine]).max()) if bool(fine.any()) else 0.0
    assert worst <= 1.0, worst
    assert bool((out[ref == 0] == 0).all())
    empty = ref_lse == -math.inf
    assert bool((lse[empty] == -math.inf).all())
    live = ~empty & torch.isfinite(ref_lse)
    if bool(live.any()):
        assert float((lse.double() - ref_lse)[live].abs().max()) < 2.0 ** -10


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1), (7, 1), (12, 3), (16, 1), (40, 2)])
def test_decode(hq, hkv, dim, dtype):
    lens = [1, 2, 63, 64, 65, 200, 1000, 333]
    check(*run_attention(lens, [1] * len(lens), hq, hkv, dim, 16, dtype, seed=hq + dim)[:5])


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_decode_pages(page):
    for dim in (64, 128, 256):
        lens = [page, page - 1, page + 1, 5 * page + 3, 700]
        check(*run_attention(lens, [1] * 5, 8, 2, dim, page, torch.bfloat16, seed=page)[:5])


@pytest.mark.parametrize("dim,group", [(64, 1), (64, 8), (128, 1), (128, 4), (128, 7), (256, 2), (256, 16)])
@pytest.mark.parametrize("causal", [True, False])
def test_many_queries(dim, group, causal):
    lens, nq = [5, 70, 300, 129, 64, 1], [5, 33, 7, 129, 1, 1]
    check(*run_attention(lens, nq, 2 * group, 2, dim, 32, torch.bfloat16, seed=dim + group, causal=causal)[:5])


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (63, 1), (64, 0), (100, 64), (100, 65), (128, 300), (5000, 4)])
@pytest.mark.parametrize("causal", [True, False])
def test_windows_and_sinks(window, sinks, causal):
    lens, nq = [400, 1, 90, 513, 700], [1, 1, 40, 3, 130]
    for dim in (64, 128, 256):
        check(*run_attention(lens, nq, 4, 2, dim, 16, torch.float16, seed=window + sinks, window=window, sinks=sinks,
                             causal=causal)[:5])


def test_rows_without_keys():
    """Sequences without keys, sequences without queries, more queries than keys."""
    lens, nq = [0, 10, 3, 0, 40, 0], [1, 0, 9, 4, 2, 0]
    for dim in (64, 128, 256):
        for group in (1, 8):
            out, lse, ref, ref_lse, mag, _ = run_attention(lens, nq, 2 * group, 2, dim, 16, torch.bfloat16, seed=dim)
            check(out, lse, ref, ref_lse, mag)
            assert bool((out[0] == 0).all()) and bool((out[1:7] == 0).all()) and bool((lse[1:7] == -math.inf).all())
    check(*run_attention([0, 0], [1, 1], 4, 2, 64, 16, torch.float16)[:5])


def test_nan_stays_with_those_who_see_it():
    """A NaN key or value (E = 255) reaches the queries that see it and no other,
    behind the causal mask, outside the window, and past the end."""
    page, hkv, hq, dim = 16, 2, 8, 128
    for window, sinks in ((0, 0), (20, 3)):
        lens, nq = [100], [60]
        table, pages = make_table(lens, page, 1)
        cache = make_cache(pages, page, hkv, dim, 2)
        k, v = torch.randn(100, hkv, dim, device="cuda"), torch.randn(100, hkv, dim, device="cuda")
        v[70, 0, 5] = math.nan
        k[90, 1, 64] = math.inf
        v[95, 1, 127] = math.inf
        fill(cache, table, lens, page, k, v)
        q = torch.randn(60, hq, dim, device="cuda", dtype=torch.bfloat16)
        lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        qs = torch.tensor([0, 60], dtype=torch.int32, device="cuda")
        out = fc2.mxfp4_cache_attention(q, cache, table, lens_t, qs, 60, window=window, sinks=sinks)
        kc, vc = cache_values(cache)
        ref, ref_lse, mag = mx.attention(q.double(), kc, vc, table, lens, [0, 60], page, dim ** -0.5, window=window,
                                         sinks=sinks)
        assert torch.equal(torch.isnan(out), torch.isnan(ref))
        fine = ~torch.isnan(ref)
        assert float((out.double() - ref)[fine].abs().max()) < 0.05
        # the decoding form, one query at a time
        for t in (69, 70, 71, 89, 90, 99):
            one = fc2.mxfp4_cache_attention(q[:1], cache, table, lens_t * 0 + t + 1, window=window, sinks=sinks)
            r1, _, _ = mx.attention(q[:1].double(), kc, vc, table, [t + 1], [0, 1], page, dim ** -0.5, window=window,
                                    sinks=sinks)
            assert torch.equal(torch.isnan(one), torch.isnan(r1)), t


def test_long_sequence_beside_short_ones():
    lens = [20000, 3, 1, 70, 8191]
    check(*run_attention(lens, [1] * 5, 16, 2, 128, 64, torch.bfloat16, seed=4)[:5])


def test_many_sequences():
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 40, (2600,), generator=g).tolist()
    check(*run_attention(lens, [1] * 2600, 2, 1, 64, 16, torch.bfloat16, seed=8)[:5])


@pytest.mark.parametrize("mul_k,mul_v,scale", [(1e-3, 1e3, None), (40.0, 1e-6, 0.01), (1.0, 1.0, -0.2),
                                               (1.0, 1.0, 0.0), (1e4, 1.0, 1e-5)])
def test_magnitudes(mul_k, mul_v, scale):
    for nq in (1, 20):
        out, lse, ref, ref_lse, mag, _ = run_attention([300, 77], [nq, nq], 8, 2, 128, 16, torch.bfloat16, seed=5,
                                                       mul_k=mul_k, mul_v=mul_v, scale=scale)
        check(out, lse, ref, ref_lse, mag)


def test_uneven_block_scales():
    """Blocks of one token, and tokens of one block, 2^12 and more apart; the
    largest values where the weights are small."""
    page, hkv, dim = 16, 1, 128
    lens = [200]
    table, pages = make_table(lens, page, 1)
    cache = make_cache(pages, page, hkv, dim, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randn(200, hkv, dim, generator=g, device="cuda")
    v = torch.randn(200, hkv, dim, generator=g, device="cuda")
    v = v * torch.exp2(torch.randint(-6, 7, (200, hkv, 4), generator=g, device="cuda").repeat_interleave(32, -1).float())
    k = k * torch.exp2(torch.randint(-6, 2, (200, hkv, 4), generator=g, device="cuda").repeat_interleave(32, -1).float())
    v[..., 32:64] *= 2.0 ** -20
    fill(cache, table, lens, page, k, v)
    kc, vc = cache_values(cache)
    for n, hq in ((1, 8), (40, 4)):
        q = torch.randn(n, hq, dim, generator=g, device="cuda").to(torch.bfloat16)
        out = fc2.mxfp4_cache_attention(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                        torch.tensor([0, n], dtype=torch.int32, device="cuda"), n)
        ref, _, mag = mx.attention(q.double(), kc, vc, table, lens, [0, n], page, dim ** -0.5)
        bound = 2.0 ** -8 * 1.01 * ref.abs() + 2.0 ** -10 * mag
        assert float(((out.double() - ref).abs() / bound).max()) <= 1.0


def test_strides_out_and_stream():
    out, lse, ref, ref_lse, mag, (q, cache, table, lens, qs, mq) = run_attention([50, 400], [3, 2], 8, 2, 64, 16,
                                                                                 torch.float16, seed=6)
    check(out, lse, ref, ref_lse, mag)
    wide = torch.zeros(5, 11, 64 + 1, dtype=torch.float16, device="cuda")
    qv = wide[:, 2:10, 1:]
    qv.copy_(q)
    buf = torch.full((5, 9, 64 + 1), 5.0, dtype=torch.float16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fc2.mxfp4_cache_attention(qv, cache, table, lens, qs, mq, out=buf[:, 1:, :64], stream=s)
    s.synchronize()
    assert torch.equal(buf[:, 1:, :64], out)
    assert bool((buf[:, 0] == 5).all()) and bool((buf[:, :, 64] == 5).all())
    for _ in range(5):
        assert torch.equal(fc2.mxfp4_cache_attention(q, cache, table, lens, qs, mq), out)


def test_decode_equals_the_last_row_of_a_chunk():
    """One query at the end sees what the last query of a chunk sees."""
    out, _, ref, _, mag, (q, cache, table, lens, qs, mq) = run_attention([500], [64], 8, 2, 128, 16, torch.bfloat16, seed=2)
    one = fc2.mxfp4_cache_attention(q[-1:], cache, table, lens)
    bound = 2.0 ** -7 * ref[-1:].abs() + 2.0 ** -9 * mag[-1:]
    assert bool(((one.double() - out[-1:].double()).abs() <= bound).all())


def test_refusals():
    cache = make_cache(4, 16, 2, 64, 1)
    q = torch.randn(1, 4, 64, device="cuda", dtype=torch.bfloat16)
    table = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    ok = fc2.mxfp4_cache_attention(q, cache, table, lens)
    assert ok.shape == q.shape
    for bad in (dict(q=q.float()), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(table=table.long()),
                dict(lens=lens.long()), dict(lens=torch.cat([lens, lens])), dict(window=-1), dict(sinks=-1),
                dict(max_queries=2), dict(out=torch.empty(1, 4, 64, device="cuda")),
                dict(lse=torch.empty(4, 1, device="cuda")), dict(q=q.cpu())):
        kw = dict(q=q, cache=cache, table=table, lens=lens)
        kw.update(bad)
        with pytest.raises(ValueError):
            fc2.mxfp4_cache_attention(**kw)
    with pytest.raises(fc2.NVFP4Error):
        fc2.mxfp4_cache_attention(q, cache, table, lens, scale=math.nan)
    k = torch.randn(3, 2, 64, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    for args in ((k[:2], k, slots), (k, k.half(), slots), (k[:, :1], k[:, :1], slots), (k, k, slots.int()),
                 (k, k, slots[:2])):
        with pytest.raises(ValueError):
            fc2.mxfp4_cache_write(cache, *args)
    odd = fc2.empty_mxfp4_cache(4, 24, 2, 64)
    with pytest.raises(fc2.NVFP4Error):
        fc2.mxfp4_cache_write(odd, k, k, slots)
    odd = fc2.empty_mxfp4_cache(4, 16, 2, 96)
    with pytest.raises(fc2.NVFP4Error):
        fc2.mxfp4_cache_write(odd, torch.randn(3, 2, 96, device="cuda"), torch.randn(3, 2, 96, device="cuda"), slots)
