"""Norm and rotary positions of heads, alone and into the 4-bit cache, against
the formulas in binary64.

What binary32 may be off by, in steps of 2^-24 relative to the larger element of
a pair: the mean of up to 256 squares 20 / 2 (half through the root), rsqrtf 4,
the two products by it and the weight 2, an angle's cosine and sine 4, rotation
3: below 2^-19 in all.  Then one rounding to the output's type."""
import math

import pytest
import torch

import diffusion_transformer_mlp_gb300 as fc2
import _mx as mx
from test_gpu_mxfp4_cache import make_cache

pytestmark = pytest.mark.gpu

EPS = 1e-6
WORK = 2.0 ** -19
SMALLEST = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0, torch.float32: 2.0 ** -149}


def make_rotary(pairs, axes, interleaved, g, theta=10000.0):
    freq = float(theta) ** (-torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))
    axis = torch.randint(0, axes, (pairs,), generator=torch.Generator().manual_seed(pairs + axes), dtype=torch.int32)
    return freq.cuda(), axis.cuda(), fc2.head_rotary(freq, axis if axes > 1 else None, interleaved)


def formula(x, w, freq, axis, interleaved, positions, eps=EPS):
    """(result, bound of the binary32 work) in binary64."""
    y = x.double()
    if w is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    pairs = len(freq)
    pos = positions.reshape(len(x), -1).double()
    t = (pos[:, axis.long()] if pos.shape[1] > 1 else pos) * freq
    c, s = t.cos().unsqueeze(1), t.sin().unsqueeze(1)
    i = torch.arange(pairs, device="cuda")
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    a, b = y[..., ia], y[..., ib]
    out, size = y.clone(), y.abs() if w is not None else torch.zeros_like(y)  # neither normed nor rotated: as it was
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return out, size * WORK


def check(got, want):
    out, work = want
    step = torch.finfo(got.dtype).eps / 2 * out.abs() * (1 + 2.0 ** -10) + SMALLEST[got.dtype]
    assert torch.equal(torch.isnan(got), torch.isnan(out))
    over = ((got.double() - out).abs() - (work + step))[~torch.isnan(out)]
    assert bool((over <= 0).all()), float(over.max())


def heads(tokens, n, dim, g, dtype):
    x = torch.randn(tokens, n, dim, generator=g, device="cuda")
    x[..., ::17] *= 8
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,pairs,axes", [(16, 8, 1), (32, 8, 2), (64, 32, 1), (80, 24, 2), (96, 48, 3), (128, 64, 3),
                                            (128, 8, 1), (192, 96, 1), (256, 128, 3), (256, 40, 2), (64, 0, 1)])
def test_heads(dim, pairs, axes, interleaved, dtype):
    g = torch.Generator(device="cuda").manual_seed(dim + pairs)
    for tokens, hq, hk, weights in ((1, 5, 2, dtype), (37, 3, 0, torch.float32), (700, 9, 9, None), (3000, 1, 1, dtype)):
        freq, axis, rotary = make_rotary(pairs, axes, interleaved, g)
        pos = torch.randint(-5000, 1 << 20, (tokens, axes), generator=g, device="cuda", dtype=torch.int32)
        q, k = heads(tokens, hq, dim, g, dtype), heads(tokens, hk, dim, g, dtype) if hk else None
        wq, wk = ((1 + 0.3 * torch.randn(2, dim, generator=g, device="cuda")).to(weights) if weights else (None, None))
        oq, ok = fc2.head_norm_rotary(q, k, rotary, pos, wq, wk if hk else None, EPS)
        check(oq, formula(q, wq, freq, axis, interleaved, pos))
        if hk:
            check(ok, formula(k, wk, freq, axis, interleaved, pos))
        else:
            assert ok is None


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(interleaved):
    """Angles keep their fraction of a turn wherever the position is."""
    g = torch.Generator(device="cuda").manual_seed(5)
    freq, axis, rotary = make_rotary(32, 1, interleaved, g, theta=1e7)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, 123456789], dtype=torch.int32, device="cuda")
    q = heads(len(pos), 2, 64, g, torch.float32)
    got, _ = fc2.head_norm_rotary(q, None, rotary, pos)
    # the formula's own product of position and frequency is rounded: 2^31 radians to 2^-22
    out, work = formula(q, None, freq, axis, interleaved, pos)
    size = work / WORK
    assert float(((got.double() - out).abs() - work - size * 2.0 ** -21).max()) <= 0
    assert torch.equal(got[0], q[0])  # position 0 does not turn


def test_strides_and_places():
    """Views of one buffer, odd strides, results in place."""
    g = torch.Generator(device="cuda").manual_seed(6)
    freq, axis, rotary = make_rotary(32, 1, False, g)
    pos = torch.arange(50, device="cuda", dtype=torch.int32)
    w = 1 + 0.1 * torch.randn(128, generator=g, device="cuda")
    for pad in (0, 3, 8):
        buf = heads(50, 10, 128 + pad, g, torch.bfloat16)
        q, k = buf[:, :6, :128], buf[:, 6:8, :128]
        want = formula(q, w, freq, axis, False, pos), formula(k, w, freq, axis, False, pos)
        rest = buf[:, 8:].clone(), buf[..., 128:].clone()
        a, b = fc2.head_norm_rotary(q, k, rotary, pos, w, w, EPS)
        check(a, want[0]), check(b, want[1])
        out = torch.full((50, 12, 131), 7.0, device="cuda", dtype=torch.bfloat16)
        c, _ = fc2.head_norm_rotary(q, None, rotary, pos, w, None, EPS, q_out=out[:, 1::2, 1:129])
        assert torch.equal(c, a) and bool((out[:, ::2] == 7).all()) and bool((out[..., 129:] == 7).all())
        a2, b2 = fc2.head_norm_rotary(q, k, rotary, pos, w, w, EPS, q_out=q, k_out=k)
        assert a2.data_ptr() == q.data_ptr() and torch.equal(q, a) and torch.equal(k, b)
        assert torch.equal(buf[:, 8:], rest[0]) and torch.equal(buf[..., 128:], rest[1])
    one = heads(50, 1, 128, g, torch.bfloat16).expand(50, 4, 128)  # heads of one row
    got, _ = fc2.head_norm_rotary(one, None, rotary, pos, w)
    check(got, formula(one, w, freq, axis, False, pos))
    e, _ = fc2.head_norm_rotary(buf[:0, :6, :128], None, rotary, pos[:0])
    assert e.shape == (0, 6, 128)


def test_large_and_special_values():
    g = torch.Generator(device="cuda").manual_seed(7)
    freq, axis, rotary = make_rotary(32, 1, True, g)
    pos = torch.arange(6, device="cuda", dtype=torch.int32)
    w = torch.ones(64, device="cuda")
    q = heads(6, 1, 64, g, torch.float32)
    q[0] *= 1e30   # squares past the range
    q[1] *= 3e37
    q[2] *= 1e-25  # far below eps
    q[3] = 0
    got, _ = fc2.head_norm_rotary(q, None, rotary, pos, w, None, EPS)
    check(got[:4], tuple(t[:4] for t in formula(q, w, freq, axis, True, pos)))
    q[4, 0, 5], q[5, 0, 60] = math.inf, math.nan
    got, _ = fc2.head_norm_rotary(q, None, rotary, pos, w, None, EPS)
    assert bool(torch.isnan(got[4, 0, 4:6]).all()) and bool((got[4, 0, 6:] == 0).all())
    assert bool(torch.isnan(got[5]).all())
    plain, _ = fc2.head_norm_rotary(q, None, rotary, pos)  # without a norm it stays in its pair
    assert int(torch.isnan(plain[5]).sum()) == 2 and bool(torch.isfinite(plain[5, 0, :60]).all())


@pytest.mark.parametrize("interleaved", [False, True])
def test_what_is_not_rotated_stays_in_its_place(interleaved):
    """An infinity or a NaN behind the pairs reaches no other element, signs of
    zeros are kept there, and rotated ones stay in their pair."""
    g = torch.Generator(device="cuda").manual_seed(8)
    freq, axis, rotary = make_rotary(8, 1, interleaved, g)
    pos = torch.arange(1, 5, device="cuda", dtype=torch.int32)
    q = heads(4, 3, 64, g, torch.float32)
    q[0, 0, 16], q[1, 1, 63], q[2, 2, 40], q[3, 0, 17] = math.inf, math.nan, -0.0, -math.inf
    got, _ = fc2.head_norm_rotary(q, None, rotary, pos)
    assert torch.equal(torch.isfinite(got), torch.isfinite(q))
    bits = lambda t: torch.where(torch.isnan(t), 0, t.view(torch.int32))
    assert torch.equal(bits(got)[..., 16:], bits(q)[..., 16:])
    q[0, 1, 3] = math.inf
    got, _ = fc2.head_norm_rotary(q, None, rotary, pos)
    assert int((~torch.isfinite(got[0, 1])).sum()) == 2
    none = fc2.head_rotary(torch.zeros(0))
    assert torch.equal(bits(fc2.head_norm_rotary(q, None, none, pos)[0]), bits(q))


def quantised_between(got, y, e):
    """got [..., dim] are MXFP4 values of y with each element off by up to e:
    blocks whose scale is certain, and in those every value between the two ends'."""
    b, w, x = (t.unflatten(-1, (-1, 32)) for t in (y, e, got))
    lo, hi = ((b.abs() + s * w).amax(-1) for s in (-1, 1))
    sure = torch.frexp(lo).exponent == torch.frexp(hi).exponent
    assert float(sure.double().mean()) > 0.99
    scale = mx.pow2(torch.frexp(hi).exponent.long() - 3).unsqueeze(-1)
    grid = torch.cat((-mx.GRID.flip(0), mx.GRID)).to(y.device)

    def code(v):  # nearest grid values, off a tie
        return grid[((v / scale).clamp(-6, 6).unsqueeze(-1) - grid).abs().argmin(-1)] * scale
    ok = (x >= torch.minimum(code(b - w), code(b + w))) & (x <= torch.maximum(code(b - w), code(b + w)))
    ok = torch.where(w == 0, x == mx.values(y).unflatten(-1, (-1, 32)), ok)  # no work: exactly these
    assert bool(ok[sure].all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,pairs,interleaved", [(64, 32, False), (64, 8, False), (64, 24, True), (128, 64, False),
                                                   (128, 40, False), (128, 64, True), (256, 128, False), (256, 104, True)])
def test_into_the_cache(dim, pairs, interleaved, dtype):
    g = torch.Generator(device="cuda").manual_seed(dim + pairs)
    for tokens, hq, hkv, page, norm in ((1, 8, 2, 16, True), (61, 7, 1, 64, False), (900, 12, 3, 32, True)):
        freq, axis, rotary = make_rotary(pairs, 2, interleaved, g)
        cache = make_cache(tokens // page + 3, page, hkv, dim, 1)
        old = [t.clone() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
        x = heads(tokens, hq + 2 * hkv, dim, g, dtype)
        q, k, v = x.split((hq, hkv, hkv), 1)
        pos = torch.randint(0, 1 << 20, (tokens, 2), generator=g, device="cuda", dtype=torch.int32)
        slots = torch.randperm(cache.k_codes.shape[0] * page, generator=g, device="cuda")[:tokens]
        wq, wk = (1 + 0.3 * torch.randn(2, dim, generator=g, device="cuda")) if norm else (None, None)
        out = fc2.mxfp4_cache_write_rotary(cache, q, k, v, slots, rotary, pos, wq, wk, EPS)
        same, _ = fc2.head_norm_rotary(q, None, rotary, pos, wq, None, EPS)
        assert torch.equal(out, same)
        at, off = slots // page, slots % page
        kv = [mx.decode(mx.unpack(c[at, :, off]), s[at, :, off])
              for c, s in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales))]
        assert torch.equal(kv[1], mx.values(v))
        quantised_between(kv[0], *formula(k, wk, freq, axis, interleaved, pos))
        # nothing else has changed
        mask = torch.ones(old[0].shape[0], page, dtype=torch.bool, device="cuda")
        mask[at, off] = False
        for t, o in zip((cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales), old):
            assert torch.equal(t.transpose(1, 2)[mask], o.transpose(1, 2)[mask])


def test_cache_without_a_rotation_is_the_cache_write():
    """No norm, position 0, tokens without a slot: the bytes of mxfp4_cache_write."""
    g = torch.Generator(device="cuda").manual_seed(9)
    _, _, rotary = make_rotary(32, 1, False, g)
    x = heads(40, 6, 64, g, torch.bfloat16)
    x[3, 4, 7], x[5, 5, 40] = math.nan, math.inf
    q, k, v = x.split((2, 2, 2), 1)
    slots = torch.randperm(64, generator=g, device="cuda")[:40]
    slots[::7] = -1
    slots[1] = 64
    zero = torch.zeros(40, dtype=torch.int32, device="cuda")
    a, b = make_cache(4, 16, 2, 64, 3), make_cache(4, 16, 2, 64, 3)
    fc2.mxfp4_cache_write(a, k, v, slots)
    out = fc2.mxfp4_cache_write_rotary(b, q, k, v, slots, rotary, zero)
    assert torch.equal(out, q)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n


def test_refusals():
    g = torch.Generator(device="cuda").manual_seed(1)
    _, _, rotary = make_rotary(32, 1, False, g)
    q = torch.randn(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    w = torch.ones(64, device="cuda")
    call = fc2.head_norm_rotary
    for args, kw, match in [
            ((q, None, rotary, pos.long()), {}, "positions"), ((q, None, rotary, pos[:3]), {}, "positions"),
            ((q[0], None, rotary, pos), {}, "tokens, heads"), ((q, q[:3], rotary, pos), {}, "k must"),
            ((q, q.half(), rotary, pos), {}, "k must"), ((q, None, rotary, pos, w[:60]), {}, "q_weight"),
            ((q, None, rotary, pos, w.half()), {}, "q_weight"), ((q, None, rotary, pos, None, w), {}, "for a k"),
            ((q, q, rotary, pos, w, w.bfloat16()), {}, "one type"), ((q.int(), None, rotary, pos), {}, "q must be"),
            ((q.transpose(1, 2), None, rotary, pos), {}, "stride"), ((q, None, rotary, pos.cpu()), {}, "device"),
            ((q, None, rotary, pos), {"q_out": q[:, :1].expand(4, 2, 64)}, "overlap"),
            ((q, None, rotary, pos), {"q_out": q[:3]}, "q_out"), ((q, None, rotary, pos), {"q_out": q.float()}, "q_out"),
            ((q.clone().requires_grad_(), None, rotary, pos), {}, "gradient"),
            ((q, None, rotary, pos, w.clone().requires_grad_()), {}, "gradient")]:
        with pytest.raises(ValueError, match=match):
            call(*args, **kw)
    with torch.no_grad():
        call(q.clone().requires_grad_(), None, rotary, pos, w.clone().requires_grad_())
    wide = fc2.HeadRotary(torch.zeros(40, dtype=torch.int64, device="cuda"))
    odd = fc2.HeadRotary(torch.zeros(12, dtype=torch.int64, device="cuda"))
    for args, kw in [((q, None, wide, pos), {}), ((q, None, odd, pos), {}), ((q[..., :40], None, odd, pos), {}),
                     ((q, None, rotary, pos, w), {"eps": 0.0}), ((q, None, rotary, pos, w), {"eps": math.nan}),
                     ((q[:, :0], None, rotary, pos), {})]:
        with pytest.raises(fc2.NVFP4Error):
            call(*args, **kw)
    cache = make_cache(1, 16, 2, 64, 0)
    slots = torch.arange(4, device="cuda")
    for args, match in [((q, q, q, slots.int(), rotary, pos), "slots"), ((q, q[:, :1], q, slots, rotary, pos), "k must"),
                        ((q, q, q[:3], slots, rotary, pos), "v must"), ((q.float(), q.float(), q.float(), slots, rotary, pos), "q must"),
                        ((q[..., :32], q, q, slots, rotary, pos), "q must"), ((q, q, q, slots[:2], rotary, pos), "slots")]:
        with pytest.raises(ValueError, match=match):
            fc2.mxfp4_cache_write_rotary(cache, *args)


def test_sections_and_frequencies():
    freq, axis = fc2.rotary_frequencies((16, 24, 24), 100.0)
    assert axis.tolist() == [0] * 8 + [1] * 12 + [2] * 12
    assert torch.allclose(freq[8:20], 100.0 ** (-torch.arange(12, dtype=torch.float64) / 12))
    r = fc2.head_rotary(torch.tensor([1.0, -1.0, 0.0, 1e-12, 7.0, -0.0, 3.5, 1e-30]))
    want = torch.tensor([1.0, -1.0, 0.0, 1e-12, 7.0, 0.0, 3.5, 0.0], dtype=torch.float64) / (2 * math.pi)
    got = r.turns.cpu().double() / 2.0 ** 64
    assert float(((got - want + 0.5) % 1.0 - 0.5).abs().max()) < 2.0 ** -52
    for bad in (torch.ones(7), torch.ones(2, 8), torch.full((8,), math.inf)):
        with pytest.raises(ValueError):
            fc2.head_rotary(bad)
    with pytest.raises(ValueError):
        fc2.rotary_frequencies((3,))


def test_past_32_bits():
    """More than 2^32 bytes of heads, and pages behind 4 GB of codes."""
    n, h, dim = 70000, 256, 128
    freq, axis, rotary = make_rotary(64, 1, False, None)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    q = torch.empty(n, h, dim, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.ones(dim, device="cuda")
    out, _ = fc2.head_norm_rotary(q, None, rotary, pos, w)
    for rows in (slice(0, 2), slice(n // 2, n // 2 + 2), slice(n - 2, n)):
        check(out[rows], formula(q[rows], w, freq, axis, False, pos[rows]))
    del out
    cache = fc2.empty_mxfp4_cache(2300, 256, 64, 256)
    assert cache.k_codes.numel() > 1 << 32
    x = torch.randn(3, 64, 256, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([2299 * 256 + 255, 5, 1200 * 256 + 7], device="cuda")
    _, _, rotary = make_rotary(128, 1, True, None)
    fc2.mxfp4_cache_write_rotary(cache, x, x, x, slots, rotary, pos[:3] * 0)
    at, off = slots // 256, slots % 256
    for codes, scales in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
        assert torch.equal(mx.decode(mx.unpack(codes[at, :, off]), scales[at, :, off]), mx.values(x))


def test_same_bits_from_a_graph():
    """Captured calls give the bits of the calls, whatever the number of tokens
    makes of a token's share of a warp."""
    g = torch.Generator(device="cuda").manual_seed(3)
    freq, axis, rotary = make_rotary(64, 1, False, g)
    w = 1 + 0.1 * torch.randn(128, generator=g, device="cuda")
    q = heads(5000, 40, 128, g, torch.bfloat16)
    pos = torch.arange(5000, dtype=torch.int32, device="cuda")
    whole, _ = fc2.head_norm_rotary(q, None, rotary, pos, w)
    for n in (1, 7, 300):
        assert torch.equal(fc2.head_norm_rotary(q[:n], None, rotary, pos[:n], w)[0], whole[:n])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = fc2.head_norm_rotary(q, None, rotary, pos, w)
    out.zero_()
    graph.replay()
    assert torch.equal(out, whole)
