"""Attention over a shared prefix: the result of the ordinary attention, whatever
is shared, and whether the call finds that worth it or not (which changes bits, so
that each case runs both ways).  Compared with the binary64 definition under the bound of the cache's
tests (each part is within it, and the join's binary32 work is 2^-20 beside)."""
import math

import pytest
import torch

import diffusion_transformer_mlp_gb300 as fc2
import _mx as mx
from test_gpu_mxfp4_cache import cache_values, check, make_cache

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Shared:
    """Groups of sequences: sizes[g] of them share prefixes[g] tokens; lens and
    queries by sequence."""

    def __init__(self, sizes, prefixes, lens, nq, hq, hkv, dim, page=16, dtype=torch.bfloat16, seed=0, lead=0):
        self.lens, self.nq, self.page, self.dim = lens, nq, page, dim
        self.groups = [lead]
        for n in sizes:
            self.groups.append(self.groups[-1] + n)
        self.prefixes = prefixes
        g = torch.Generator(device="cuda").manual_seed(seed)
        counts = [-(-max(n, 0) // page) for n in lens]
        table = torch.zeros(len(lens), max(counts) + 2, dtype=torch.int32)
        at = 0
        for b, c in enumerate(counts):
            table[b, :c] = torch.arange(at, at + c)
            at += c
        order = torch.randperm(at + 2, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        table = order[table.long()]
        self.cache = make_cache(at + 2, page, hkv, dim, seed + 1)
        for t in (self.cache.k_codes, self.cache.k_scales, self.cache.v_codes, self.cache.v_scales):
            t.random_(0, 256, generator=g)
        self.cache.k_scales.random_(118, 128, generator=g)
        self.cache.v_scales.random_(118, 128, generator=g)
        for k, p in enumerate(prefixes):  # what is shared lies in the same pages, the rest of its last page in a copy
            first = self.groups[k]
            for b in range(first + 1, self.groups[k + 1]):
                n = min(p, max(lens[b], 0), max(lens[first], 0))
                table[b, :n // page] = table[first, :n // page]
                if n % page:
                    for t in (self.cache.k_codes, self.cache.k_scales, self.cache.v_codes, self.cache.v_scales):
                        t[table[b, n // page], :, :n % page] = t[table[first, n // page], :, :n % page]
        self.table = table.cuda()
        self.starts = [0]
        for n in nq:
            self.starts.append(self.starts[-1] + n)
        self.q = torch.randn(self.starts[-1], hq, dim, generator=g, device="cuda").to(dtype)

    def run(self, q=None, always=True, **kw):
        q = self.q if q is None else q
        self.lse = torch.full((len(q), q.shape[1]), 7.0, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        explicit = kw.pop("explicit", False)
        starts = None if all(n == 1 for n in self.nq) and not explicit else i32(self.starts)
        self.out = fc2.mxfp4_cache_attention_shared(q, self.cache, self.table, i32(self.lens), i32(self.groups),
                                                    i32(self.prefixes), starts, max(self.nq), lse=self.lse,
                                                    status=status, always=always, **kw)
        assert int(status) == 0
        return self.out

    def check(self, causal=True):
        kc, vc = cache_values(self.cache)
        want = mx.attention(self.q.double(), kc, vc, self.table, self.lens, self.starts, self.page, self.dim ** -0.5,
                            causal=causal)
        check(self.out, self.lse, *want)
        kept = self.out, self.lse
        self.run(always=False, causal=causal)
        check(self.out, self.lse, *want)
        self.out, self.lse = kept


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 1), (28, 4)])
def test_decode(hq, hkv, dim, dtype):
    c = Shared([3, 1, 5, 20], [100, 257, 64, 400], [101, 100 + 70, 300, 500] + [65, 90, 128, 129, 64 + 200] +
               [401 + 13 * i for i in range(20)], [1] * 29, hq, hkv, dim, dtype=dtype, seed=dim + hq)
    c.run()
    c.check()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_pages_and_prefixes(page):
    """Prefixes that end in, before and behind a page's end, and of no page."""
    for prefix in (1, page - 1, page, page + 1, 3 * page, 5 * page - 2):
        c = Shared([6], [prefix], [prefix + n for n in (1, 2, page, page + 1, 3 * page, 700)], [1] * 6, 8, 2, 64, page,
                   seed=prefix)
        c.run()
        c.check()


@pytest.mark.parametrize("dim,group", [(64, 1), (64, 8), (128, 4), (256, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_several_queries(dim, group, causal):
    lens = [230, 205, 201, 333] + [90, 81] + [700, 650, 651]
    nq = [7, 5, 1, 130] + [3, 1] + [1, 0, 2]
    c = Shared([4, 2, 3], [200, 80, 640], lens, nq, 2 * group, 2, dim, 32, seed=dim + group)
    c.run(causal=causal)
    c.check(causal)


def test_queries_within_the_prefix():
    """A group shares no more than what lies before all its queries, or what all have."""
    lens, nq = [120, 150, 101, 130], [1, 60, 40, 2]  # queries from 90 and 61 on
    for causal in (True, False):
        c = Shared([4], [100], lens, nq, 4, 2, 64, seed=3)
        c.run(causal=causal)
        c.check(causal)
    c = Shared([3], [100], [100, 100, 100], [1, 1, 1], 4, 2, 64, seed=4)  # the prefix is all there is
    for causal in (True, False):
        c.run(causal=causal)
        c.check(causal)


def test_empty_rows_and_groups():
    """Groups of none, sequences without keys or queries, sequences of no group."""
    lens = [40, 0, 90] + [0, 100, 120, 0] + [200, 210]
    nq = [1, 1, 2] + [0, 1, 0, 0] + [1, 1]
    c = Shared([0, 4, 0], [500, 96, 32], lens, nq, 8, 2, 64, seed=5, lead=3)
    c.run()
    c.check()
    c = Shared([2], [64], [0, 0], [1, 1], 4, 2, 64, seed=6)
    assert bool((c.run() == 0).all()) and bool((c.lse == -math.inf).all())
    c = Shared([], [], [70, 33], [1, 3], 4, 2, 64, seed=7)  # no groups at all
    c.run()
    c.check()
    none = c.q[:0]
    assert fc2.mxfp4_cache_attention_shared(none, c.cache, c.table[:0], i32([]), i32([0]), i32([]), i32([0]), 1).shape == none.shape


def test_rows_behind_the_last_sequence():
    c = Shared([2], [64], [100, 90], [2, 1], 4, 2, 64, seed=8)
    q = torch.cat((c.q, c.q))
    out = torch.full_like(q, 5.0)
    c.run(q, out=out)
    assert bool((out[3:] == 5).all()) and bool((c.lse[3:] == 7).all())
    c.out, c.lse = out[:3], c.lse[:3]
    c.check()


def test_many_sequences_and_groups():
    """More of them than one launch takes."""
    n = 1100
    c = Shared([1] * n, [16 + i % 20 for i in range(n)], [40 + i % 50 for i in range(n)], [1] * n, 2, 1, 64, seed=9)
    c.run()
    c.check()
    c.run(max_group=1)  # few rows: prefixes and own tokens in one list
    c.check()
    c = Shared([n], [64], [65 + i % 50 for i in range(n)], [1] * n, 2, 1, 64, seed=10)
    c.run(max_group=n)
    c.check()


def test_no_other_bytes_matter():
    """NaN everywhere but in the tokens that are seen, and in copies of the prefix
    that are not read."""
    c = Shared([3], [64], [70, 81, 200], [1, 1, 1], 8, 2, 128, seed=11)
    want = c.run().clone()
    used = torch.zeros(len(c.cache.k_codes), c.page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(c.lens):
        t = torch.arange(n, device="cuda")
        used[c.table[b, t // c.page].long(), t % c.page] = True
    for s in (c.cache.k_scales, c.cache.v_scales):
        s.transpose(1, 2)[~used] = 255
    c.table[1:, :4] = c.table[0, :4]
    assert torch.equal(c.run(), want)


@pytest.mark.parametrize("n,nq", [(4, 1), (20, 1), (3, 2)])
def test_nan_blocks(n, nq):
    """NaN keys and values of the prefix reach all rows, own ones their sequence's."""
    c = Shared([n], [64], [90 + i for i in range(n)], [nq] * n, 8, 2, 64, seed=n)
    page, off = int(c.table[0, 1]), 5
    c.cache.v_scales[page, 0, off, 1] = 255
    c.cache.k_scales[int(c.table[1, 5]), 1, 2] = 255  # key 82 of sequence 1
    c.run()
    c.check()
    assert bool(torch.isnan(c.out[:, :4, 32:]).all()) and bool(torch.isfinite(c.out[:, :4, :32]).all())
    assert bool(torch.isnan(c.out[c.starts[1]:c.starts[2], 4:]).all()) and bool(torch.isfinite(c.out[:nq, 4:]).all())


@pytest.mark.parametrize("n", [4, 40])
def test_values_at_the_end_of_the_range(n):
    """Parts of large values join without leaving the range."""
    c = Shared([n], [64], [80 + i for i in range(n)], [1] * n, 8, 2, 64, seed=n)
    c.cache.v_scales.fill_(252)  # up to 6 2^125, 0.75 of the largest binary32
    c.cache.v_codes.fill_(0x77)
    c.run()
    assert bool(torch.isfinite(c.out).all())
    want = torch.full_like(c.out, 6 * 2.0 ** 125)
    # weights of 11 bits each, sums of them, one rounding to bf16
    assert float((c.out.double() / want.double() - 1).abs().max()) < 2.0 ** -8


def test_strided_queries_and_outputs():
    c = Shared([3], [64], [70, 81, 200], [1, 1, 1], 8, 2, 64, seed=12)
    want, lse = c.run().clone(), c.lse.clone()
    buf = torch.zeros(3, 11, 67, dtype=torch.bfloat16, device="cuda")
    buf[:, 1:9, 2:66] = c.q
    out = torch.zeros(3, 10, 66, dtype=torch.bfloat16, device="cuda")
    got = c.run(buf[:, 1:9, 2:66], out=out[:, 1:9, 1:65], explicit=True)
    assert torch.equal(got, want) and torch.equal(c.lse, lse)
    assert bool((out[:, 0] == 0).all()) and bool((out[..., 0] == 0).all()) and bool((out[..., 65] == 0).all())


def test_same_bits_again_and_in_a_graph():
    c = Shared([40, 3], [1000, 333], [1001 + 7 * i for i in range(40)] + [400, 334, 900], [1] * 43, 16, 2, 128, seed=13)
    want = c.run().clone()
    for _ in range(3):
        assert torch.equal(c.run(), want)
    args = (c.q, c.cache, c.table, i32(c.lens), i32(c.groups), i32(c.prefixes))
    graphs = []
    for _ in range(2):  # two graphs of one pool, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=graphs[0][0].pool() if graphs else None):
            graphs.append((g, fc2.mxfp4_cache_attention_shared(*args, always=True)))
    for g, out in graphs + graphs:
        g.replay()
        assert torch.equal(out, want)


@pytest.mark.parametrize("hq,dim,n,nq", [(32, 128, 24, 1), (8, 64, 60, 1), (16, 64, 10, 3), (8, 256, 20, 1)])
def test_by_the_estimate(hq, dim, n, nq):
    """Large block tables are worth sharing, small ones are not: the bits of the one
    way or of the other."""
    c = Shared([n], [96], [100 + i for i in range(n)], [nq] * n, hq, 2, dim, seed=n)
    shared = c.run().clone()
    apart = c.run(always=False).clone()
    starts = i32(c.starts)
    assert torch.equal(apart, fc2.mxfp4_cache_attention(c.q, c.cache, c.table, i32(c.lens), starts, nq))
    c.table = torch.cat((c.table, torch.zeros(n, 20000, dtype=torch.int32, device="cuda")), 1)
    assert torch.equal(c.run(always=False, explicit=True), c.run(explicit=True))
    assert not torch.equal(shared, apart)


def test_refusals():
    c = Shared([2], [64], [70, 81], [1, 1], 8, 2, 64, seed=14)
    f = fc2.mxfp4_cache_attention_shared
    lens, groups, shared = i32(c.lens), i32(c.groups), i32(c.prefixes)
    for args, kw, match in [((groups[:1], shared), {}, "groups"), ((groups.long(), shared), {}, "groups"),
                            ((groups, shared.float()), {}, "shared"), ((groups, shared), {"max_group": -1}, "max_group"),
                            ((groups, shared), {"max_group": 0}, "no query"), ((groups, shared.cpu()), {}, "device")]:
        with pytest.raises(ValueError, match=match):
            f(c.q, c.cache, c.table, lens, *args, **kw)
    with pytest.raises(ValueError, match="gradient"):
        f(c.q.clone().requires_grad_(), c.cache, c.table, lens, groups, shared)


@pytest.mark.parametrize("hq,nq", [(8, 1), (256, 1), (32, 5)])
def test_pages_past_32_bits(hq, nq):
    """Pages behind 4 GB of codes: the bits of the same pages in a small cache."""
    big, small = fc2.empty_mxfp4_cache(16420, 256, 8, 256), fc2.empty_mxfp4_cache(24, 256, 8, 256)
    assert big.k_codes.numel() > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(3)
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        t = getattr(small, name)
        t.random_(0, 256, generator=g) if "codes" in name else t.random_(118, 128, generator=g)
        getattr(big, name)[16396:] = t
    table = torch.randperm(24, generator=torch.Generator().manual_seed(4)).to(torch.int32).reshape(3, 8)
    table[1:, :4] = table[0, :4]
    q = torch.randn(3 * nq, hq, 256, generator=g, device="cuda").bfloat16()
    args = i32([0, 3]), i32([1024]), i32([0, nq, 2 * nq, 3 * nq]), nq
    for always in (False, True):
        out = [fc2.mxfp4_cache_attention_shared(q, c, (table + add).cuda(), i32([2000, 1500, 1100]), *args,
                                                always=always) for c, add in ((small, 0), (big, 16396))]
        assert torch.equal(out[0].view(torch.int16), out[1].view(torch.int16))
