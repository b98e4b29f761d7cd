"""Results of the attention over the cache that do not depend on how a call is
carried out: partials joined by segments or by the boundaries between runs, tiles
counted by each warp or by a block, outputs in 16 bits or in binary32."""
import pytest
import torch

import diffusion_transformer_mlp_gb300 as fc2
from test_gpu_mxfp4_many import lengths

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Batch:
    def __init__(self, lens, nq, hq, hkv, dim, page=32, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.nq = lens, nq
        self.cache = fc2.empty_mxfp4_cache(200, page, hkv, dim)
        for t in (self.cache.k_codes, self.cache.v_codes):
            t.random_(0, 256, generator=g)
        for t in (self.cache.k_scales, self.cache.v_scales):
            t.random_(118, 128, generator=g)
        width = max(1, max(-(-n // page) for n in lens))
        self.table = torch.randint(0, 200, (len(lens), width), generator=g, device="cuda", dtype=torch.int32)
        self.q = torch.randn(sum(nq), hq, dim, generator=g, device="cuda").bfloat16()

    def run(self, empty=0, f=fc2.mxfp4_cache_attention, groups=(), **kw):
        """(out, lse) of the batch's own rows, with `empty` sequences of no keys behind it."""
        one = all(n == 1 for n in self.nq)
        q = torch.cat((self.q, self.q[:1].expand(empty, -1, -1))) if one else self.q
        starts = None if one else i32([0] + self.nq + [0] * empty).cumsum(0).to(torch.int32)
        table = torch.cat((self.table, self.table[:1].expand(empty, -1)))
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        out = f(q, self.cache, table.contiguous(), i32(self.lens + [0] * empty), *groups, q_starts=starts,
                max_queries=max(self.nq), lse=lse, **kw)
        n = len(self.q)
        assert bool((out[n:] == 0).all()) and bool(torch.isneginf(lse[n:]).all())
        return out[:n], lse[:n]


def same(a, b):
    return torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dim,hq,hkv,n,nq,empty", [
    (64, 32, 8, 30, (1,), 200), (128, 32, 8, 100, (1,), 60), (128, 8, 8, 20, (1,), 300), (256, 32, 4, 60, (1,), 300),
    (128, 32, 2, 70, (1,), 954), (64, 64, 4, 90, (1,), 500), (128, 16, 8, 80, (2, 1, 0, 3), 300),
    (256, 16, 4, 50, (4, 2, 3), 500), (128, 32, 4, 60, (2, 1, 0, 2), 500), (64, 32, 4, 60, (8, 0, 3), 200)])
def test_joined_by_segments_or_by_boundaries(dim, hq, hkv, n, nq, empty):
    """Sequences without keys add to the segments that a join is chosen by, and to no
    worker's run."""
    lens = lengths(n, n + dim, [(1, 30001), (3, 2), (n // 2, 9000), (n - 1, 5000)])
    b = Batch(lens, [nq[i % len(nq)] for i in range(n)], hq, hkv, dim, seed=n)
    few = b.run()
    many = b.run(empty)
    assert same(few, many)
    assert same(few, b.run(3))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,nq", [(32, 8, (1,)), (32, 2, (1,)), (8, 4, (2, 0, 4)), (32, 4, (2, 1)), (64, 8, (2, 2, 1))])
@pytest.mark.parametrize("n", [5, 70])
def test_outputs_by_way_of_binary32(dim, hq, hkv, nq, n):
    """Groups that share nothing: the parts' binary32 outputs, rounded at the end."""
    lens = lengths(n, n + dim, [(0, 7000), (3, 1)])
    b = Batch(lens, [nq[i % len(nq)] for i in range(n)], hq, hkv, dim, seed=n + 1)
    ordinary = b.run()
    groups = torch.arange(n + 1, dtype=torch.int32, device="cuda"), i32([0] * n)
    assert same(ordinary, b.run(f=fc2.mxfp4_cache_attention_shared, groups=groups, max_group=max(nq), always=True))
