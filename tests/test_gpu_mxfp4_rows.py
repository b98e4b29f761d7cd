"""Attention of many query rows over the MXFP4 cache: the keys of all
(sequence, rows, head) segments are dealt in equal runs over the GPU, so a
segment may be one block's, several blocks', or one of many of a block.
Definition, layout helpers and tolerance are those of the cache's tests."""
import math

import pytest
import torch

import diffusion_transformer_mlp_gb300 as fc2
import _mx as mx
from test_gpu_mxfp4_cache import cache_values, check, fill, make_cache, make_table, run_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,hq,hkv", [(64, 8, 1), (64, 3, 3), (128, 8, 2), (128, 5, 1), (256, 4, 2)])
def test_segments_of_many_blocks(dim, hq, hkv, dtype):
    """Few segments: each is split over many blocks."""
    for lens, nq in (([3000], [100]), ([1500, 700, 64], [65, 129, 64])):
        check(*run_attention(lens, nq, hq, hkv, dim, 16, dtype, seed=dim + hq)[:5])


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_blocks_of_many_segments(dim):
    """More segments than blocks, some without queries, one without keys."""
    g = torch.Generator().manual_seed(dim)
    lens = torch.randint(1, 150, (90,), generator=g).tolist()
    nq = [min(n, int(m)) for n, m in zip(lens, torch.randint(0, 90, (90,), generator=g))]
    lens[7], nq[7], nq[11], lens[40], nq[40] = 0, 2, 0, 150, 150
    check(*run_attention(lens, nq, 4, 4, dim, 32, torch.bfloat16, seed=dim)[:5])


@pytest.mark.parametrize("window,sinks", [(1, 1), (100, 0), (130, 65), (700, 4)])
@pytest.mark.parametrize("causal", [True, False])
def test_windows(window, sinks, causal):
    for dim in (64, 128, 256):
        check(*run_attention([900, 2000], [300, 70], 4, 2, dim, 16, torch.float16, seed=window, window=window,
                             sinks=sinks, causal=causal)[:5])


def test_more_queries_than_keys():
    """Whole row tiles that see nothing, beside one that is split."""
    for dim in (64, 256):
        out, lse, ref, ref_lse, mag, _ = run_attention([0, 5, 2000], [400, 700, 90], 4, 2, dim, 16, torch.bfloat16,
                                                       seed=dim)
        check(out, lse, ref, ref_lse, mag)
        assert bool((out[:1095] == 0).all()) and bool((lse[:1095] == -math.inf).all())


def test_more_sequences_than_one_launch_takes():
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 20, (1100,), generator=g).tolist()
    nq = [min(n, 3) for n in lens]
    nq[1050], lens[1050] = 70, 400
    check(*run_attention(lens, nq, 2, 2, 64, 16, torch.bfloat16, seed=3)[:5])


@pytest.mark.parametrize("nq", [1, 8, 90])
def test_values_near_the_end_of_the_range(nq):
    """Values of 2^100 and of 2^-100, whose sums with the weights' factors must
    not leave the range where partial results are joined."""
    for mul_v in (2.0 ** 100, 2.0 ** -100):
        check(*run_attention([2500, 900], [nq, nq], 8, 1, 128, 16, torch.bfloat16, seed=nq, mul_v=mul_v)[:5])


def test_nan_across_blocks():
    """NaN keys and values reach the queries that see them, however the keys are
    split; the rows before them stay finite."""
    page, hkv, hq, dim = 16, 1, 4, 128
    lens, nq = [1200], [400]
    table, pages = make_table(lens, page, 1)
    cache = make_cache(pages, page, hkv, dim, 2)
    g = torch.Generator(device="cuda").manual_seed(4)
    k = torch.randn(1200, hkv, dim, generator=g, device="cuda")
    v = torch.randn(1200, hkv, dim, generator=g, device="cuda")
    v[900, 0, 5] = math.nan
    v[1100, 0, 70] = math.inf
    k[1150, 0, 64] = math.inf
    fill(cache, table, lens, page, k, v)
    q = torch.randn(400, hq, dim, generator=g, device="cuda").to(torch.bfloat16)
    out = fc2.mxfp4_cache_attention(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    torch.tensor([0, 400], dtype=torch.int32, device="cuda"), 400)
    ref, _, mag = mx.attention(q.double(), *cache_values(cache), table, lens, [0, 400], page, dim ** -0.5)
    assert torch.equal(torch.isnan(out), torch.isnan(ref))
    fine = ~torch.isnan(ref)
    bound = 2.0 ** -8 * 1.01 * ref.abs() + 2.0 ** -10 * mag
    assert bool(((out.double() - ref).abs() <= bound)[fine].all())


@pytest.mark.parametrize("rows", [(1, 16), (2, 16), (4, 16), (5, 13), (9, 8), (64, 1), (65, 1), (17, 1)])
def test_around_the_rule(rows):
    """Row counts on both sides of the choice between the two kernels."""
    nq, group = rows
    for dim in (64, 128, 256):
        check(*run_attention([700, 90], [nq, nq], group, 1, dim, 64, torch.bfloat16, seed=nq)[:5])


def test_strides_and_repeats():
    out, lse, ref, ref_lse, mag, (q, cache, table, lens, qs, mq) = run_attention([300, 1700], [90, 200], 8, 2, 128, 16,
                                                                                 torch.float16, seed=6)
    check(out, lse, ref, ref_lse, mag)
    wide = torch.zeros(290, 11, 128 + 1, dtype=torch.float16, device="cuda")
    qv = wide[:, 2:10, 1:]
    qv.copy_(q)
    buf = torch.full((290, 9, 128 + 1), 5.0, dtype=torch.float16, device="cuda")
    fc2.mxfp4_cache_attention(qv, cache, table, lens, qs, mq, out=buf[:, 1:, :128])
    assert torch.equal(buf[:, 1:, :128], out)
    assert bool((buf[:, 0] == 5).all()) and bool((buf[:, :, 128] == 5).all())
    for _ in range(5):
        assert torch.equal(fc2.mxfp4_cache_attention(q, cache, table, lens, qs, mq), out)
