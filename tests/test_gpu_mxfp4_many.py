"""Attention over the cache for many segments (sequences times kv heads times row
tiles, 1,024 and more), whose partials are joined by the boundaries between the
workers' runs; a long sequence among them has many."""
import pytest
import torch

import diffusion_transformer_mlp_gb300 as fc2
from test_gpu_mxfp4_cache import check, run_attention

pytestmark = pytest.mark.gpu


def lengths(n, seed, longer=()):
    lens = torch.randint(0, 700, (n,), generator=torch.Generator().manual_seed(seed)).tolist()
    for i, v in longer:
        lens[i] = v
    return lens


@pytest.mark.parametrize("dim,hq,hkv,n", [(64, 32, 32, 32), (64, 32, 32, 33), (128, 64, 16, 67), (256, 64, 32, 34)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_short_sequences(dim, hq, hkv, n, dtype):
    check(*run_attention(lengths(n, n), [1] * n, hq, hkv, dim, 32, dtype, seed=n)[:5])


@pytest.mark.parametrize("dim,hq,hkv", [(64, 32, 32), (128, 32, 16), (256, 32, 16)])
def test_long_sequences_among_them(dim, hq, hkv):
    lens = lengths(67, 5, [(0, 9001), (5, 7000), (6, 6500), (12, 0), (13, 0), (14, 0), (66, 9999)])
    check(*run_attention(lens, [1] * 67, hq, hkv, dim, 64, torch.bfloat16, seed=6)[:5])


@pytest.mark.parametrize("dim,causal", [(64, True), (128, True), (256, True), (128, False)])
def test_several_queries(dim, causal):
    nq = [(0, 1, 4, 2, 6)[b % 5] for b in range(35)]  # queries before every key, and no query
    lens = lengths(35, 9, [(2, 1), (4, 3), (9, 0), (33, 5000)])
    check(*run_attention(lens, nq, 64, 32, dim, 16, torch.bfloat16, seed=10, causal=causal)[:5])


def test_rows_of_several_tiles():
    nq = [(1, 5, 0, 8)[b % 4] for b in range(37)]  # up to 32 rows: two tiles
    lens = lengths(37, 13, [(1, 2), (3, 4), (20, 3000)])
    check(*run_attention(lens, nq, 64, 16, 128, 64, torch.bfloat16, seed=14)[:5])


def test_window_and_sinks():
    lens = lengths(40, 11, [(7, 6000), (30, 9000)])
    check(*run_attention(lens, [1] * 40, 64, 32, 64, 64, torch.bfloat16, seed=12, window=2500, sinks=3)[:5])


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_queries_at_odd_places(dim):
    """Rows of a kv head by the hundred, whose loads are not aligned to 16 bytes: the same bits."""
    out, lse, _, _, _, (q, cache, table, lens, starts, most) = run_attention(
        [300, 77, 5], [200, 77, 9], 6, 2, dim, 16, torch.bfloat16, seed=15)
    wide = torch.zeros(len(q), 6, dim + 3, dtype=q.dtype, device="cuda")
    wide[..., 1:dim + 1] = q
    odd = fc2.mxfp4_cache_attention(wide[..., 1:dim + 1], cache, table, lens, q_starts=starts, max_queries=most)
    assert torch.equal(odd.view(torch.int16), out.view(torch.int16))
