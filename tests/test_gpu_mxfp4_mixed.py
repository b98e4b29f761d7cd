"""Attention over a shared prefix of batches in which most sequences share nothing:
the results, what is written for the queries outside of the groups, and which way
a call takes."""
import ctypes

import pytest
import torch

import diffusion_transformer_mlp_gb300 as fc2
from diffusion_transformer_mlp_gb300 import _lib
from test_gpu_mxfp4_shared import Shared, i32
from test_mxfp4_abi import Attention, Cache
from test_mxfp4_more_abi import SharedArgs

pytestmark = pytest.mark.gpu


def mixed(grouped, others, lead, hq, hkv, dim, prefix=70, nq=1, seed=0):
    """`grouped` sequences of one prefix, `lead` of the `others` before them."""
    lens = [1 + (i * 29) % 150 for i in range(others)]
    lens[lead:lead] = [prefix + nq + (i * 13) % 90 for i in range(grouped)]
    return Shared([grouped], [prefix], lens, [min(nq, n) for n in lens], hq, hkv, dim, seed=seed, lead=lead)


@pytest.mark.parametrize("hq,hkv,dim,grouped,others,lead", [
    (8, 8, 64, 4, 200, 0), (8, 8, 64, 4, 200, 77), (32, 8, 128, 2, 140, 140), (16, 16, 128, 8, 130, 3),
    (32, 4, 64, 2, 520, 9), (8, 4, 256, 3, 300, 100), (4, 2, 64, 4, 1500, 1100), (8, 2, 64, 3, 5, 2), (16, 2, 128, 5, 9, 0)])
def test_few_of_many(hq, hkv, dim, grouped, others, lead):
    """One query a sequence, and a bound of a group's queries that leaves few rows."""
    c = mixed(grouped, others, lead, hq, hkv, dim, seed=grouped + lead)
    c.run(max_group=grouped)
    c.check()
    c.run(max_group=grouped, explicit=True)
    c.check()


def address(t):
    return t.data_ptr()


def call(c, max_group, workspace, always=1):
    """The C entry point on a workspace of the test's own; returns its status."""
    pages, hkv, page, half = c.cache.k_codes.shape
    cache = Cache()
    for f in ("k_codes", "k_scales", "v_codes", "v_scales"):
        setattr(cache, f, address(getattr(c.cache, f)))
    cache.pages, cache.page_size, cache.kv_heads, cache.dim = pages, page, hkv, 2 * half
    c.out = torch.zeros_like(c.q)
    c.lse = torch.full((len(c.q), c.q.shape[1]), 7.0, device="cuda")
    held = [i32(v) for v in (c.lens, c.groups, c.prefixes, c.starts)]
    a = Attention()
    a.q, a.out, a.lse, a.table, a.lens, a.q_starts = map(address, (c.q, c.out, c.lse, c.table, held[0], held[3]))
    a.workspace, a.workspace_bytes = address(workspace), workspace.numel()
    a.q_st, a.q_sh, a.o_st, a.o_sh = *c.q.stride()[:2], *c.out.stride()[:2]
    a.table_ld, a.seqs, a.total_q, a.max_queries = c.table.shape[1], len(c.lens), len(c.q), max(c.nq)
    a.q_heads, a.dtype, a.causal, a.scale = c.q.shape[1], 0, 1, c.dim ** -0.5
    s = SharedArgs()
    s.groups, s.shared, s.count, s.max_group, s.always = address(held[1]), address(held[2]), len(c.prefixes), max_group, always
    torch.cuda.synchronize()
    status = _lib.load().mxfp4_cache_attention_shared(ctypes.byref(cache), ctypes.byref(a), ctypes.byref(s), None)
    torch.cuda.synchronize()
    return status


@pytest.mark.parametrize("hq,hkv,dim,grouped,others", [(8, 8, 64, 4, 200), (32, 8, 128, 2, 200), (64, 16, 128, 4, 200)])
def test_nothing_is_worked_out_for_queries_outside(hq, hkv, dim, grouped, others):
    """They have no prefix, and no part of the outputs is written for one: the
    workspace keeps its bytes, where rows of zeros were."""
    c = mixed(grouped, others, 0, hq, hkv, dim, seed=1)
    need = _lib.load().mxfp4_attention_shared_workspace_bytes(hkv, hq, dim, len(c.q), 1, len(c.lens), c.table.shape[1], 1,
                                                              grouped)
    workspace = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
    assert call(c, grouped, workspace) == _lib.NVFP4_OK
    c.check()
    zeros = int((workspace.view(torch.int32) == 0).sum())
    assert zeros < others * hq * dim // 8


@pytest.mark.parametrize("hq,hkv,dim,grouped,others,nq", [(32, 8, 128, 2, 126, 1), (32, 8, 128, 8, 300, 1),
                                                          (8, 8, 64, 2, 150, 1), (16, 4, 256, 3, 90, 1), (8, 4, 64, 2, 60, 3),
                                                          (32, 8, 128, 4, 124, 4)])
def test_sequences_outside_save_nothing(hq, hkv, dim, grouped, others, nq):
    """A small group among many sequences is not worth sharing, however large the
    block tables are: the bits of the ordinary attention.  One that most belong to is."""
    c = mixed(grouped, others, 5, hq, hkv, dim, nq=nq, seed=grouped)
    c.table = torch.cat((c.table, torch.zeros(len(c.lens), 1000 - c.table.shape[1], dtype=torch.int32, device="cuda")), 1)
    apart = fc2.mxfp4_cache_attention(c.q, c.cache, c.table, i32(c.lens), i32(c.starts), max(c.nq))
    assert not torch.equal(c.run(max_group=sum(c.nq[5:5 + grouped])), apart)
    assert torch.equal(c.run(always=False, max_group=sum(c.nq[5:5 + grouped])), apart)
    c = mixed(others, grouped, 1, hq, hkv, dim, nq=nq, seed=grouped)
    c.table = torch.cat((c.table, torch.zeros(len(c.lens), 1000 - c.table.shape[1], dtype=torch.int32, device="cuda")), 1)
    kw = dict(max_group=sum(c.nq[1:1 + others]))
    shared = c.run(**kw).clone()
    assert torch.equal(c.run(always=False, **kw), shared)


@pytest.mark.parametrize("hq,hkv,dim,page", [(8, 2, 64, 16), (8, 2, 128, 64), (6, 2, 256, 32), (32, 2, 128, 16)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_chunks_behind_a_prefix(hq, hkv, dim, page, causal):
    """Hundreds of queries a sequence, beside sequences that decode and one outside."""
    lens, nq = [700, 1201, 513, 400, 90], [300, 801, 1, 17, 33]
    c = Shared([4], [383], lens, nq, hq, hkv, dim, page, seed=dim + page)
    c.run(causal=causal)
    c.check(causal)
