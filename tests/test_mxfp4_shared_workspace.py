"""The workspace of attention over a shared prefix: as much as the call's own way
takes, which is the ordinary attention's where nothing is shared."""
import ctypes

import pytest
import torch

import diffusion_transformer_mlp_gb300 as fc2
from diffusion_transformer_mlp_gb300 import _lib
from test_mxfp4_abi import BF16, INVALID, NUL, _attention, _cache
from test_mxfp4_more_abi import SharedArgs, made

by = ctypes.byref


def sizes(kv, hq, dim, total, most, seqs, ld, count, max_group, always=0, page=16, **kw):
    """(of the call, the most, the ordinary attention's), and the call's arguments."""
    L = _lib.load()
    c = _cache(kv_heads=kv, dim=dim, page_size=page)
    a = _attention(q_heads=hq, total_q=total, max_queries=most, seqs=seqs, table_ld=ld, **kw)
    s = made(SharedArgs, dict(groups=0x10000, shared=0x10000, count=count, max_group=max_group, always=always), {})
    of_call = L.mxfp4_attention_shared_call_workspace_bytes(by(c), by(a), by(s))
    return (of_call, L.mxfp4_attention_shared_workspace_bytes(kv, hq, dim, total, most, seqs, ld, count, max_group),
            L.mxfp4_attention_workspace_bytes(kv, hq, dim, most)), (c, a, s)


PROMPTS = (8, 64, 128, 8192, 2048, 4, 600, 1, 8192)  # chunks of prompts: their rows fill whole tiles
FEW = (8, 32, 128, 128, 1, 128, 1000, 1, 2)          # two sequences of 128 share something
MOST = (8, 32, 128, 128, 1, 128, 1000, 1, 126)


@pytest.mark.parametrize("args", [PROMPTS, FEW, (8, 32, 64, 4, 1, 4, 40, 1, 4)])
def test_what_is_not_shared_takes_no_room(args):
    (call, most, own), _ = sizes(*args)
    assert call == own < most
    (call, most, own), _ = sizes(*args, always=1)
    assert call == most
    outputs = 2 * args[3] * args[1] * args[2] * 4
    assert most >= own + outputs


def test_what_is_shared_does():
    (call, most, _), _ = sizes(*MOST)
    assert call == most
    (call, _, own), _ = sizes(*MOST[:6], 12, *MOST[7:])  # not with such short tables
    assert call == own
    (call, _, own), _ = sizes(*MOST[:6], 12, *MOST[7:], page=256)  # of such small pages
    assert call > own


def test_no_groups_and_nothing_to_do():
    for kw in (dict(count=0), dict(max_group=0)):
        args = dict(zip(("kv", "hq", "dim", "total", "most", "seqs", "ld", "count", "max_group"), MOST)) | kw
        (call, most, own), _ = sizes(**args, always=1)
        assert call == most == own
    assert sizes(8, 32, 128, 0, 1, 128, 100, 1, 2)[0][0] == 0 and sizes(8, 32, 96, 8, 1, 8, 100, 1, 2)[0][0] == 0
    assert _lib.load().mxfp4_attention_shared_call_workspace_bytes(None, None, None) == 0
    # a count that does not leave 32 bits for what follows it
    assert _lib.load().mxfp4_attention_shared_workspace_bytes(8, 32, 128, 4, 1, 4, 16, 2 ** 31 - 1, 4) > 2 ** 31


@pytest.mark.parametrize("args", [PROMPTS, FEW, MOST])
def test_a_byte_less_is_refused(args):
    (call, _, _), (c, a, s) = sizes(*args)
    a.dtype, a.workspace_bytes = BF16, call - 1
    assert _lib.load().mxfp4_cache_attention_shared(by(c), by(a), by(s), NUL) == INVALID
    assert str(call) in _lib.last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("always", [False, True])
def test_allocated(always):
    """Chunks of prompts behind a prefix, which each sequence reads for itself."""
    from test_gpu_mxfp4_shared import Shared, i32
    c = Shared([2], [160], [1200, 1100], [1024, 900], 32, 8, 128, seed=2)
    args = c.q, c.cache, c.table, i32(c.lens)
    starts = i32(c.starts)
    calls = [lambda: fc2.mxfp4_cache_attention(*args, starts, 1024),
             lambda: fc2.mxfp4_cache_attention_shared(*args, i32(c.groups), i32(c.prefixes), starts, 1024, always=always)]
    taken, outs = [], []
    for f in calls:
        f()
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        outs.append(f())
        torch.cuda.synchronize()
        taken.append(torch.cuda.max_memory_allocated() - before)
    outputs = 2 * c.q.numel() * 4
    if always:
        assert taken[1] >= taken[0] + outputs
    else:
        assert taken[1] <= taken[0] + 4096 and torch.equal(*outs)
