"""The rotary, page and shared-prefix functions on a stream that is not the
current one: workspaces and outputs belong to the stream of the call."""
import pytest
import torch

import diffusion_transformer_mlp_gb300 as fc2
from test_gpu_mxfp4_shared import Shared, i32
from test_gpu_mxfp4_streams import DELAY

pytestmark = pytest.mark.gpu


def rotary(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn(300, 8, 64, generator=g, device="cuda")
    rot = fc2.head_rotary(10.0 ** (-torch.arange(32, dtype=torch.float64)))
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    return lambda **kw: fc2.head_norm_rotary(q, None, rot, pos, **kw)[0]


def write(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(300, 8, 64, generator=g, device="cuda", dtype=torch.bfloat16)
    cache = fc2.empty_mxfp4_cache(20, 16, 2, 64)
    rot = fc2.head_rotary(10.0 ** (-torch.arange(32, dtype=torch.float64)))
    pos, slots = torch.arange(300, dtype=torch.int32, device="cuda"), torch.arange(300, device="cuda")
    return lambda **kw: fc2.mxfp4_cache_write_rotary(cache, x[:, :4], x[:, 4:6], x[:, 6:], slots, rot, pos, **kw)


def shared(nq, n):
    def make(seed):
        c = Shared([n], [500], [600 + i for i in range(n)], [nq] * n, 8, 2, 64, seed=seed)
        args = c.q, c.cache, c.table, i32(c.lens), i32(c.groups), i32(c.prefixes), i32(c.starts), nq
        return lambda **kw: fc2.mxfp4_cache_attention_shared(*args, always=True, **kw)
    return make


def extend(total):
    def make(seed):
        state = [t.clone() for t in (fc2.empty_mxfp4_pages(70000 + seed, 16, 5, 12000).__dict__[n]
                                     for n in ("refs", "table", "lens"))]
        counts = i32([total // 5] * 5)

        def call(stream=None):
            pages = fc2.MXFP4Pages(*(t.clone() for t in state), 16)
            ready = torch.cuda.current_stream().record_event()
            if stream is not None:
                stream.wait_event(ready)
                for t in (pages.refs, pages.table, pages.lens):
                    t.record_stream(stream)
            return fc2.mxfp4_pages_extend(pages, counts, total, stream=stream)[0]
        return call
    return make


CALLS = [rotary, write, shared(1, 4), shared(40, 6), extend(500), extend(500000)]
IDS = ["rotary", "write", "few rows", "many rows", "few tokens", "many tokens"]


@pytest.mark.parametrize("make", CALLS, ids=IDS)
def test_workspaces_are_not_handed_out_while_in_use(make):
    call = make(1)
    want = call()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(DELAY)
    out = call(stream=s)
    taken = [torch.full((1 << b,), 77, dtype=torch.uint8, device="cuda") for b in range(9, 26) for _ in range(3)]
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all(bool((t == 77).all()) for t in taken)


@pytest.mark.parametrize("make", CALLS[:4], ids=IDS[:4])
def test_two_at_once(make):
    """Calls on two streams have workspaces of their own."""
    call = make(3)
    want = call()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [call(stream=s) for _ in range(10) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
