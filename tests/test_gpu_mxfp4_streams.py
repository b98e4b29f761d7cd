"""The MXFP4 functions on a stream that is not the current one: workspaces and
outputs belong to the stream of the call."""
import pytest
import torch

import diffusion_transformer_mlp_gb300 as fc2
from test_gpu_mxfp4_hidden import Case

pytestmark = pytest.mark.gpu

DELAY = 40_000_000  # cycles, about 20 ms: far longer than the host takes for what follows


def linear(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(70, 2048, generator=g, device="cuda", dtype=torch.bfloat16)
    w = fc2.mxfp4_quantize(torch.randn(1000, 2048, generator=g, device="cuda", dtype=torch.bfloat16))
    return lambda **kw: fc2.mxfp4_linear(x, w, **kw)


def attention(nq):
    def make(seed):
        case = Case([3000, 700], [nq, nq], 8, 2, 64, seed=seed)
        case.write()
        lens = torch.tensor(case.lens, dtype=torch.int32, device="cuda")
        starts = torch.tensor(case.starts, dtype=torch.int32, device="cuda")
        return lambda **kw: fc2.mxfp4_cache_attention(case.q, case.cache, case.table, lens, starts, nq, **kw)
    return make


def quantize(seed):
    x = torch.randn(300, 2048, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
    return lambda **kw: fc2.mxfp4_quantize(x, **kw).qdata


def dequantize(seed):
    t = fc2.mxfp4_quantize(torch.randn(300, 2048, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
    return lambda **kw: fc2.mxfp4_dequantize(t, **kw)


def cache_read(seed):
    case = Case([300], [1], 2, 2, 64, seed=seed)
    case.write()
    starts = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    return lambda **kw: fc2.mxfp4_cache_read(case.cache, case.table, starts, 300, **kw)[0]


CALLS = [linear, attention(1), attention(40), quantize, dequantize, cache_read]
IDS = ["linear", "attention of few rows", "attention of many rows", "quantize", "dequantize", "cache_read"]


@pytest.mark.parametrize("make", CALLS, ids=IDS)
def test_workspaces_are_not_handed_out_while_in_use(make):
    """Memory that the call has given back is not the current stream's."""
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


@pytest.mark.parametrize("make", CALLS, ids=IDS)
def test_outputs_are_not_what_the_current_stream_still_reads(make):
    """A block that was freed here, but is still to be read here."""
    call = make(2)
    want = call()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    olds = [torch.full_like(want, 3) for _ in range(4)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(DELAY)
    copies = [t.clone() for t in olds]
    olds.clear()
    out = call(stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all(bool((t == 3).all()) for t in copies)


@pytest.mark.parametrize("make", CALLS, ids=IDS)
def test_outputs_stay_while_the_current_stream_reads_them(make):
    first, second = make(3), make(4)
    want = first()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = first(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(DELAY)
    copy = out.clone()
    del out
    others = [second(stream=s) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and len(others) == 3


def test_streams_of_every_kind():
    call = linear(5)
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (torch.cuda.default_stream(), torch.cuda.current_stream(), side, torch.cuda.ExternalStream(side.cuda_stream)):
        out = call(stream=s)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        with torch.cuda.stream(side):
            out = call(stream=s)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    with pytest.raises(AttributeError):
        call(stream=7)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(stream=torch.cuda.current_stream())
    out.zero_()
    g.replay()
    assert torch.equal(out, want)
