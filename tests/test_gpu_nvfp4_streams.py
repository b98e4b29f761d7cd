"""The NVFP4 functions on a stream that is not the current one: what they
allocate belongs to the stream of the call."""
import pytest
import torch

import diffusion_transformer_mlp_gb300 as fc2

pytestmark = pytest.mark.gpu

M, K, N = 300, 512, 384
DELAY = 40_000_000  # cycles, about 20 ms


def rand(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(torch.bfloat16)


def weight(seed):
    x = rand(N, K, seed=seed)
    return lambda **kw: fc2.nvfp4_quantize_weight(x, **kw).qdata


def swiglu(seed):
    x = rand(M, 2 * K, seed=seed)
    return lambda **kw: fc2.swiglu_nvfp4_quantize(x, **kw).qdata


def step(seed):
    x, w = rand(M, 2 * K, seed=seed), fc2.nvfp4_quantize_weight(rand(N, K, seed=seed + 50))
    return lambda **kw: fc2.fc2(x, w, **kw)


def fc1(seed):
    a, w = fc2.swiglu_nvfp4_quantize(rand(M, 2 * K, seed=seed)), fc2.nvfp4_quantize_weight(rand(256, K, seed=seed + 50))
    return lambda **kw: fc2.nvfp4_fc1_swiglu(a, w, **kw)[0]


CALLS = [weight, swiglu, step, fc1]


@pytest.mark.parametrize("make", CALLS)
def test_memory_of_the_call_is_not_handed_out_while_in_use(make):
    call = make(1)
    want = call()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(DELAY)
    out = call(stream=s)
    taken = [torch.full((1 << b,), 77, dtype=torch.uint8, device="cuda") for b in range(4, 24) for _ in range(3)]
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all(bool((t == 77).all()) for t in taken)


@pytest.mark.parametrize("make", CALLS)
def test_outputs_are_not_what_the_current_stream_still_reads(make):
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


@pytest.mark.parametrize("make", CALLS)
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


def test_host_step_without_a_workspace():
    x = rand(M, 2 * K, seed=7)
    w = fc2.nvfp4_quantize_weight(rand(N, K, seed=8))
    want = fc2.fc2(x, w).cpu()
    host = x.cpu().pin_memory()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(DELAY)
    out, event = fc2.fc2_host(host, w, stream=s, sync=False)
    taken = [torch.full((1 << b,), 77, dtype=torch.uint8, device="cuda") for b in range(4, 24) for _ in range(3)]
    event.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all(bool((t == 77).all()) for t in taken)
