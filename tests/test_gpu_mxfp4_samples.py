"""Rotary positions, pages and attention over a shared prefix together, as
examples/mxfp4_parallel_samples.py runs them."""
import importlib.util
import os

import pytest
import torch

import diffusion_transformer_mlp_gb300 as fc2
import _mx as mx

pytestmark = pytest.mark.gpu

_path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mxfp4_parallel_samples.py")
_spec = importlib.util.spec_from_file_location("mxfp4_parallel_samples", _path)
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)

HIDDEN, HQ, HKV, DIM, PAGE, SAMPLES, STEPS = 320, 8, 2, 64, 16, 3, 40


def rotate(x, w, positions):
    y = x.double()
    y = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
    t = positions.double().unsqueeze(1) * 10000.0 ** (-torch.arange(DIM // 2, device="cuda", dtype=torch.float64) / (DIM // 2))
    c, s = t.cos().unsqueeze(1), t.sin().unsqueeze(1)
    a, b = y[..., :DIM // 2], y[..., DIM // 2:]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def plain(layer, x):
    """The layer's output for the last of the tokens x [n, hidden] of one sequence, in binary64 with the
    operators' roundings (to bf16, to MXFP4)."""
    w_qkv, w_out = (fc2.mxfp4_dequantize(w, torch.float32).double() for w in (layer.w_qkv, layer.w_out))
    q, k, v = (mx.values(x) @ w_qkv.T).to(torch.bfloat16).unflatten(1, (-1, DIM)).split((HQ, HKV, HKV), 1)
    pos = torch.arange(len(x), device="cuda")
    q = rotate(q[-1:], layer.q_weight, pos[-1:]).to(torch.bfloat16).double()
    k, v = mx.values(rotate(k, layer.k_weight, pos)), mx.values(v)
    o = torch.stack([torch.softmax(q[0, h] @ k[:, h // (HQ // HKV)].T * DIM ** -0.5, 0) @ v[:, h // (HQ // HKV)]
                     for h in range(HQ)])
    return mx.values(o.to(torch.bfloat16).flatten().unsqueeze(0)) @ w_out.T


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("prompts", [[37, 200], [16, 1, 64]])
def test_samples(prompts):
    """Every step of every sample against the plain layer on the tokens that the
    sample has seen (samples part because their inputs do).  An activation next to
    the middle of two codes may round the other way, and one next to a power of two
    may change its block's scale: an element M = 8 s is then 6 s or 8 s, a quarter
    off, and smaller ones by no more of M than half a step of the coarser grid, an
    eighth.  The block's 32 of the 512 inputs of the output projection carry a
    quarter of the row's norm, or up to 0.4 of it where they are larger: 0.4 / 4 =
    0.1 of the output."""
    g = torch.Generator(device="cuda").manual_seed(len(prompts))
    layer = example.make_layer(HIDDEN, HQ, HKV, DIM, prompts, SAMPLES, PAGE, STEPS, g)
    x = [torch.randn(n, HIDDEN, generator=g, device="cuda").to(torch.bfloat16) for n in prompts]
    y = layer.take_in(x)
    for p, xp in enumerate(x):
        assert off(y[p * SAMPLES], plain(layer, xp)[0]) < 0.1
    history = [xp for xp in x for _ in range(SAMPLES)]
    y = (y + 0.5 * torch.randn(y.shape, generator=g, device="cuda").to(torch.bfloat16))
    sampler = example.Sampler(layer, y)
    for step in range(STEPS):
        history = [torch.cat((h, sampler.x[r:r + 1])) for r, h in enumerate(history)]
        y = sampler.step()
        if step in (0, 1, 15, 16, STEPS - 1):
            for r, h in enumerate(history):
                assert off(y[r], plain(layer, h)[0]) < 0.1, (step, r)
    # what is held is what the rows hold, shared once
    held = torch.zeros_like(layer.pages.refs)
    for b, n in enumerate(layer.pages.lens.tolist()):
        held[layer.pages.table[b, :-(-n // PAGE)].long()] += 1
    assert torch.equal(held, layer.pages.refs)
    assert layer.pages.lens.tolist() == [n + STEPS for n in prompts for _ in range(SAMPLES)]
    for p, n in enumerate(prompts):
        assert bool((layer.pages.refs[layer.pages.table[p * SAMPLES, :n // PAGE].long()] == SAMPLES).all())
    # compact: the same tokens in fewer ids
    starts = torch.cat((layer.pages.lens.new_zeros(1), layer.pages.lens)).cumsum(0).to(torch.int32)
    total = int(starts[-1])
    fc2.mxfp4_pages_select(layer.pages, torch.arange(len(y), dtype=torch.int32, device="cuda"))
    before = fc2.mxfp4_cache_read(layer.cache, layer.pages.table, starts, total)
    moves, used = fc2.mxfp4_pages_compact(layer.pages)
    fc2.mxfp4_cache_copy(layer.cache, moves)
    after = fc2.mxfp4_cache_read(layer.cache, layer.pages.table, starts, total)
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    assert int(used) == int((layer.pages.refs > 0).sum()) and bool((layer.pages.refs[int(used):] == 0).all())


def test_graph_and_calls_alike():
    """Replayed steps give the bits of the calls one by one; and sharing or not
    changes the attention by roundings only."""
    prompts = [50, 90]
    outs = []
    for replay in (True, False):
        g = torch.Generator(device="cuda").manual_seed(9)
        layer = example.make_layer(HIDDEN, HQ, HKV, DIM, prompts, SAMPLES, PAGE, 20, g)
        x = [torch.randn(n, HIDDEN, generator=g, device="cuda").to(torch.bfloat16) for n in prompts]
        y = layer.take_in(x)
        counts = torch.ones(len(y), dtype=torch.int32, device="cuda")
        sampler = example.Sampler(layer, y) if replay else None
        got = []
        for _ in range(20):
            y = sampler.step().clone() if replay else layer.step(y, counts)
            got.append(y)
        outs.append(torch.stack(got))
    assert torch.equal(outs[0], outs[1])
