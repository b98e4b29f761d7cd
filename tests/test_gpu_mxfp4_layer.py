"""The operators together, as examples/mxfp4_attention_layer.py runs them:
prompts by chunks, then decoding from a graph."""
import importlib.util
import os

import pytest
import torch

import diffusion_transformer_mlp_gb300 as fc2
import _mx as mx

pytestmark = pytest.mark.gpu

_path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mxfp4_attention_layer.py")
_spec = importlib.util.spec_from_file_location("mxfp4_attention_layer", _path)
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)

HIDDEN, HQ, HKV, DIM, PAGE = 320, 8, 2, 64, 16
PROMPTS = [37, 200, 1]


def make(seed=0, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    per_seq = -(-(max(PROMPTS) + 20) // PAGE)
    table = torch.randperm(per_seq * len(PROMPTS), generator=g, device="cuda").to(torch.int32).view(-1, per_seq)
    layer = example.AttentionLayer(rand((HQ + 2 * HKV) * DIM, HIDDEN) * HIDDEN ** -0.5,
                                   rand(HIDDEN, HQ * DIM) * (HQ * DIM) ** -0.5, HQ, HKV, DIM, table.numel(), PAGE, **kw)
    return layer, [rand(n, HIDDEN) for n in PROMPTS], table


def read(layer, table, lens):
    starts = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    return fc2.mxfp4_cache_read(layer.cache, table, starts, sum(lens), dtype=torch.float32)


def plain(layer, x, lens, n, table, window=0, sinks=0):
    """The layer in binary64 from its own quantised weights; activations are
    rounded where the operators round them (to bf16, to MXFP4)."""
    w_qkv, w_out = (fc2.mxfp4_dequantize(w, torch.float32).double() for w in (layer.w_qkv, layer.w_out))
    qkv = (mx.values(x) @ w_qkv.T).to(torch.bfloat16).double().unflatten(1, (-1, DIM))
    q, k, v = qkv.split((HQ, HKV, HKV), 1)
    start = [0]
    for m in n:
        start.append(start[-1] + m)
    o = torch.zeros_like(q)
    for b, m in enumerate(n):
        rows = slice(start[b], start[b + 1])
        kb, vb = mx.values(k[rows]), mx.values(v[rows])
        for h in range(HQ):
            s = q[rows, h] @ kb[:, h // (HQ // HKV)].T * DIM ** -0.5
            i, j = torch.arange(m, device="cuda").unsqueeze(1), torch.arange(m, device="cuda")
            seen = (j <= i) & ((j > i - window) | (j < sinks) if window else j >= 0)
            o[rows, h] = torch.softmax(s.masked_fill(~seen, -float("inf")), 1) @ vb[:, h // (HQ // HKV)]
    return mx.values(o.to(torch.bfloat16).flatten(1)) @ w_out.T


@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_prompts_by_chunks(window, sinks):
    """Whatever the chunks, the cache holds the same bytes and the outputs are
    those of the plain layer.  An activation next to the middle of two codes may
    round the other way here and there (a code is a third of its value at
    most, one of 512 of a row's products), hence the mean over a row: 2% of its
    norm."""
    layer, x, table = make(window=window, sinks=sinks)
    ref = plain(layer, torch.cat(x), PROMPTS, PROMPTS, table, window, sinks)
    ends = torch.tensor(PROMPTS, device="cuda").cumsum(0) - 1
    kept = None
    for chunk in (1000, 64, 7):
        y = example.take_in(layer, x, table, chunk).double()
        assert float(((y - ref[ends]).norm(dim=1) / ref[ends].norm(dim=1)).max()) < 0.02
        k, v = read(layer, table, PROMPTS)
        if kept is None:
            kept = k.clone(), v.clone()
        assert torch.equal(k, kept[0]) and torch.equal(v, kept[1])


def test_decoding_from_a_graph():
    """A captured step gives what the calls give one by one."""
    layer, x, table = make(seed=3)
    y = example.take_in(layer, x, table, 64)
    lens = torch.tensor(PROMPTS, dtype=torch.int32, device="cuda")
    decoder = example.Decoder(layer, y, table, lens)
    got = [decoder.step().clone() for _ in range(5)]
    k1, v1 = read(layer, table, [n + 5 for n in PROMPTS])
    step = y
    for i in range(5):
        at = lens.long() + i
        slots = table.gather(1, (at // PAGE).unsqueeze(1)).squeeze(1).long() * PAGE + at % PAGE
        step = layer(step, slots, table, lens + i + 1)
        assert torch.equal(step, got[i]), i
    k2, v2 = read(layer, table, [n + 5 for n in PROMPTS])
    assert torch.equal(k1, k2) and torch.equal(v1, v2)
