"""An attention layer in MXFP4, serving: 4-bit weights and a 4-bit paged KV
cache.  Prompts are taken in by chunks, then every sequence decodes a token a
step from a CUDA graph.

    python examples/mxfp4_attention_layer.py [--prompts 100 4000 1500] [--chunk 512] [--steps 64]

Weights and activations are random; the layer's outputs feed its next inputs,
as a model's further layers would.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import diffusion_transformer_mlp_gb300 as fc2  # noqa: E402


class AttentionLayer:
    """qkv projection, cache, attention and output projection of one layer.
    Token t of sequence b lies in page table[b, t // page_size]."""

    def __init__(self, w_qkv: torch.Tensor, w_out: torch.Tensor, q_heads: int, kv_heads: int, dim: int, pages: int,
                 page_size: int, window: int = 0, sinks: int = 0):
        self.q_heads, self.kv_heads, self.dim = q_heads, kv_heads, dim
        self.window, self.sinks = window, sinks
        self.w_qkv, self.w_out = fc2.mxfp4_quantize(w_qkv), fc2.mxfp4_quantize(w_out)
        self.cache = fc2.empty_mxfp4_cache(pages, page_size, kv_heads, dim, device=w_qkv.device)

    def __call__(self, x, slots, table, lens, q_starts=None, max_queries=None):
        """x [tokens, hidden]: the new tokens of all sequences; slots [tokens]
        int64 where they go in the cache; lens [seqs] int32 with them counted.
        Without q_starts every sequence has one new token."""
        q, k, v = fc2.mxfp4_linear(x, self.w_qkv).unflatten(1, (-1, self.dim)).split(
            (self.q_heads, self.kv_heads, self.kv_heads), 1)
        fc2.mxfp4_cache_write(self.cache, k, v, slots)
        o = fc2.mxfp4_cache_attention(q, self.cache, table, lens, q_starts, max_queries, window=self.window,
                                      sinks=self.sinks)
        return fc2.mxfp4_linear(o.flatten(1), self.w_out)


def take_in(layer: AttentionLayer, x: list[torch.Tensor], table: torch.Tensor, chunk: int) -> torch.Tensor:
    """Prompts x[b] [n_b, hidden], `chunk` tokens of each at a time.  Returns
    the last token's output of every sequence."""
    page, last = layer.cache.page_size, [None] * len(x)
    for t0 in range(0, max(len(p) for p in x), chunk):
        part = [p[t0:t0 + chunk] for p in x]
        n = torch.tensor([len(p) for p in part])
        slots = torch.cat([table[b, torch.arange(t0, t0 + len(p), device=table.device) // page].long() * page +
                           torch.arange(t0, t0 + len(p), device=table.device) % page for b, p in enumerate(part)])
        lens = torch.tensor([min(len(p), t0 + chunk) for p in x], dtype=torch.int32, device=table.device)
        starts = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])
        y = layer(torch.cat(part), slots, table, lens, starts.to(device=table.device, dtype=torch.int32), int(n.max()))
        for b, p in enumerate(part):
            if len(p):
                last[b] = y[starts[b + 1] - 1]
    return torch.stack(last)


class Decoder:
    """One token a sequence and call; the step is captured once and replayed."""

    def __init__(self, layer: AttentionLayer, x: torch.Tensor, table: torch.Tensor, lens: torch.Tensor):
        self.layer, self.table = layer, table
        self.x, self.lens = x.clone(), lens.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self._step()  # loads modules and fills the allocator's pools before the capture
            self.x.copy_(x)
            self.lens.copy_(lens)
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self._step()

    def _step(self):
        page = self.layer.cache.page_size
        at = self.lens.long()  # the new token's position
        slots = self.table.gather(1, (at // page).unsqueeze(1)).squeeze(1).long() * page + at % page
        self.lens += 1
        self.x.copy_(self.layer(self.x, slots, self.table, self.lens))

    def step(self) -> torch.Tensor:
        self.graph.replay()
        return self.x


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--prompts", type=int, nargs="+", default=[100, 4000, 1500, 8000])
    p.add_argument("--chunk", type=int, default=512)
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--hidden", type=int, default=5376)
    p.add_argument("--heads", type=int, nargs=3, default=[32, 8, 128], metavar=("Q", "KV", "DIM"))
    p.add_argument("--page", type=int, default=64)
    p.add_argument("--window", type=int, default=0)
    p.add_argument("--sinks", type=int, default=0)
    a = p.parse_args()
    hq, hkv, dim = a.heads
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    per_seq = -(-(max(a.prompts) + a.steps) // a.page)
    table = torch.randperm(per_seq * len(a.prompts), generator=g, device="cuda").to(torch.int32).view(-1, per_seq)
    layer = AttentionLayer(rand((hq + 2 * hkv) * dim, a.hidden) * a.hidden ** -0.5,
                           rand(a.hidden, hq * dim) * (hq * dim) ** -0.5, hq, hkv, dim, table.numel(), a.page,
                           a.window, a.sinks)
    x = [rand(n, a.hidden) for n in a.prompts]
    take_in(layer, x, table, a.chunk)  # warm-up
    t = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    t[0].record()
    y = take_in(layer, x, table, a.chunk)
    t[1].record()
    decoder = Decoder(layer, y, table, torch.tensor(a.prompts, dtype=torch.int32, device="cuda"))
    t[2].record()
    for _ in range(a.steps):
        y = decoder.step()
    t[3].record()
    torch.cuda.synchronize()
    assert bool(torch.isfinite(y).all())
    print(f"prompts: {sum(a.prompts)} tokens in {t[0].elapsed_time(t[1]):.2f} ms by chunks of {a.chunk}; "
          f"decoding: {t[2].elapsed_time(t[3]) / a.steps * 1000:.1f} us a step of {len(a.prompts)} tokens")
    bits = 8 * sum(c.nbytes for c in (layer.cache.k_codes, layer.cache.k_scales, layer.cache.v_codes,
                                      layer.cache.v_scales))
    print(f"cache: {bits / 8e6:.1f} MB, {bits / (2 * layer.cache.k_codes.numel() * 2):.2f} bits an element")


if __name__ == "__main__":
    main()
