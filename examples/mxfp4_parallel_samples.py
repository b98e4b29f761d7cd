"""Several samples of each prompt from one attention layer in MXFP4: the prompts
are taken in once, their rows of the block table fork, and the samples decode
from a CUDA graph, with norms of queries and keys, rotary positions, pages that
are copied when a sample first writes in one that others hold, and attention
that reads a prompt once for all its samples.

    python examples/mxfp4_parallel_samples.py [--prompts 3000 9000] [--samples 16] [--steps 64]

Weights and activations are random; the layer's outputs feed its next inputs.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import diffusion_transformer_mlp_gb300 as fc2  # noqa: E402


class SampledLayer:
    """qkv projection, norm and rotation into the cache, attention and output
    projection of one layer; row p * samples + i of the pages is sample i of
    prompt p."""

    def __init__(self, w_qkv, w_out, q_weight, k_weight, q_heads, kv_heads, dim, rotary, pages: fc2.MXFP4Pages, samples):
        self.q_heads, self.kv_heads, self.dim, self.samples = q_heads, kv_heads, dim, samples
        self.w_qkv, self.w_out = fc2.mxfp4_quantize(w_qkv), fc2.mxfp4_quantize(w_out)
        self.q_weight, self.k_weight, self.rotary, self.pages = q_weight, k_weight, rotary, pages
        self.cache = fc2.empty_mxfp4_cache(len(pages.refs), pages.page_size, kv_heads, dim, device=w_qkv.device)
        rows = len(pages.lens)
        self.groups = torch.arange(0, rows + 1, samples, dtype=torch.int32, device=w_qkv.device)
        self.shared = torch.zeros(rows // samples, dtype=torch.int32, device=w_qkv.device)

    def _project(self, x, slots, positions):
        q, k, v = fc2.mxfp4_linear(x, self.w_qkv).unflatten(1, (-1, self.dim)).split(
            (self.q_heads, self.kv_heads, self.kv_heads), 1)
        return fc2.mxfp4_cache_write_rotary(self.cache, q, k, v, slots, self.rotary, positions, self.q_weight,
                                            self.k_weight)

    def take_in(self, x: list[torch.Tensor]) -> torch.Tensor:
        """Prompts x[p] [n_p, hidden] into their first rows, which fork.  Returns
        the last token's output for every row."""
        n, dev = [len(p) for p in x], x[0].device
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
        counts = [c for m in n for c in [m] + [0] * (self.samples - 1)]
        slots, _, missing = fc2.mxfp4_pages_extend(self.pages, i32(counts), sum(n))
        if int(missing) != 0:
            raise RuntimeError(f"{int(missing)} pages are lacking")
        q = self._project(torch.cat(x), slots, i32([t for m in n for t in range(m)]))
        starts = i32([0] + counts).cumsum(0).to(torch.int32)
        o = fc2.mxfp4_cache_attention(q, self.cache, self.pages.table, self.pages.lens, starts, max(n))
        rows = torch.arange(len(counts), device=dev) // self.samples
        fc2.mxfp4_pages_select(self.pages, (rows * self.samples).to(torch.int32))
        self.shared.copy_(i32(n))
        last = i32(n).cumsum(0) - 1
        return fc2.mxfp4_linear(o.flatten(1)[last], self.w_out)[rows]

    def step(self, x, counts):
        """One token of every row: x [rows, hidden]."""
        slots, copies, _ = fc2.mxfp4_pages_extend(self.pages, counts, len(x))  # the graph's user checks the pool's size
        fc2.mxfp4_cache_copy(self.cache, copies)
        q = self._project(x, slots, self.pages.lens - 1)
        o = fc2.mxfp4_cache_attention_shared(q, self.cache, self.pages.table, self.pages.lens, self.groups, self.shared,
                                             max_group=self.samples)
        return fc2.mxfp4_linear(o.flatten(1), self.w_out)


class Sampler:
    """The step, captured once and replayed; `x` holds the newest outputs."""

    def __init__(self, layer: SampledLayer, x: torch.Tensor):
        self.layer, self.x = layer, x.clone()
        self.counts = torch.ones(len(x), dtype=torch.int32, device=x.device)  # the graph reads it: kept
        state = [layer.pages.refs, layer.pages.table, layer.pages.lens]
        kept = [t.clone() for t in state]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.x.copy_(layer.step(self.x, self.counts))  # loads modules before the capture; then everything as it was
            for t, old in zip(state + [self.x], kept + [x]):
                t.copy_(old)
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.x.copy_(layer.step(self.x, self.counts))

    def step(self) -> torch.Tensor:
        self.graph.replay()
        return self.x


def make_layer(hidden, q_heads, kv_heads, dim, prompts, samples, page, steps, g) -> SampledLayer:
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    per_row = -(-(max(prompts) + steps) // page)
    pool = sum(-(-n // page) for n in prompts) + len(prompts) * samples * (-(-steps // page) + 1)
    rotary = fc2.head_rotary(10000.0 ** (-torch.arange(dim // 2, dtype=torch.float64) / (dim // 2)))
    return SampledLayer(rand((q_heads + 2 * kv_heads) * dim, hidden) * hidden ** -0.5,
                        rand(hidden, q_heads * dim) * (q_heads * dim) ** -0.5,
                        1 + 0.1 * rand(dim), 1 + 0.1 * rand(dim), q_heads, kv_heads, dim, rotary,
                        fc2.empty_mxfp4_pages(pool, page, len(prompts) * samples, per_row), samples)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--prompts", type=int, nargs="+", default=[3000, 9000])
    p.add_argument("--samples", type=int, default=16)
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--hidden", type=int, default=5376)
    p.add_argument("--heads", type=int, nargs=3, default=[32, 8, 128], metavar=("Q", "KV", "DIM"))
    p.add_argument("--page", type=int, default=64)
    a = p.parse_args()
    hq, hkv, dim = a.heads
    g = torch.Generator(device="cuda").manual_seed(0)
    layer = make_layer(a.hidden, hq, hkv, dim, a.prompts, a.samples, a.page, a.steps, g)
    x = [torch.randn(n, a.hidden, generator=g, device="cuda").to(torch.bfloat16) for n in a.prompts]
    sampler = Sampler(layer, layer.take_in(x))
    t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    t[0].record()
    for _ in range(a.steps):
        y = sampler.step()
    t[1].record()
    torch.cuda.synchronize()
    assert bool(torch.isfinite(y).all())
    held, lone = int((layer.pages.refs > 0).sum()), int(((layer.pages.lens + a.page - 1) // a.page).sum())
    print(f"{t[0].elapsed_time(t[1]) / a.steps * 1000:.1f} us a step of {len(y)} samples; "
          f"{held} pages held, {lone} without sharing")


if __name__ == "__main__":
    main()
