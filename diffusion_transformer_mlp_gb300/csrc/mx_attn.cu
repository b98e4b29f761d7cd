// Entry points of the attention over the MXFP4 cache: argument checks, the
// workspace, and the choice between the kernels.
#include <cmath>
#include <string>

#include "mx_attn.cuh"

namespace nvfp4 {

nvfp4_status check_cache(const mxfp4_cache* cache, int* page_shift, const std::string& nm);
int64_t attn_stream_workspace(int32_t dim);
int64_t attn_chunk_workspace(int32_t dim);
nvfp4_status attn_chunk(const mxfp4_cache* cache, const AttnParams& base, int32_t b, int32_t max_queries,
                        void* workspace, cudaStream_t stream, Pending& w);
nvfp4_status attn_stream(const mxfp4_cache* cache, const AttnParams& base, int32_t b, int32_t max_queries,
                         void* workspace, cudaStream_t stream, Pending& w);

namespace {
// Which kernel takes the rows (queries x heads of the group) of a sequence's kv
// head: k_attn_chunk works on 256 of them (dim 256: 128) at once, k_attn_stream
// on 8 or 16, each time decoding the keys anew.  32 sequences of 8,000 keys, 8
// kv heads, one query, stream / chunk in us:
//   rows         8         16         48         64        128
//   dim  64   51 / 283   62 / 283  155 / 268  200 / 265  385 / 250
//   dim 128   83 / 333   96 / 333  247 / 321  319 / 315  619 / 315
//   dim 256  184 / 338  345 / 339  931 / 396 1193 / 393 2371 / 317
// One sequence of 16,000 keys, dim 128: 16 rows 25 / 44, 64 rows 35 / 45, 128 rows
// 53 / 44.  At 16 rows of dim 256 the two differ by 5% at most from 2,000 keys on
// (16 sequences of 4,000: 117 / 115; 4 queries of 4 heads: 121 / 116), and short
// sequences are the stream kernel's (8 of 500 keys: 27 / 35; 64 of 300: 71 / 91).
bool many_rows(int32_t dim, int64_t rows) { return rows > (dim == 256 ? 16 : 64); }
}  // namespace

bool attn_has_many_rows(int32_t dim, int64_t rows) { return many_rows(dim, rows); }
int64_t attn_workspace(int32_t dim, bool many) {
  return many ? attn_chunk_workspace(dim) : attn_stream_workspace(dim);
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" int64_t mxfp4_attention_workspace_bytes(int32_t kv_heads, int32_t q_heads, int32_t dim,
                                                   int32_t max_queries) {
  if (kv_heads < 1 || q_heads < 1 || max_queries < 1 || (dim != 64 && dim != 128 && dim != 256)) return 0;
  const int64_t rows = int64_t(max_queries) * (q_heads / kv_heads);
  return attn_workspace(dim, many_rows(dim, rows));
}

namespace nvfp4 {

nvfp4_status attn_params(const mxfp4_cache* cache, const mxfp4_attention* args, int64_t workspace_bytes,
                         const std::string& nm, AttnParams& p) {
  int sh = 0;
  const nvfp4_status st = check_cache(cache, &sh, nm);
  if (st != NVFP4_OK) return st;
  if (!args) return fail(NVFP4_EINVAL, nm + ": null pointer");
  const mxfp4_attention& g = *args;
  if (g.dtype != MXFP4_BF16 && g.dtype != MXFP4_FP16) return fail(NVFP4_EINVAL, nm + ": q must be BF16 or FP16");
  if (g.seqs < 0 || g.total_q < 0 || g.max_queries < 0 || g.window < 0 || g.sinks < 0)
    return fail(NVFP4_EINVAL, nm + ": negative size");
  if (g.q_heads < 1 || g.q_heads % cache->kv_heads != 0)
    return fail(NVFP4_EINVAL, nm + ": q_heads must be a positive multiple of kv_heads");
  if (!std::isfinite(g.scale)) return fail(NVFP4_EINVAL, nm + ": scale must be finite");
  p = {};
  if (g.seqs == 0 || g.total_q == 0 || g.max_queries == 0) return NVFP4_OK;
  if (!g.q || !g.out || !g.table || !g.lens || !g.workspace) return fail(NVFP4_EINVAL, nm + ": null pointer");
  if (g.table_ld < 1) return fail(NVFP4_EINVAL, nm + ": a block table row needs an entry");
  if (g.q_starts == nullptr && (g.max_queries != 1 || g.total_q != g.seqs))
    return fail(NVFP4_EINVAL, nm + ": without q_starts every sequence has one query");
  const int64_t group = g.q_heads / cache->kv_heads;
  if (int64_t(g.max_queries) * group > (int64_t(1) << 24) || g.table_ld > (int64_t(1) << 31) / cache->page_size)
    return fail(NVFP4_EUNSUPPORTED, nm + ": problem too large");
  if (!aligned16(g.workspace) || reinterpret_cast<uintptr_t>(g.q) % 2 != 0 ||
      reinterpret_cast<uintptr_t>(g.out) % 2 != 0 || reinterpret_cast<uintptr_t>(g.table) % 4 != 0 ||
      reinterpret_cast<uintptr_t>(g.lens) % 4 != 0 || reinterpret_cast<uintptr_t>(g.q_starts) % 4 != 0 ||
      reinterpret_cast<uintptr_t>(g.lse) % 4 != 0)
    return fail(NVFP4_EALIGN, nm + ": workspace must be 16-byte aligned, the others aligned to their elements");
  if (g.workspace_bytes < workspace_bytes)
    return fail(NVFP4_EINVAL, nm + ": workspace too small, " + std::to_string(workspace_bytes) + " bytes are needed");
  p.q = g.q, p.out = g.out, p.lse = g.lse;
  p.table = g.table, p.lens = g.lens, p.q_starts = g.q_starts;
  p.q_ends = g.q_starts != nullptr ? g.q_starts + 1 : nullptr;
  p.k_codes = static_cast<const uint8_t*>(cache->k_codes);
  p.v_codes = static_cast<const uint8_t*>(cache->v_codes);
  p.k_scales = static_cast<const uint8_t*>(cache->k_scales);
  p.v_scales = static_cast<const uint8_t*>(cache->v_scales);
  p.dev_status = g.dev_status;
  p.q_st = g.q_st, p.q_sh = g.q_sh, p.o_st = g.o_st, p.o_sh = g.o_sh, p.table_ld = g.table_ld;
  p.pages = cache->pages;
  p.page_shift = sh, p.kv_heads = cache->kv_heads, p.group = int32_t(group), p.seqs = g.seqs, p.total_q = g.total_q;
  p.q_rows = g.total_q;
  p.bf16 = g.dtype == MXFP4_BF16, p.causal = g.causal != 0, p.window = g.window, p.sinks = g.sinks;
  // A window that reaches from a query (at -2^24 or later) past every key hides
  // none; smaller ones leave the kernels' differences of positions in 32 bits.
  const int64_t keys = g.table_ld * cache->page_size, most = (int64_t(1) << 31) - (int64_t(1) << 25);
  if (g.window >= (keys < most ? keys : most)) p.window = p.sinks = 0;
  p.q_vec = aligned16(g.q) && g.q_st % 8 == 0 && g.q_sh % 8 == 0;
  p.o_vec = aligned16(g.out) && g.o_st % 8 == 0 && g.o_sh % 8 == 0;
  p.scale_log2 = g.scale * 1.4426950408889634f;
  p.wait_limit_cycles = kAttnWaitLimitCycles;
  return NVFP4_OK;
}

nvfp4_status attn_begin(const mxfp4_cache* cache, const AttnParams& p, int32_t b, int32_t max_queries, bool many,
                        void* workspace, cudaStream_t stream, Pending& w) {
  w = {};
  return many ? attn_chunk(cache, p, b, max_queries, workspace, stream, w)
              : attn_stream(cache, p, b, max_queries, workspace, stream, w);
}

nvfp4_status attn_run(const mxfp4_cache* cache, const AttnParams& p, int32_t max_queries, bool many, void* workspace,
                      cudaStream_t stream) {
  // kMaxSeqs sequences a launch; the workspace is reused in stream order
  for (int32_t b = 0; b < p.seqs; b += kMaxSeqs) {
    Pending w;
    nvfp4_status st = attn_begin(cache, p, b, max_queries, many, workspace, stream, w);
    if (st == NVFP4_OK) st = attn_finish(cache->dim, w, stream);
    if (st != NVFP4_OK) return st;
  }
  return NVFP4_OK;
}

}  // namespace nvfp4

extern "C" nvfp4_status mxfp4_cache_attention(const mxfp4_cache* cache, const mxfp4_attention* args,
                                              nvfp4_stream_t stream) {
  AttnParams p;
  const int64_t need = cache && args ? mxfp4_attention_workspace_bytes(cache->kv_heads, args->q_heads, cache->dim,
                                                                       args->max_queries)
                                     : 0;
  const nvfp4_status st = attn_params(cache, args, need, "mxfp4_cache_attention", p);
  if (st != NVFP4_OK || p.seqs == 0) return st;
  return attn_run(cache, p, args->max_queries, many_rows(cache->dim, int64_t(args->max_queries) * p.group),
                  args->workspace, reinterpret_cast<cudaStream_t>(stream));
}
