// Attention of sequences that share a prefix, over the paged MXFP4 cache.
//
// softmax over the keys [prefix | own] joins from the softmaxes over both parts:
//
//   out = (e^(l1 - m) o1 + e^(l2 - m) o2) / (e^(l1 - m) + e^(l2 - m)),  m = max(l1, l2)
//
// with l the logarithm of a part's sum of exponentials.  The prefix is one
// sequence whose queries are those of all sequences of the group, every one of
// which sees all of it: its keys are read and decoded once for many rows, which is
// work for k_attn_chunk where they are more than k_attn_stream is made for (64, dim
// 256: 16) or where it is estimated to be quicker (plan_of).  What a sequence has of
// its own is a sequence whose block table begins behind the prefix; positions
// only count relative to its end, so nothing else changes.  That takes whole
// pages, hence the prefix is rounded down to them.
//
// k_shared_parts writes the two sets of lengths and tables, attention runs for
// each with binary32 outputs, and k_shared_join joins them.  Where both parts are
// k_attn_stream's and every sequence has one query, which sees all keys of either
// part, both sets are one list of sequences for one launch: rows total_q and
// above of the outputs are the own tokens' (4 samples of a prompt of 2,049
// tokens: 32 us in two launches, so 20).  Queries outside of the groups are rows
// between those of the prefixes and the own ones, and of no sequence.
//
// What bounds it: the latencies of five launches and of k_attn_chunk's first and last
// tiles, before the work itself.  Two prompts of 16,001 and 12,001 tokens, 32 and 16
// sequences, 32 / 8 heads of 128: parts 3.7, prefixes 33, own tokens 11.1, the joins of
// both 10.1 (in two launches 7.0 + 6.1), this join 2.8 us; the pass 58 us, 185 if each
// sequence reads its prompt.  One of 32,769 tokens, 128 sequences of 64 heads: 162 us
// instead of 1,009; 116 of them are k_attn_chunk at 61% of the tensor rate.  Where
// reading prefixes each time is as fast, that is done (plan_of).
#include <algorithm>
#include <string>

#include "mx_attn.cuh"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;

struct SharedParams {
  AttnParams a;  // of the call
  const int32_t* groups;
  const int32_t* shared;
  int32_t count;
  // The groups' prefixes and the sequences' own tokens: count + seqs sequences.
  int32_t *table, *lens, *starts, *ends;
  int32_t* before;  // [seqs] tokens of the prefix
  float *o, *l;     // [2 * total_q] rows: of the prefixes, of the own tokens
};

__device__ __forceinline__ int32_t group_start(const SharedParams& p, int32_t g) {
  return min(max(p.groups[g], 0), p.a.seqs);
}

// Tokens that the sequences of group g share, by a whole block.
__device__ int32_t prefix_of(const SharedParams& p, int32_t g, int32_t* red) {
  const AttnParams& a = p.a;
  const int32_t s0 = group_start(p, g), s1 = group_start(p, g + 1);
  int32_t n = s0 < s1 ? min(p.shared[g], a.lens[s0]) : 0;  // the first one's table names it
  for (int32_t b = s0 + int32_t(threadIdx.x); b < s1; b += kThreads) {
    const int32_t nq = seq_queries(a, b);
    if (nq > 0) n = min(n, a.causal ? a.lens[b] - nq : a.lens[b]);
  }
  n = __reduce_min_sync(0xFFFFFFFFu, n);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = n;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) n = min(n, red[i]);
  const int64_t room = a.table_ld << a.page_shift;
  return int32_t(min(int64_t(max(n, 0)), room)) & ~((1 << a.page_shift) - 1);
}

// A block for each group, then one for each sequence.
__global__ void __launch_bounds__(kThreads) k_shared_parts(const __grid_constant__ SharedParams p) {
  __shared__ int32_t red[kThreads / 32];
  const AttnParams& a = p.a;
  grid_wait();
  if (int32_t(blockIdx.x) < p.count) {
    const int32_t g = blockIdx.x, s0 = group_start(p, g), n = prefix_of(p, g, red);
    if (threadIdx.x == 0) {
      const int32_t s1 = group_start(p, g + 1);
      p.lens[g] = n;
      p.starts[g] = s0 < s1 ? seq_start(a, s0) : 0;
      p.ends[g] = s0 < s1 ? seq_start(a, s1 - 1) + seq_queries(a, s1 - 1) : 0;
    }
    const int32_t* src = a.table + s0 * a.table_ld;
    for (int32_t i = threadIdx.x; i < n >> a.page_shift; i += kThreads) p.table[g * a.table_ld + i] = src[i];
    return;
  }
  const int32_t b = int32_t(blockIdx.x) - p.count;
  int32_t n = 0;
  if (b >= group_start(p, 0) && b < group_start(p, p.count)) {
    int32_t lo = 0, hi = p.count;  // groups[lo] <= b < groups[hi]
    while (hi - lo > 1) {
      const int32_t mid = (lo + hi) >> 1;
      if (group_start(p, mid) <= b) lo = mid;
      else hi = mid;
    }
    n = prefix_of(p, lo, red);
    n = min(n, max(a.lens[b], 0) & ~((1 << a.page_shift) - 1));  // without queries it limits nothing
  }
  const int32_t len = a.lens[b] - n;
  const int32_t own = p.count + b;
  if (threadIdx.x == 0) {
    p.before[b] = n, p.lens[own] = len;
    p.starts[own] = a.total_q + seq_start(a, b);
    p.ends[own] = a.total_q + seq_start(a, b) + seq_queries(a, b);
  }
  const int64_t skip = n >> a.page_shift, most = a.table_ld - skip;
  const int64_t pages = min((int64_t(max(len, 0)) + (int64_t(1) << a.page_shift) - 1) >> a.page_shift, most);
  for (int64_t i = threadIdx.x; i < pages; i += kThreads) p.table[own * a.table_ld + i] = a.table[b * a.table_ld + skip + i];
}

// Eight columns of a row and head a thread; the rows of sequence blockIdx.x.
template <int D>
__global__ void __launch_bounds__(kThreads) k_shared_join(const __grid_constant__ SharedParams p) {
  const AttnParams& a = p.a;
  grid_wait();
  const int32_t b = blockIdx.x, heads = a.kv_heads * a.group;
  const int64_t q0 = seq_start(a, b), items = int64_t(seq_queries(a, b)) * heads * (D / 8);
  const bool prefix = p.before[b] > 0;
  for (int64_t i = int64_t(blockIdx.y) * kThreads + threadIdx.x; i < items; i += int64_t(gridDim.y) * kThreads) {
    const int64_t rh = q0 * heads + i / (D / 8);  // (row, head)
    const int32_t d = int32_t(i % (D / 8)) * 8;
    const int64_t own = int64_t(a.total_q) * heads + rh;
    const float l2 = p.l[own], l1 = prefix ? p.l[rh] : -INFINITY;
    const float4* s2 = reinterpret_cast<const float4*>(p.o + own * D + d);
    float4 u = s2[0], v = s2[1];
    float f[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
    float lse = l2;
    if (prefix) {
      const float4* s1 = reinterpret_cast<const float4*>(p.o + rh * D + d);
      u = s1[0], v = s1[1];
      const float g[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
      const float m = fmaxf(l1, l2), ref = m == -INFINITY ? 0.0f : m;
      const float e1 = expf(l1 - ref), e2 = expf(l2 - ref), sum = e1 + e2;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      const float w1 = e1 * inv, w2 = e2 * inv;  // no more than 1 together: values near the end of the range stay in it
#pragma unroll
      for (int x = 0; x < 8; ++x) f[x] = w1 * g[x] + w2 * f[x];
      lse = m == -INFINITY ? m : ref + logf(sum);
    }
    const int64_t row = rh / heads, h = rh - row * heads;
    store_o8(a, row * a.o_st + h * a.o_sh + d, f);
    if (d == 0 && a.lse != nullptr) a.lse[rh] = lse;
  }
}

// How to work: every sequence for itself, or prefixes (by either kernel) and own
// tokens, in one launch or two.
struct Plan {
  bool share, one_list, prefix_many, own_many;
};

// The host knows the sizes of the tables, not the lengths: times in us as if all
// tables were full and all of them shared, which is the most that sharing can save.
// Rates are key heads (keys times kv heads) a us and row tile (of 8 or 16 rows, of 256
// or 128), measured with 2 to 32 sequences of 1 and 6 queries on prefixes of 512 to
// 32,768 keys, 4 and 8 kv heads, groups of 4 and 8.  Each for itself / shared:
//   dim 128, 4 sequences, 1 query      11.8 / 19.9   14.1 / 20.5   22.6 / 26.0   45.0 / 36.1
//   16 sequences                       13.8 / 20.9   22.5 / 23.9   44.7 / 34.9  137.4 / 55.9
//   32 sequences                       17.8 / 33.2   30.5 / 33.0   76.5 / 38.4  260.0 / 56.1
//   8 sequences, 6 queries             18.1 / 36.6   28.2 / 35.9   54.5 / 43.9  170.4 / 66.4
//   dim 64, 32 sequences, 1 query      11.9 / 28.3   18.0 / 28.9   29.7 / 36.5   82.5 / 47.7
//   dim 256, 8 sequences, 1 query      14.4 / 40.2   19.4 / 39.5   34.0 / 47.6   89.7 / 62.6
// (prefixes of 512, 2,048, 8,192, 32,768 keys).  Where a sequence has rows for whole
// tiles there is nothing to save: the work is the rows', and they are as many.
//
// Sequences outside of the groups are read either way, and at most count * max_group
// queries lie in one.  In one list they go through the rows' kernel of the groups, which
// takes twice as long for them if it is that of 16 rows: 512 sequences of up to 1,000
// keys, 8 of them behind 16,000 common ones, 146 us for itself and 189 in one list.
Plan plan_of(int32_t dim, int64_t kv_heads, int64_t group, int64_t total_q, int64_t max_queries, int64_t seqs,
             int64_t capacity, int64_t count, int64_t max_group) {
  const int i = dim == 64 ? 0 : (dim == 128 ? 1 : 2);
  const double few8[3] = {58e3, 33e3, 14e3}, few16[3] = {40e3, 24e3, 9e3}, many[3] = {10e3, 10e3, 6e3};
  // in one list the own tokens' short segments come last, to workers of their own
  const double list8[3] = {16e3, 15e3, 9e3}, list16[3] = {20e3, 16e3, 4e3};
  auto stream = [&](int64_t n, int64_t rows, const double* rate8, const double* rate16) {  // n sequences' keys
    const double work = double(n) * double(capacity) * double(kv_heads);
    return rows <= 8 ? work / rate8[i] : work * double((rows + 15) / 16) / rate16[i];
  };
  auto chunk = [&](int64_t n, int64_t rows) {
    const int64_t tile = dim == 256 ? 128 : 256;
    return double(n) * double(capacity) * double(kv_heads) * double((rows + tile - 1) / tile) / many[i];
  };
  const int64_t own_rows = max_queries * group, most_rows = max_group * group;
  const int64_t grouped = std::min(total_q, count * max_group);
  const int64_t rows = (grouped + count - 1) / count * group;                   // of a group, about
  const int64_t readers = int64_t(double(seqs) * double(grouped) / double(total_q) + 0.5);  // of prefixes, about
  Plan p = {};
  p.own_many = attn_has_many_rows(dim, own_rows);
  auto own = [&](int64_t n) { return p.own_many ? chunk(n, own_rows) : stream(n, own_rows, few8, few16); };
  const double others = own(seqs - readers);
  const double apart = (p.own_many ? 25.0 : 12.0) + own(readers) + others;
  const bool one = max_queries == 1;
  const double others_listed = most_rows <= 8 ? others : stream(seqs - readers, 16, list8, list16);
  const double by_stream = one ? 18.0 + stream(count, rows, list8, list16) + others_listed
                               : 30.0 + stream(count, rows, few8, few16) + others;
  const double by_chunk = (dim == 256 ? 44.0 : 36.0) + chunk(count, rows) + others;
  p.prefix_many = attn_has_many_rows(dim, most_rows) || by_chunk < by_stream;
  p.one_list = one && !p.prefix_many;
  p.share = (p.prefix_many ? by_chunk : by_stream) < apart;
  return p;
}

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

// Places in the workspace, from its start on; returns its size.
int64_t layout(SharedParams& p, uint8_t* ws, int64_t attention, int64_t rows, int64_t heads, int32_t dim, int64_t seqs,
               int64_t table_ld) {
  int64_t at = align256(attention);
  auto take = [&](auto*& ptr, int64_t n) {
    ptr = reinterpret_cast<std::remove_reference_t<decltype(ptr)>>(ws + at);
    at += align256(n * 4);
  };
  take(p.o, 2 * rows * heads * dim);
  take(p.l, 2 * rows * heads);
  take(p.table, (p.count + seqs) * table_ld);
  take(p.lens, p.count + seqs);
  take(p.starts, p.count + seqs);
  take(p.ends, p.count + seqs);
  take(p.before, seqs);
  return at;
}
int64_t parts_workspace(int32_t dim) { return align256(attn_workspace(dim, true)) + attn_workspace(dim, false); }

// How the call works, and the bytes of workspace that this takes.
Plan plan_call(const mxfp4_cache* cache, const mxfp4_attention* args, const mxfp4_shared* shared, int64_t* bytes) {
  Plan plan = {};
  *bytes = 0;
  if (args->total_q < 1 || args->seqs < 1 || args->table_ld < 1 || args->max_queries < 1) return plan;
  *bytes = mxfp4_attention_workspace_bytes(cache->kv_heads, args->q_heads, cache->dim, args->max_queries);
  if (*bytes == 0) return plan;
  const int32_t dim = cache->dim, max_group = std::min(shared->max_group, args->total_q);
  const int64_t group = args->q_heads / cache->kv_heads;
  plan.own_many = attn_has_many_rows(dim, args->max_queries * group);
  if (shared->count < 1 || max_group < 1) return plan;
  plan = plan_of(dim, cache->kv_heads, group, args->total_q, args->max_queries, args->seqs,
                 args->table_ld * cache->page_size, shared->count, max_group);
  if (shared->always != 0) plan.share = true;
  SharedParams p;
  p.count = shared->count;
  if (plan.share)
    *bytes = layout(p, nullptr, parts_workspace(dim), args->total_q, args->q_heads, dim, args->seqs, args->table_ld);
  return plan;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" int64_t mxfp4_attention_shared_workspace_bytes(int32_t kv_heads, int32_t q_heads, int32_t dim,
                                                          int32_t total_q, int32_t max_queries, int32_t seqs,
                                                          int64_t table_ld, int32_t count, int32_t max_group) {
  if (total_q < 1 || seqs < 1 || table_ld < 1 || count < 0 || max_queries < 1) return 0;
  const int64_t own = mxfp4_attention_workspace_bytes(kv_heads, q_heads, dim, max_queries);
  if (own == 0 || count == 0 || max_group < 1) return own;
  SharedParams p;
  p.count = count;
  return layout(p, nullptr, parts_workspace(dim), total_q, q_heads, dim, seqs, table_ld);
}

extern "C" int64_t mxfp4_attention_shared_call_workspace_bytes(const mxfp4_cache* cache, const mxfp4_attention* args,
                                                               const mxfp4_shared* shared) {
  if (!cache || !args || !shared) return 0;
  int64_t bytes;
  plan_call(cache, args, shared, &bytes);
  return bytes;
}

extern "C" nvfp4_status mxfp4_cache_attention_shared(const mxfp4_cache* cache, const mxfp4_attention* args,
                                                     const mxfp4_shared* shared, nvfp4_stream_t stream) {
  const std::string nm("mxfp4_cache_attention_shared");
  if (!cache || !args || !shared) return fail(NVFP4_EINVAL, nm + ": null pointer");
  if (args->window != 0) return fail(NVFP4_EUNSUPPORTED, nm + ": a window would hide the prefix");
  if (shared->count < 0 || shared->max_group < 0) return fail(NVFP4_EINVAL, nm + ": negative size");
  const int32_t max_group = std::min(shared->max_group, args->total_q);
  int64_t need;
  const Plan plan = plan_call(cache, args, shared, &need);
  SharedParams p = {};
  const nvfp4_status bad = attn_params(cache, args, need, nm, p.a);
  if (bad != NVFP4_OK || p.a.seqs == 0) return bad;
  p.a.sinks = 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (shared->count > 0 && max_group > 0) {
    if (!shared->groups || !shared->shared) return fail(NVFP4_EINVAL, nm + ": null pointer");
    if (reinterpret_cast<uintptr_t>(shared->groups) % 4 != 0 || reinterpret_cast<uintptr_t>(shared->shared) % 4 != 0)
      return fail(NVFP4_EALIGN, nm + ": groups and shared must be aligned to their elements");
    if (int64_t(max_group) * p.a.group > (int64_t(1) << 24) || int64_t(shared->count) + args->seqs > 0x7FFFFF00 ||
        args->total_q > 0x3FFFFFFF)
      return fail(NVFP4_EUNSUPPORTED, nm + ": problem too large");
  }
  const int64_t heads = args->q_heads;
  const int32_t dim = cache->dim;
  if (!plan.share) return attn_run(cache, p.a, args->max_queries, plan.own_many, args->workspace, s);
  p.groups = shared->groups, p.shared = shared->shared, p.count = shared->count;
  layout(p, static_cast<uint8_t*>(args->workspace), parts_workspace(dim), args->total_q, heads, dim, args->seqs,
         args->table_ld);
  nvfp4_status st = launch("launch k_shared_parts", k_shared_parts, dim3(unsigned(p.count + args->seqs)), dim3(kThreads),
                           0, 0, s, p);
  if (st != NVFP4_OK) return st;
  AttnParams part = p.a;
  part.o_f32 = 1, part.o_vec = 1;
  part.o_st = heads * dim, part.o_sh = dim;
  part.out = p.o, part.lse = p.l;
  part.table = p.table, part.lens = p.lens, part.q_starts = p.starts, part.q_ends = p.ends;
  part.causal = 0;
  if (plan.one_list) {
    part.seqs = p.count + args->seqs, part.total_q = 2 * args->total_q;
    st = attn_run(cache, part, max_group, false, args->workspace, s);
    if (st != NVFP4_OK) return st;
  } else {
    // of k_attn_chunk and k_attn_stream the partials are joined at once, from workspaces of their own
    const bool both = plan.prefix_many && !plan.own_many && p.count <= kMaxSeqs && args->seqs <= kMaxSeqs;
    Pending prefix, own;
    part.seqs = p.count;
    st = both ? attn_begin(cache, part, 0, max_group, true, args->workspace, s, prefix)
              : attn_run(cache, part, max_group, plan.prefix_many, args->workspace, s);
    if (st != NVFP4_OK) return st;
    part.out = p.o + args->total_q * heads * dim, part.lse = p.l + args->total_q * heads;
    part.table = p.table + p.count * args->table_ld, part.lens = p.lens + p.count;
    part.q_starts = p.a.q_starts, part.q_ends = p.a.q_ends;
    part.seqs = args->seqs, part.causal = p.a.causal;
    if (both) {
      uint8_t* ws = static_cast<uint8_t*>(args->workspace) + align256(attn_workspace(dim, true));
      st = attn_begin(cache, part, 0, args->max_queries, false, ws, s, own);
      if (st == NVFP4_OK) st = attn_finish_both(dim, prefix, own, s);
    } else {
      st = attn_run(cache, part, args->max_queries, plan.own_many, args->workspace, s);
    }
    if (st != NVFP4_OK) return st;
  }
  const int64_t items = args->max_queries * heads * (dim / 8);
  const unsigned y = unsigned(std::min<int64_t>((items + kThreads - 1) / kThreads, 1024));
  auto join = dim == 64 ? k_shared_join<64> : (dim == 128 ? k_shared_join<128> : k_shared_join<256>);
  return launch("launch k_shared_join", join, dim3(unsigned(args->seqs), y), dim3(kThreads), 0, 0, s, p);
}
