// What the attention kernels over the MXFP4 cache share: parameters, the
// masks' geometry, small PTX helpers.
#pragma once

#include "mx_common.cuh"

namespace nvfp4 {

constexpr int kMaxSeqs = 1024;        // sequences of one launch (their tile counts sit in shared memory)
constexpr float kWeightLog2 = 10.0f;  // weights are held times 2^10
constexpr uint64_t kAttnWaitLimitCycles = 4000000000ull;  // about two seconds

struct AttnParams {
  const void* q;
  void* out;
  float* lse;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* q_starts;  // null: one query a sequence
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  uint32_t* dev_status;
  int64_t q_st, q_sh, o_st, o_sh, table_ld;
  int64_t pages;
  int32_t page_shift, kv_heads, group, seqs, total_q;
  int32_t bf16, causal, window, sinks;
  int32_t q_vec, o_vec;  // 16-byte accesses to q / out are aligned
  float scale_log2;      // softmax scale times log2(e)
  uint64_t wait_limit_cycles;
};

// The keys that rows [i0, i1] (queries of one sequence) may see, in tiles of
// `tok` keys: tiles [0, sink_tiles) and [lo_tile, hi_tile).  The tiles at their
// ends also hold keys that none of the rows sees, whose bytes may be anything
// (pages that left the window are used again): those enter nothing.
struct Span {
  int32_t lo, hi;      // seen by some row: keys of [lo, hi) and, with a window, those below p.sinks and hi
  int32_t lo_tile, sink_tiles, n;
  __device__ __forceinline__ int32_t tile(int32_t s) const { return s < sink_tiles ? s : s - sink_tiles + lo_tile; }
  __device__ __forceinline__ bool has(const AttnParams& p, int32_t j) const {
    return j < hi && (j >= lo || j < p.sinks);  // lo is 0 without a window
  }
};

__device__ __forceinline__ Span span_of(const AttnParams& p, int32_t len, int32_t nq, int32_t i0, int32_t i1,
                                        int32_t tok) {
  Span s;
  const int32_t base = len - nq;  // position of query 0 (negative if there are more queries than keys)
  int32_t hi = p.causal ? min(len, base + i1 + 1) : len;
  hi = max(hi, 0);
  int32_t lo = p.window > 0 ? base + i0 + 1 - p.window : 0;
  lo = min(max(lo, 0), hi);
  const int32_t hi_tile = (hi + tok - 1) / tok;
  s.lo = lo, s.hi = hi;
  s.lo_tile = lo / tok;
  s.sink_tiles = p.window > 0 ? min((min(p.sinks, hi) + tok - 1) / tok, s.lo_tile) : 0;
  s.n = s.sink_tiles + hi_tile - s.lo_tile;
  return s;
}

// Whether the query at position pos sees key j (j < len is the caller's).
__device__ __forceinline__ bool sees(const AttnParams& p, int32_t pos, int32_t j) {
  return (!p.causal || j <= pos) && (p.window <= 0 || j > pos - p.window || j < p.sinks);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 2^e for a whole e (0 below the normal range).
__device__ __forceinline__ float pow2i(int32_t e) {
  return e < -126 ? 0.0f : __uint_as_float(uint32_t(min(e, 127) + 127) << 23);
}

__device__ __forceinline__ void tma_load_3d_plain(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t x,
                                                  int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// A launch whose work is dealt in equal runs of tiles over its workers (warps of
// k_attn_stream, blocks of k_attn_chunk), whatever the sequences' lengths: the
// tiles of all (sequence, row tile, kv head) segments in a row, worker w taking
// [total w / W, total (w+1) / W).  A segment may weigh `edge` tiles more than it
// has: places of the list before its first tile.  A worker writes the output of a segment that
// it has all of; of others a partial goes to the workspace, at most two a
// worker: its first segment's to slot 0, a later one's to slot 1.
struct SplitParams {
  AttnParams a;
  int32_t workers;
  int32_t least, even;  // tiles of a run: at least, if there are that many; see live_workers
  int32_t edge;
  float* part_o;     // [2 * workers][rows][D] (k_attn_chunk: [D / 4][rows][4]); see part_exponent
  float2* part_ml;   // [2 * workers][rows]  (reference, sum)
  int64_t* prefix;   // [seqs + 1] places before each sequence, written by block 0 for k_attn_combine
  struct Cursor* start;  // [workers] first tiles of the runs, written by k_attn_chunk for k_attn_join
};

__device__ __forceinline__ int32_t seq_queries(const AttnParams& a, int32_t b) {
  return a.q_starts != nullptr ? a.q_starts[b + 1] - a.q_starts[b] : 1;
}

// Span of row tile rt (rows [rt * rows, ...) of the nq * group rows).
__device__ __forceinline__ Span row_span(const AttnParams& a, int32_t len, int32_t nq, int32_t rt, int32_t rows,
                                         int32_t tok) {
  const int32_t last = min((rt + 1) * rows, nq * a.group) - 1;
  return span_of(a, len, nq, rt * rows / a.group, last / a.group, tok);
}

// Workers that get tiles, all of them one or more, so that all workers of a
// segment's range have a partial of it.  Of runs of up to `even` tiles all get
// the longest: a worker less is partials less to join.
__device__ __forceinline__ int32_t live_workers(const SplitParams& sp, int64_t total) {
  const int64_t run = max(int64_t(sp.least), (total + sp.workers - 1) / sp.workers);
  if (run <= sp.even) return int32_t((total + run - 1) / run);
  return int32_t(min(int64_t(sp.workers), (total + sp.least - 1) / sp.least));
}
__device__ __forceinline__ int64_t worker_start(int64_t total, int32_t w, int32_t workers) {
  return total * w / workers;
}
// The worker whose run holds tile x: the largest w with worker_start(w) <= x.
__device__ __forceinline__ int32_t worker_of(int64_t total, int64_t x, int32_t workers) {
  return int32_t(((x + 1) * workers - 1) / total);
}

// A tile of the list.
struct Cursor {
  int32_t b, rt, h, t;  // t: tile of the segment
  int32_t len, nq, q0;
  Span s;
};

__device__ __forceinline__ void cursor_seq(Cursor& c, const AttnParams& a) {
  c.len = a.lens[c.b];
  c.nq = seq_queries(a, c.b);
  c.q0 = a.q_starts != nullptr ? a.q_starts[c.b] : c.b;
}

// The first tile at place x or behind it, by a whole warp: 32 row tiles at a
// time.  Returns how far behind.
__device__ __forceinline__ int32_t cursor_at(Cursor& c, const AttnParams& a, const int64_t* prefix, int64_t x,
                                             int32_t rows, int32_t tok, int32_t edge) {
  const int lane = threadIdx.x & 31;
  int32_t lo = 0, hi = a.seqs;  // prefix[lo] <= x < prefix[hi]
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (prefix[mid] <= x) lo = mid;
    else hi = mid;
  }
  c.b = lo;
  cursor_seq(c, a);
  int64_t rem = x - prefix[lo];
  for (int32_t rt = 0;; rt += 32) {
    int64_t n = (rt + lane) * rows < c.nq * a.group ? row_span(a, c.len, c.nq, rt + lane, rows, tok).n : 0;
    n = n > 0 ? (n + edge) * a.kv_heads : 0;
    int64_t upto = n;  // of this row tile and those before it
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += u;
    }
    const uint32_t there = __ballot_sync(0xFFFFFFFFu, rem < upto);
    if (there != 0) {
      const int at = __ffs(there) - 1;
      c.rt = rt + at;
      rem -= __shfl_sync(0xFFFFFFFFu, upto - n, at);
      break;
    }
    rem -= __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  c.s = row_span(a, c.len, c.nq, c.rt, rows, tok);
  c.h = int32_t(rem / (c.s.n + edge));
  const int32_t off = int32_t(rem - int64_t(c.h) * (c.s.n + edge));
  c.t = max(off - edge, 0);
  return max(edge - off, 0);
}

// The next tile; the caller knows that there is one.
__device__ __forceinline__ void cursor_next(Cursor& c, const AttnParams& a, int32_t rows, int32_t tok) {
  if (++c.t < c.s.n) return;
  c.t = 0;
  if (++c.h < a.kv_heads) return;
  c.h = 0;
  do {
    if ((c.rt + 1) * rows < c.nq * a.group) {
      ++c.rt;
    } else {
      c.rt = 0;
      do {
        ++c.b;
        cursor_seq(c, a);
      } while (c.nq <= 0);
    }
    c.s = row_span(a, c.len, c.nq, c.rt, rows, tok);
  } while (c.s.n == 0);
}

// Places before each sequence, in prefix[0 .. seqs] (kMaxSeqs + 1 + kThreads
// entries of shared memory); block 0 leaves them for k_attn_combine.  With few
// sequences up to 32 threads share the row tiles of one.  Then every thread sums
// a run of sequences and the first warp scans the runs' sums.
template <int kThreads>
__device__ __forceinline__ void tile_counts(const SplitParams& sp, int64_t* prefix, int32_t rows, int32_t tok) {
  constexpr int kEach = (kThreads + 31) / 32;
  const AttnParams& a = sp.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t* run = prefix + kMaxSeqs + 1;
  int share = 1;
  while (share < 32 && a.seqs * share * 2 <= kThreads) share *= 2;
  for (int first = 0; first < a.seqs; first += kThreads / share) {
    const int b = first + int(threadIdx.x) / share;
    int64_t n = 0;
    if (b < a.seqs) {
      const int32_t len = a.lens[b], nq = seq_queries(a, b);
      for (int32_t rt = int(threadIdx.x) % share; rt * rows < nq * a.group; rt += share)
        if (const int32_t t = row_span(a, len, nq, rt, rows, tok).n; t > 0) n += t + sp.edge;
    }
    for (int o = 1; o < share; o <<= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
    if (b < a.seqs && threadIdx.x % share == 0) prefix[b] = n * a.kv_heads;
  }
  __syncthreads();
  const int per = (a.seqs + kThreads - 1) / kThreads;
  const int b0 = min(int(threadIdx.x) * per, a.seqs), b1 = min(b0 + per, a.seqs);
  int64_t sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int64_t n = prefix[b];
    prefix[b] = sum;
    sum += n;
  }
  run[threadIdx.x] = sum;
  __syncthreads();
  if (warp == 0) {
    int64_t v[kEach], s = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      v[i] = s;
      if (lane * kEach + i < kThreads) s += run[lane * kEach + i];
    }
    int64_t inc = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += u;
    }
    const int64_t before = inc - s;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (lane * kEach + i < kThreads) run[lane * kEach + i] = before + v[i];
    if (lane == 31) prefix[a.seqs] = inc;
  }
  __syncthreads();
  for (int b = b0; b < b1; ++b) prefix[b] += run[threadIdx.x];
  __syncthreads();
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= a.seqs; b += kThreads) sp.prefix[b] = prefix[b];
}

// A partial is (reference + e, sum 2^-e, output 2^-e) with 2^e <= sum < 2^(e + 1):
// an exact change, after which the output is no larger than twice the largest
// value, however many keys it sums.  Where partials are joined, references stand
// kJoinLog2 above the maximum, for as many partials.
constexpr float kJoinLog2 = 12.0f;
__device__ __forceinline__ int32_t part_exponent(float sum) {
  const int32_t e = int32_t(__float_as_uint(sum) >> 23) & 0xFF;
  return e == 0 || e == 255 ? 0 : e - 127;
}

// Eight consecutive 16-bit outputs of a row.
__device__ __forceinline__ void store_o8_words(const AttnParams& a, uint16_t* dst, uint4 w) {
  if (a.o_vec) {
    *reinterpret_cast<uint4*>(dst) = w;
  } else {
    dst[0] = uint16_t(w.x), dst[1] = uint16_t(w.x >> 16), dst[2] = uint16_t(w.y), dst[3] = uint16_t(w.y >> 16);
    dst[4] = uint16_t(w.z), dst[5] = uint16_t(w.z >> 16), dst[6] = uint16_t(w.w), dst[7] = uint16_t(w.w >> 16);
  }
}
__device__ __forceinline__ void store_o8(const AttnParams& a, uint16_t* dst, const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = a.bf16 ? f32_to_word<__nv_bfloat16>(f[2 * i], f[2 * i + 1]) : f32_to_word<__half>(f[2 * i], f[2 * i + 1]);
  store_o8_words(a, dst, make_uint4(w[0], w[1], w[2], w[3]));
}

// The queries and outputs of the sequences from b on.
inline void split_queries(AttnParams& a, const AttnParams& base, int32_t b) {
  if (base.q_starts != nullptr) {
    a.q_starts = base.q_starts + b;
    return;
  }
  a.q = static_cast<const uint16_t*>(base.q) + int64_t(b) * base.q_st;
  a.out = static_cast<uint16_t*>(base.out) + int64_t(b) * base.o_st;
  if (base.lse != nullptr) a.lse = base.lse + int64_t(b) * base.kv_heads * base.group;
}

// mx_attn_combine.cu: the partials of k_attn_stream (rows: 8 or 16), of k_attn_chunk.
nvfp4_status attn_combine(int dim, int rows, int tok, int row_tiles, const SplitParams& sp, cudaStream_t stream);
nvfp4_status attn_join(int dim, int tok, const SplitParams& sp, cudaStream_t stream);

}  // namespace nvfp4
