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
  const uint8_t* k_codes;
  const uint8_t* v_codes;
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
  int32_t several;   // sequences may have several queries
  float* part_o;     // [2 * workers][rows][D] (k_attn_chunk: [D / 4][rows][4]); see part_exponent
  float2* part_ml;   // [2 * workers][rows]  (reference, sum)
  int64_t* prefix;   // [seqs + 1] places before each sequence, written by block 0 for k_attn_combine
  struct Cursor* start;  // [workers] first tiles of the runs, written by k_attn_chunk for k_attn_join
};

// First query row of sequence b, and the number of its queries: none outside of
// the rows that there are, whatever q_starts holds.
__device__ __forceinline__ int32_t seq_start(const AttnParams& a, int32_t b) {
  return a.q_starts != nullptr ? min(max(a.q_starts[b], 0), a.total_q) : b;
}
__device__ __forceinline__ int32_t seq_queries(const AttnParams& a, int32_t b) {
  return a.q_starts != nullptr ? max(min(a.q_starts[b + 1], a.total_q) - seq_start(a, b), 0) : 1;
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
  c.q0 = seq_start(a, c.b);
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

// Keys that only some rows see.  Both kernels put the values of all rows of a
// tile (k_attn_chunk the keys of a tile too) under one power of two, which comes
// from the keys that some row sees.  Where the largest is one that not all see,
// the others may lose bits to it: such segments (their parts that a worker has)
// are worked once more at the end of the worker's run, a row at a time in
// binary32 throughout (too_wide, wide_segment).  The kernels' loops only notice
// where that may be so (Spread).
//
// The keys that the rows of a row tile have in common, of those that one has:
// j < end with j >= from or j < sinks.
struct Common {
  int32_t end, from;
  bool one;  // all rows are of one query
};
__device__ __forceinline__ Common common_of(const AttnParams& a, int32_t len, int32_t nq, int32_t rt, int32_t rows) {
  const int32_t i0 = rt * rows / a.group, i1 = (min((rt + 1) * rows, nq * a.group) - 1) / a.group;
  Common c;
  c.one = i0 == i1;
  c.end = a.causal ? min(len, len - nq + i0 + 1) : len;
  c.from = a.window > 0 ? len - nq + i1 + 1 - a.window : 0;
  return c;
}
// Whether all rows see all keys of [j, j + n).
__device__ __forceinline__ bool all_see(const AttnParams& a, const Common& c, int32_t j, int32_t n) {
  return j + n <= c.end && (j >= c.from || j + n <= a.sinks);
}

// A lane's block column of a segment, at its tiles (or parts of them) that not all
// rows see.  Every row's largest scale code is at least `floor`, the largest of
// keys that all rows see (0: none so far), or else `least`, the smallest code but
// 0 of the keys that some see.
struct Spread {
  int32_t floor, least;
  __device__ __forceinline__ void reset() { floor = 0, least = 255; }
  __device__ __forceinline__ bool open() const { return floor == 0 && least < 255; }
  // Codes of up to `top`, the smallest but 0 being `low`; those before had up to
  // `old`.  False if some row's values may be more than `spread` below the others.
  __device__ __forceinline__ bool some_see(int32_t old, int32_t top, int32_t low, int32_t spread) {
    if (floor == 0 && least == 255) floor = old;  // all before were seen by all
    if (floor == 0) least = min(least, low);
    return max(old, top) <= (floor > 0 ? floor : least) + spread;
  }
  __device__ __forceinline__ bool all_see(int32_t old, int32_t top, int32_t spread) {
    if (!open() || top == 0) return true;
    floor = top;
    return old <= top + spread;
  }
};

// Row of key j of the segment at c in the cache.
__device__ __forceinline__ int64_t key_row(const AttnParams& a, const Cursor& c, int32_t j) {
  const int32_t page = a.table[int64_t(c.b) * a.table_ld + min(j >> a.page_shift, int32_t(a.table_ld) - 1)];
  const int32_t z = min(max(page, 0), int32_t(a.pages) - 1) * a.kv_heads + c.h;
  return (int64_t(z) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
}

// Whether n tiles from tile c.t on have to be worked once more, by a whole warp.
// Every row sees the keys that all see, or else at least one of the others; so
// no row's largest value is more than 2^spread_v below the reference if in each
// block column the largest scale code of the others is no more than that above
// the largest that all see or, where they see none, above the smallest (0 is the
// code of no value).  The kernel's keys are exact within 2^spread_k of the largest
// of their tile.
// (Code that runs once costs its fetching, so it is kept short: a lane takes one
// block column of every 32 / C-th key.)
template <int D, int kRows>
__device__ __forceinline__ bool too_wide(const AttnParams& a, const Cursor& c, int32_t n, int32_t tok, int32_t spread_v,
                                         int32_t spread_k) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31;
  const Common rows = common_of(a, c.len, c.nq, c.rt, kRows);
  if (rows.one) return false;
  int32_t all = 0, some = 0, least = 255;  // of this lane's keys
  bool k_wide = false;
  auto over_lanes = [&](int32_t v) {  // the largest of the lanes that have this block column
#pragma unroll 1
    for (int o = C; o < 32; o <<= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
  };
  bool any = false, wide = false;
  // first the tiles that not all see, whose other keys mostly tell already
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int32_t s = 0; s < n; ++s) {
      if (pass == 0 && s % 32 == 0) {  // 32 tiles at a time
        const int32_t mine = s + lane;
        if (__all_sync(0xFFFFFFFFu, mine >= n || all_see(a, rows, c.s.tile(c.t + min(mine, n - 1)) * tok, tok))) {
          s += 31;
          continue;
        }
      }
      const int32_t tok0 = c.s.tile(c.t + s) * tok;
      if (all_see(a, rows, tok0, tok) != (pass == 1)) continue;
      any = true;
      int32_t kmax = 0, kmin = 255;
#pragma unroll 4
      for (int32_t i = lane / C; i < tok; i += 32 / C) {
        const int32_t j = tok0 + i;
        if (!c.s.has(a, j)) continue;
        const int64_t at = key_row(a, c, j) * C + lane % C;
        const int32_t v = a.v_scales[at], k = spread_k > 0 && pass == 0 ? a.k_scales[at] : 0;
        const bool common = all_see(a, rows, j, 1);
        if (v != 255 && common) all = max(all, v);
        if (v != 255 && v > 0 && !common) some = max(some, v), least = min(least, v);
        if (k != 255 && k > 0) kmax = max(kmax, k), kmin = min(kmin, k);
      }
      if (spread_k > 0 && pass == 0)
        k_wide = k_wide || __reduce_min_sync(0xFFFFFFFFu, kmin) < __reduce_max_sync(0xFFFFFFFFu, kmax) - spread_k;
      if (pass == 1) {
        wide = __any_sync(0xFFFFFFFFu, over_lanes(some) > over_lanes(all) + spread_v);
        if (!wide) return false;
      }
    }
    if (k_wide) return true;
    if (!any) return false;
    wide = __any_sync(0xFFFFFFFFu, over_lanes(some) > over_lanes(all) + spread_v);
    if (!wide) return false;
  }
  // no keys that all see: every row sees one of the others
  if (__any_sync(0xFFFFFFFFu, all > 0)) return true;
  return __any_sync(0xFFFFFFFFu, some > int32_t(__reduce_min_sync(0xFFFFFFFFu, least)) + spread_v);
}

// One row (of the segment at c) over n tiles of `tok` keys from tile c.t on, by a
// whole warp: a lane is a key for the scores and has D / 32 columns of the output.
// part_o is null for a row of the output, else column d of its partial lies at
// (d / 4) * part_step + d % 4.  Rarely called, and slow: where a last token 2^30
// times as large sends all rows here, 16 sequences of 4,000 keys with 4 queries of
// 32 heads take 1.1 ms instead of 39 us, 2 x 512 queries on 4,096 keys 10.7 ms
// instead of 78 us (with a load at a time 3.1 and 28 ms).
template <int D>
__device__ __forceinline__ void wide_row(const AttnParams& a, const Cursor& cu, int32_t n, int32_t tok, int32_t row,
                                         float* part_o, int64_t part_step, float2* part_ml) {
  constexpr int C = D / 32;
  constexpr int kAtOnce = 8;  // keys of p v whose loads are under way
  const int lane = threadIdx.x & 31;
  const int32_t qi = row / a.group, hq = cu.h * a.group + row - qi * a.group, pos = cu.len - cu.nq + qi;
  const int32_t end = a.causal ? min(cu.len, pos + 1) : cu.len, from = a.window > 0 ? pos - a.window + 1 : 0;
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + int64_t(cu.q0 + qi) * a.q_st + int64_t(hq) * a.q_sh;
  float qv[C];  // element 32 c + lane
  float o[C];   // column C lane + c
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const uint32_t x = q[32 * c + lane];
    qv[c] = a.bf16 ? word_to_f32<__nv_bfloat16>(x).x : word_to_f32<__half>(x).x;
    o[c] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
#pragma unroll 1
  for (int32_t i = 0; i < n * (tok / 32); ++i) {
    const int32_t t = i / (tok / 32);
    const int32_t j = cu.s.tile(cu.t + t) * tok + (i - t * (tok / 32)) * 32 + lane;
    const bool seen = j < end && (j >= from || j < a.sinks);
    const uint32_t any = __ballot_sync(0xFFFFFFFFu, seen);
    if (any == 0) continue;
    const int64_t at = seen ? key_row(a, cu, j) : 0;  // of the others any row that there is
    uint4 codes[C];
    uint32_t scales[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      codes[c] = reinterpret_cast<const uint4*>(a.k_codes + at * (D / 2))[c];
      scales[c] = a.k_scales[at * C + c];
    }
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t w[4] = {codes[c].x, codes[c].y, codes[c].z, codes[c].w};
      float part = 0.0f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t h[4];
        e2m1x8_to_half(w[x], h);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float2 k = word_to_f32<__half>(h[y]);
          part = fmaf(k.x, __shfl_sync(0xFFFFFFFFu, qv[c], 8 * x + 2 * y), part);
          part = fmaf(k.y, __shfl_sync(0xFFFFFFFFu, qv[c], 8 * x + 2 * y + 1), part);
        }
      }
      s = fmaf(part, e8m0_value(scales[c]), s);
    }
    s = seen ? s * a.scale_log2 : -INFINITY;
    float top = s;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
    top = fmaxf(top, m);
    const float ref = top == -INFINITY ? 0.0f : top;
    const float alpha = exp2_approx(m - ref), p = exp2_approx(s - (ref - kWeightLog2));
    m = top;
    l = l * alpha + p;
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] *= alpha;
#pragma unroll 1
    for (int u0 = 0; u0 < 32; u0 += kAtOnce) {
      if ((any >> u0 & ((1u << kAtOnce) - 1)) == 0) continue;
      uint32_t v[kAtOnce], e[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int64_t key = __shfl_sync(0xFFFFFFFFu, at, u0 + u);
        const uint8_t* src = a.v_codes + key * (D / 2) + lane * (C / 2);
        if constexpr (C == 2) v[u] = *src;
        else if constexpr (C == 4) v[u] = *reinterpret_cast<const uint16_t*>(src);
        else v[u] = *reinterpret_cast<const uint32_t*>(src);
        e[u] = a.v_scales[key * C + lane * C / 32];
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const float pu = __shfl_sync(0xFFFFFFFFu, p, u0 + u);
        if (!(any >> (u0 + u) & 1)) continue;  // what is not seen may be NaN
        uint32_t h[4];
        e2m1x8_to_half(v[u], h);
        const float f = e8m0_value(e[u]);
#pragma unroll
        for (int c = 0; c < C; c += 2) {
          const float2 x = word_to_f32<__half>(h[c / 2]);
          o[c] = fmaf(pu, x.x * f, o[c]), o[c + 1] = fmaf(pu, x.y * f, o[c + 1]);
        }
      }
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
  const int32_t pe = part_exponent(l);
  if (part_o != nullptr) {
#pragma unroll
    for (int c = 0; c < C; ++c) part_o[(lane * C + c) / 4 * part_step + (lane * C + c) % 4] = o[c] * pow2i(-pe);
    if (lane == 0) *part_ml = make_float2(m + float(pe), l * pow2i(-pe));
    return;
  }
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
  uint16_t* out = static_cast<uint16_t*>(a.out) + int64_t(cu.q0 + qi) * a.o_st + int64_t(hq) * a.o_sh + lane * C;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const float f = o[c] * inv;
    out[c] = uint16_t(a.bf16 ? f32_to_word<__nv_bfloat16>(f, 0.0f) : f32_to_word<__half>(f, 0.0f));
  }
  if (lane == 0 && a.lse != nullptr)
    a.lse[int64_t(cu.q0 + qi) * (a.kv_heads * a.group) + hq] =
        l == 0.0f ? -INFINITY : (m - kWeightLog2 + log2f(l)) * 0.6931471805599453f;
}

// Calls f(segment, its tiles, its place among the workers' partials) for the
// segments of the worker's run of `places` places from `first` on.
template <int kRows, class F>
__device__ __forceinline__ void walk_run(const SplitParams& sp, const Cursor& first, int32_t places, int32_t worker,
                                         int32_t tok, F f) {
  Cursor c = first;
#pragma unroll 1
  for (int64_t part = int64_t(worker) * 2;; part = int64_t(worker) * 2 + 1) {
    const int32_t n = min(c.s.n - c.t, places);
    f(c, n, part);
    places -= n + sp.edge;
    if (places <= 0) return;
    c.t += n - 1;
    cursor_next(c, sp.a, kRows, tok);
  }
}
// Rows r0, r0 + dr, .. of a segment (or of the run's part of it) anew.
template <int D, int kRows, bool kByColumns>
__device__ __forceinline__ void wide_segment(const SplitParams& sp, const Cursor& c, int32_t n, int64_t part, int32_t tok,
                                             int32_t r0, int32_t dr) {
  const bool whole = c.t == 0 && n == c.s.n;
#pragma unroll 1
  for (int32_t r = r0; r < kRows && c.rt * kRows + r < c.nq * sp.a.group; r += dr)
    wide_row<D>(sp.a, c, n, tok, c.rt * kRows + r,
                whole ? nullptr : sp.part_o + (kByColumns ? (part * (D / 4) * kRows + r) * 4 : (part * kRows + r) * D),
                kByColumns ? kRows * 4 : 4, sp.part_ml + part * kRows + r);
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
