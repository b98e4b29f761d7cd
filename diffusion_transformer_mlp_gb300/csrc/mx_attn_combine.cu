// The last step of attention over the cache: joining partial results.
#include <string>

#include "mx_attn.cuh"

namespace nvfp4 {
namespace {

// Joins the partials of the segments that more than one worker had (see
// SplitParams), in worker order, and writes the rows that see no key at all.
// One block takes kCols columns of a segment of kRows rows: the rows' weights
// of all partials first (a thread each), then the outputs, eight columns a
// thread with the partials dealt over kSlices threads.  Few segments have many
// partials each (one conversation of 16,000 keys, 8 heads: 125), and are spread
// over more blocks: 32 columns a block below 128 segments (8 heads, dim 128, the
// whole attention: 24.2 us, with 64 columns 27.4), else 64 (256 segments of 300
// keys: 16.9 us, with 32 columns 19.4).
constexpr int kCombineThreads = 256;
constexpr int kMostParts = 512;  // weights held at a time
constexpr int kFewParts = 4;

template <int D, int kRows, int kCols>
__device__ __forceinline__ void combine_block(const SplitParams& sp, int32_t tok, int32_t bx, int32_t rt, int32_t b) {
  const AttnParams& a = sp.a;
  constexpr int kItems = kRows * kCols / 8;
  constexpr int kSlices = kCombineThreads / kItems;
  constexpr int kHeld = kMostParts / kRows;
  __shared__ float weight[kHeld][kRows];
  __shared__ float red[kCombineThreads / 32][kRows], row_m[kRows], row_l[kRows];
  __shared__ float4 sum[(kSlices - 1) * kItems * 2];
  const int32_t h = bx / (D / kCols), col0 = bx % (D / kCols) * kCols;
  const int32_t len = a.lens[b], nq = seq_queries(a, b);
  const int32_t q0 = seq_start(a, b);
  const int32_t live = min(kRows, nq * a.group - rt * kRows);
  if (live <= 0) return;
  int64_t first = sp.prefix[b];
  for (int32_t r = 0; r < rt; ++r) first += int64_t(row_span(a, len, nq, r, kRows, tok).n) * a.kv_heads;
  const int32_t n = row_span(a, len, nq, rt, kRows, tok).n;
  first += int64_t(h) * n;
  const int64_t total = sp.prefix[a.seqs];
  const int32_t workers = live_workers(sp, total);
  int32_t w0 = 0, parts = 0, slot0 = 0;
  if (n > 0) {
    w0 = worker_of(total, first, workers);
    parts = worker_of(total, first + n - 1, workers) - w0 + 1;
    if (parts == 1) return;  // written by its worker
    slot0 = worker_start(total, w0, workers) == first ? 0 : 1;
  }
  auto write = [&](int32_t r, int32_t d, const float (&f)[8], float lse) {
    const int32_t row = rt * kRows + r, qi = row / a.group, hq = h * a.group + row - qi * a.group;
    store_o8(a, int64_t(q0 + qi) * a.o_st + int64_t(hq) * a.o_sh + d, f);
    if (d == 0 && a.lse != nullptr) a.lse[int64_t(q0 + qi) * (a.kv_heads * a.group) + hq] = lse;
  };
  // first row of the i-th partial
  auto rows_of = [&](int32_t i) { return (int64_t(w0 + i) * 2 + (i == 0 ? slot0 : 0)) * kRows; };
  if (parts <= kFewParts) {
    // Short sequences: a thread an item, with all its loads at once and no barrier.
    // The sums are those of the way below, in its order and with its roundings, so
    // that results do not depend on where a run ends (120 sequences of 32 to 1,025
    // keys, 8 heads: the pass 41.6 us without this, so 39.7; 16 of them 15.2 and 14.7).
    const int item = threadIdx.x;
    const int32_t r = item / (kCols / 8), d = col0 + item % (kCols / 8) * 8;
    if (item >= kItems || r >= live) return;
    float2 ml[kFewParts];
    float4 u[kFewParts], v[kFewParts];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kFewParts; ++i) {
      ml[i] = make_float2(-INFINITY, 0.0f);
      u[i] = v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (i < parts) {
        const float4* src = reinterpret_cast<const float4*>(sp.part_o + (rows_of(i) + r) * D + d);
        ml[i] = sp.part_ml[rows_of(i) + r], u[i] = src[0], v[i] = src[1];
      }
      m = fmaxf(m, ml[i].x);
    }
    const float ref = m == -INFINITY ? 0.0f : m + kJoinLog2;
    float w[kFewParts], l[kFewParts];
#pragma unroll
    for (int i = 0; i < kFewParts; ++i) {
      w[i] = i < parts ? exp2_approx(ml[i].x - ref) : 0.0f;
      l[i] = __fmul_rn(ml[i].y, w[i]);
    }
    const float sum = __fadd_rn(__fadd_rn(l[0], l[1]), __fadd_rn(l[2], l[3]));
    const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
    float f[8];
#pragma unroll
    for (int s = 0; s < kSlices; ++s) {
      float t[8] = {};
#pragma unroll
      for (int i = s; i < kFewParts; i += kSlices) {
        if (i >= parts) break;
        const float x[8] = {u[i].x, u[i].y, u[i].z, u[i].w, v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = __fmaf_rn(x[k], w[i], t[k]);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = s == 0 ? t[k] : __fadd_rn(f[k], t[k]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] *= inv;
    write(r, d, f, sum == 0.0f ? -INFINITY : (m + kJoinLog2 - kWeightLog2 + log2f(sum)) * 0.6931471805599453f);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, mine = threadIdx.x % kRows;
  // `v` of all threads of a row, into out[row]
  auto over_rows = [&](float v, auto op, float* out) {
#pragma unroll
    for (int o = kRows; o < 32; o <<= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if (lane < kRows) red[warp][lane] = v;
    __syncthreads();
    if (threadIdx.x < kRows) {
      v = red[0][threadIdx.x];
#pragma unroll
      for (int i = 1; i < kCombineThreads / 32; ++i) v = op(v, red[i][threadIdx.x]);
      out[threadIdx.x] = v;
    }
    __syncthreads();
  };
  // the rows' maxima over all partials: kRows threads a partial
  float m = -INFINITY;
  for (int32_t i = threadIdx.x / kRows; i < parts; i += kCombineThreads / kRows)
    m = fmaxf(m, sp.part_ml[rows_of(i) + mine].x);
  over_rows(m, [](float x, float y) { return fmaxf(x, y); }, row_m);
  m = row_m[mine];
  const float ref = m == -INFINITY ? 0.0f : m + kJoinLog2;
  const int item = threadIdx.x % kItems, slice = threadIdx.x / kItems;
  const int32_t r = item / (kCols / 8), d = col0 + item % (kCols / 8) * 8;
  float l = 0.0f;  // of this thread's partials
  float f[8] = {};
  for (int32_t i0 = 0; i0 < parts; i0 += kHeld) {
    const int32_t cnt = min(parts - i0, kHeld);
    for (int32_t i = threadIdx.x / kRows; i < cnt; i += kCombineThreads / kRows) {
      const float2 ml = sp.part_ml[rows_of(i0 + i) + mine];
      const float w = exp2_approx(ml.x - ref);
      weight[i][mine] = w;
      l += ml.y * w;
    }
    __syncthreads();
#pragma unroll 4
    for (int32_t i = slice; i < cnt; i += kSlices) {
      const float4* src = reinterpret_cast<const float4*>(sp.part_o + (rows_of(i0 + i) + r) * D + d);
      const float4 u = src[0], v = src[1];
      const float c = weight[i][r];
      f[0] += u.x * c, f[1] += u.y * c, f[2] += u.z * c, f[3] += u.w * c;
      f[4] += v.x * c, f[5] += v.y * c, f[6] += v.z * c, f[7] += v.w * c;
    }
    __syncthreads();
  }
  over_rows(l, [](float x, float y) { return x + y; }, row_l);
  if (slice > 0) {
    sum[((slice - 1) * kItems + item) * 2] = make_float4(f[0], f[1], f[2], f[3]);
    sum[((slice - 1) * kItems + item) * 2 + 1] = make_float4(f[4], f[5], f[6], f[7]);
  }
  __syncthreads();
  if (slice > 0 || r >= live) return;
#pragma unroll
  for (int x = 0; x < kSlices - 1; ++x) {
    const float4 u = sum[(x * kItems + item) * 2], v = sum[(x * kItems + item) * 2 + 1];
    f[0] += u.x, f[1] += u.y, f[2] += u.z, f[3] += u.w;
    f[4] += v.x, f[5] += v.y, f[6] += v.z, f[7] += v.w;
  }
  l = row_l[r];
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] *= inv;
  write(r, d, f, l == 0.0f ? -INFINITY : (row_m[r] + kJoinLog2 - kWeightLog2 + log2f(l)) * 0.6931471805599453f);
}

template <int D, int kRows, int kCols>
__global__ void __launch_bounds__(kCombineThreads) k_attn_combine(const __grid_constant__ SplitParams sp, int32_t tok) {
  grid_wait();
  combine_block<D, kRows, kCols>(sp, tok, blockIdx.x, blockIdx.y, blockIdx.z);
}

// The same where segments are many and thus short: not a block for each of them, most
// of which a worker has all of, but warps for each boundary between two workers' runs
// that lies in a segment; those of a segment of several such boundaries share its rows.
// A lane is a row and four columns.  A row's weights are worked out by its kLanes
// lanes, a partial each at a time, and passed on by shuffles.  All sums are in the
// order, and with the roundings, of k_attn_combine's, so that a result does not depend
// on which of them joins it.  Warps behind those write the rows that see no key.
// 192 sequences of 33 to 1,025 keys, 8 heads: writing and attending 54.9 us by
// segments, most of whose instructions looked for partials that were not there, and
// 48.0 so (with eight columns a lane a long sequence among short ones was up to 13 us
// slower).
constexpr int kBoundaryThreads = 128, kUnder = 8;  // loads under way
// Warps of a boundary (192 sequences of 8 rows with four of them 1.1 us more).
__host__ __device__ constexpr int32_t split_of(int rows) { return rows / 4; }

template <int D, int kRows>
__device__ __forceinline__ void combine_boundary(const SplitParams& sp, int32_t tok, int32_t unit) {
  constexpr int kLanes = D == 64 ? 16 : 32, kAtOnce = 32 / kLanes;  // lanes of a row, rows of a warp
  constexpr int kPieces = D / 4 / kLanes;  // of a row
  constexpr int kSlices = 32 / kRows, kSums = 256 / kRows;  // of k_attn_combine's threads: partials of a row's outputs, sums
  constexpr int kAtATime = kLanes < kSums ? kLanes : kSums;  // partials
  constexpr int kHeld = kSums / kAtATime;
  constexpr int32_t kSplit = split_of(kRows);
  const AttnParams& a = sp.a;
  const int lane = threadIdx.x & 31, col = lane % kLanes, lane0 = lane - col;
  const int32_t w = unit / kSplit, part_of_unit = unit - w * kSplit;
  Cursor c;
  auto write = [&](int32_t row, int32_t d, const float (&f)[4], float lse) {
    if (row >= c.nq * a.group) return;
    const int32_t qi = row / a.group, hq = c.h * a.group + row - qi * a.group;
    store_o4(a, int64_t(c.q0 + qi) * a.o_st + int64_t(hq) * a.o_sh + d, f);
    if (d == 0 && a.lse != nullptr) a.lse[int64_t(c.q0 + qi) * (a.kv_heads * a.group) + hq] = lse;
  };
  if (w >= sp.workers) {
    c.b = w - sp.workers;
    if (c.b >= a.seqs) return;
    cursor_seq(c, a);
    const float zero[4] = {};
    for (c.rt = 0; c.rt * kRows < c.nq * a.group && row_span(a, c.len, c.nq, c.rt, kRows, tok).n == 0; ++c.rt)
      for (c.h = part_of_unit; c.h < a.kv_heads; c.h += kSplit)
        for (int32_t i = lane; i < kRows * (D / 4); i += 32)
          write(c.rt * kRows + i / (D / 4), i % (D / 4) * 4, zero, -INFINITY);
    return;
  }
  const int64_t total = sp.prefix[a.seqs];
  c = sp.start[w];  // not written of workers without a run, and not looked at
  const int32_t workers = live_workers(sp, total);
  if (w == 0 || w >= workers || c.t == 0) return;
  const int64_t first = worker_start(total, w, workers) - c.t;  // place of the segment's first tile
  const int32_t begin = worker_of(total, first, workers);
  const int32_t parts = worker_of(total, first + c.s.n - 1, workers) - begin + 1;
  const int32_t slot0 = worker_start(total, begin, workers) == first ? 0 : 1;
  auto row_of = [&](int32_t i, int32_t r) { return (int64_t(begin + i) * 2 + (i == 0 ? slot0 : 0)) * kRows + r; };
  const int32_t live = min(kRows, c.nq * a.group - c.rt * kRows);
  for (int32_t x0 = (w - begin - 1) * kSplit + part_of_unit; x0 * kAtOnce < live * kPieces; x0 += (parts - 1) * kSplit) {
    const int32_t r = x0 / kPieces * kAtOnce + lane / kLanes;  // less than kRows
    const int32_t d = (x0 % kPieces * kLanes + col) * 4;
    float m = -INFINITY;
    for (int32_t i = col; i < parts; i += kLanes) m = fmaxf(m, sp.part_ml[row_of(i, r)].x);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float ref = m == -INFINITY ? 0.0f : m + kJoinLog2;
    float l[kHeld] = {}, f[kSlices][4] = {};
    for (int32_t i0 = 0; i0 < parts; i0 += kSums) {
#pragma unroll
      for (int x = 0; x < kHeld; ++x) {
        const int32_t from = i0 + x * kAtATime;
        if (from >= parts) break;
        float weight = 0.0f;
        if (col < kAtATime && from + col < parts) {
          const float2 ml = sp.part_ml[row_of(from + col, r)];
          weight = exp2_approx(ml.x - ref);
          l[x] = __fmaf_rn(ml.y, weight, l[x]);
        }
        const int32_t n = min(parts - from, kAtATime);
#pragma unroll 1
        for (int32_t i = 0; i < n; i += kUnder) {
          float4 u[kUnder];
#pragma unroll
          for (int k = 0; k < kUnder; ++k) {
            if (i + k >= n) break;
            u[k] = *reinterpret_cast<const float4*>(sp.part_o + row_of(from + i + k, r) * D + d);
          }
#pragma unroll
          for (int k = 0; k < kUnder; ++k) {
            if (i + k >= n) break;
            const float g = __shfl_sync(0xFFFFFFFFu, weight, lane0 + i + k);
            const float y[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) f[k % kSlices][e] = __fmaf_rn(y[e], g, f[k % kSlices][e]);
          }
        }
      }
    }
    float sum = 0.0f;
#pragma unroll
    for (int x = 0; x < kHeld; ++x) {
      if (x * kAtATime >= parts) break;
#pragma unroll
      for (int o = 1; o < kSlices; o <<= 1) l[x] += __shfl_xor_sync(0xFFFFFFFFu, l[x], o);
      for (int32_t i = 0; i < min(parts - x * kAtATime, kAtATime); i += kSlices)
        sum = __fadd_rn(sum, __shfl_sync(0xFFFFFFFFu, l[x], lane0 + i));
    }
    const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int x = 1; x < kSlices; ++x) f[0][e] = __fadd_rn(f[0][e], f[x][e]);
      f[0][e] *= inv;
    }
    if (r < live)
      write(c.rt * kRows + r, d, f[0], sum == 0.0f ? -INFINITY : (m + kJoinLog2 - kWeightLog2 + log2f(sum)) * 0.6931471805599453f);
  }
}

template <int D, int kRows>
__global__ void __launch_bounds__(kBoundaryThreads)
    k_attn_combine_boundaries(const __grid_constant__ SplitParams sp, int32_t tok) {
  grid_wait();
  combine_boundary<D, kRows>(sp, tok, int32_t(blockIdx.x * (kBoundaryThreads / 32) + (threadIdx.x >> 5)));
}

// The same for segments of 128 or 256 rows.  Of those few are split, at the
// boundaries between two workers' runs: blocks (x, w) are for the segment that
// worker w's run starts inside of, whose columns they share with the blocks of
// the other runs that start inside of it.  A thread is a row and eight columns
// at a time.  (Blocks of all columns for the first of these runs, which left the
// others' without work: 9.5 us for 19 partials of 16 segments, so 7.1; eight or
// sixteen blocks a worker 1 to 4 us more.)  Blocks
// behind those write the row tiles that see no key: the first ones of a sequence
// that has fewer keys than queries.
constexpr int kJoinBlocks = 4;  // for each worker

template <int D, int kRows>
__device__ __forceinline__ void join_block(const SplitParams& sp, int32_t tok, int32_t bx, int32_t w) {
  constexpr int kCols = 256 / kRows * 8;  // of a block at a time
  const AttnParams& a = sp.a;
  const int32_t r = threadIdx.x % kRows, d0 = int32_t(threadIdx.x) / kRows * 8;
  auto write = [&](const Cursor& c, int32_t d, const float (&f)[8], float lse) {
    const int32_t row = c.rt * kRows + r;
    if (row >= c.nq * a.group) return;
    const int32_t qi = row / a.group, hq = c.h * a.group + row - qi * a.group;
    store_o8(a, int64_t(c.q0 + qi) * a.o_st + int64_t(hq) * a.o_sh + d, f);
    if (d == 0 && a.lse != nullptr) a.lse[int64_t(c.q0 + qi) * (a.kv_heads * a.group) + hq] = lse;
  };
  Cursor c;
  if (w >= sp.workers) {
    c.b = w - sp.workers;
    cursor_seq(c, a);
    const float zero[8] = {};
    for (c.rt = 0; c.rt * kRows < c.nq * a.group && row_span(a, c.len, c.nq, c.rt, kRows, tok).n == 0; ++c.rt)
      for (c.h = 0; c.h < a.kv_heads; ++c.h)
        for (int32_t d = bx * kCols; d < D; d += kJoinBlocks * kCols) write(c, d + d0, zero, -INFINITY);
    return;
  }
  const int64_t total = sp.prefix[a.seqs];
  const int32_t workers = live_workers(sp, total);
  if (w == 0 || w >= workers) return;
  c = sp.start[w];
  if (c.t == 0) return;  // its run starts with the segment
  if (c.rt * kRows + r >= c.nq * a.group) return;  // no row, and no partial of it
  const int64_t first = worker_start(total, w, workers) - c.t;  // place of the segment's first tile
  const int32_t begin = worker_of(total, first, workers);
  const int32_t parts = worker_of(total, first + c.s.n - 1, workers) - begin + 1;
  const int32_t slot0 = worker_start(total, begin, workers) >= first - sp.edge ? 0 : 1;
  auto part_of = [&](int32_t i) { return int64_t(begin + i) * 2 + (i == 0 ? slot0 : 0); };
  const int32_t mine = (w - begin - 1) * kJoinBlocks + bx, all = (parts - 1) * kJoinBlocks;
  for (int32_t d = mine * kCols + d0; d < D; d += all * kCols) {
    // in one pass, against the maximum so far
    float f[8] = {}, l = 0.0f, m = -INFINITY;
#pragma unroll 4
    for (int32_t i = 0; i < parts; ++i) {
      const float2 ml = sp.part_ml[part_of(i) * kRows + r];
      const float4* src = reinterpret_cast<const float4*>(sp.part_o) + (part_of(i) * (D / 4) + d / 4) * kRows + r;
      const float4 u = src[0], v = src[kRows];
      const float top = fmaxf(m, ml.x), ref = top == -INFINITY ? 0.0f : top + kJoinLog2;
      const float old = top == -INFINITY ? 1.0f : exp2_approx(m - top), g = exp2_approx(ml.x - ref);
      m = top;
      l = l * old + ml.y * g;
      f[0] = f[0] * old + u.x * g, f[1] = f[1] * old + u.y * g, f[2] = f[2] * old + u.z * g, f[3] = f[3] * old + u.w * g;
      f[4] = f[4] * old + v.x * g, f[5] = f[5] * old + v.y * g, f[6] = f[6] * old + v.z * g, f[7] = f[7] * old + v.w * g;
    }
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] *= inv;
    write(c, d, f, l == 0.0f ? -INFINITY : (m + kJoinLog2 - kWeightLog2 + log2f(l)) * 0.6931471805599453f);
  }
}

template <int D, int kRows>
__global__ void __launch_bounds__(256) k_attn_join(const __grid_constant__ SplitParams sp, int32_t tok) {
  grid_wait();
  join_block<D, kRows>(sp, tok, blockIdx.x, blockIdx.y);
}

// Both at once, of two launches that went before: k_attn_join's blocks, then
// k_attn_combine's or (kBoundaries) the others'.
template <int D, int kRows, bool kBoundaries>
__global__ void __launch_bounds__(256)
    k_attn_join_both(const __grid_constant__ SplitParams many, const __grid_constant__ SplitParams few, int32_t many_tok,
                     int32_t few_tok, int32_t joins, int32_t bx, int32_t by) {
  grid_wait();
  const int32_t i = blockIdx.x, j = i - joins;
  if (j < 0)
    join_block<D, D == 256 ? 128 : 256>(many, many_tok, i % kJoinBlocks, i / kJoinBlocks);
  else if constexpr (kBoundaries)
    combine_boundary<D, kRows>(few, few_tok, j * 8 + int32_t(threadIdx.x >> 5));
  else
    combine_block<D, kRows, 64>(few, few_tok, j % bx, j / bx % by, j / bx / by);
}

template <int D, int kRows>
nvfp4_status combine_launch(const Pending& w, cudaStream_t stream) {
  const SplitParams& sp = w.sp;
  if (sp.start != nullptr) {
    constexpr int64_t kSplit = split_of(kRows), kWarps = kBoundaryThreads / 32;
    return launch("launch k_attn_combine_boundaries", k_attn_combine_boundaries<D, kRows>,
                  dim3(unsigned((kSplit * (sp.workers + sp.a.seqs) + kWarps - 1) / kWarps)), dim3(kBoundaryThreads), 0, 0,
                  stream, sp, w.tok);
  }
  const bool few = int64_t(sp.a.kv_heads) * w.row_tiles * sp.a.seqs < 128;
  return launch("launch k_attn_combine", few ? k_attn_combine<D, kRows, 32> : k_attn_combine<D, kRows, 64>,
                dim3(unsigned(sp.a.kv_heads) * (D / (few ? 32 : 64)), unsigned(w.row_tiles), unsigned(sp.a.seqs)),
                dim3(kCombineThreads), 0, 0, stream, sp, w.tok);
}

template <int D>
nvfp4_status join_launch(const Pending& w, cudaStream_t stream) {
  return launch("launch k_attn_join", k_attn_join<D, D == 256 ? 128 : 256>,
                dim3(unsigned(kJoinBlocks), unsigned(w.sp.workers + w.sp.a.seqs)), dim3(256), 0, 0, stream, w.sp, w.tok);
}

template <int D, int kRows>
nvfp4_status both_launch(const Pending& many, const Pending& few, cudaStream_t stream) {
  const SplitParams& sp = few.sp;
  const int64_t segments = int64_t(sp.a.kv_heads) * few.row_tiles * sp.a.seqs, bx = sp.a.kv_heads * int64_t(D / 64);
  const int64_t joins = int64_t(kJoinBlocks) * (many.sp.workers + many.sp.a.seqs);
  const int64_t blocks = sp.start != nullptr ? (int64_t(split_of(kRows)) * (sp.workers + sp.a.seqs) + 7) / 8 : segments * (D / 64);
  if (segments < 128 || joins + blocks > 0x7FFFFFFF) {  // blocks of fewer columns; too large
    const nvfp4_status st = join_launch<D>(many, stream);
    return st != NVFP4_OK ? st : combine_launch<D, kRows>(few, stream);
  }
  return launch("launch k_attn_join_both",
                sp.start != nullptr ? k_attn_join_both<D, kRows, true> : k_attn_join_both<D, kRows, false>,
                dim3(unsigned(joins + blocks)), dim3(256), 0, 0, stream, many.sp, sp, many.tok, few.tok, int32_t(joins),
                int32_t(bx), few.row_tiles);
}

}  // namespace

nvfp4_status attn_finish(int dim, const Pending& w, cudaStream_t stream) {
  if (w.many) return dim == 64 ? join_launch<64>(w, stream) : (dim == 128 ? join_launch<128>(w, stream) : join_launch<256>(w, stream));
  auto f = w.rows == 8 ? (dim == 64 ? combine_launch<64, 8> : (dim == 128 ? combine_launch<128, 8> : combine_launch<256, 8>))
                       : (dim == 64 ? combine_launch<64, 16> : (dim == 128 ? combine_launch<128, 16> : combine_launch<256, 16>));
  return f(w, stream);
}

nvfp4_status attn_finish_both(int dim, const Pending& many, const Pending& few, cudaStream_t stream) {
  auto f = few.rows == 8 ? (dim == 64 ? both_launch<64, 8> : (dim == 128 ? both_launch<128, 8> : both_launch<256, 8>))
                         : (dim == 64 ? both_launch<64, 16> : (dim == 128 ? both_launch<128, 16> : both_launch<256, 16>));
  return f(many, few, stream);
}

}  // namespace nvfp4
