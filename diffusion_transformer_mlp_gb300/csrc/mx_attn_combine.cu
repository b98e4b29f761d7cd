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

template <int D, int kRows, int kCols>
__global__ void __launch_bounds__(kCombineThreads) k_attn_combine(const __grid_constant__ SplitParams sp, int32_t tok) {
  const AttnParams& a = sp.a;
  constexpr int kItems = kRows * kCols / 8;
  constexpr int kSlices = kCombineThreads / kItems;
  constexpr int kHeld = kMostParts / kRows;
  __shared__ float weight[kHeld][kRows];
  __shared__ float red[kCombineThreads / 32][kRows], row_m[kRows], row_l[kRows];
  __shared__ float4 sum[(kSlices - 1) * kItems * 2];
  grid_wait();
  const int32_t h = blockIdx.x / (D / kCols), col0 = int32_t(blockIdx.x % (D / kCols)) * kCols;
  const int32_t rt = blockIdx.y, b = blockIdx.z;
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
  // first row of the i-th partial
  auto rows_of = [&](int32_t i) { return (int64_t(w0 + i) * 2 + (i == 0 ? slot0 : 0)) * kRows; };
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
  const int32_t row = rt * kRows + r, qi = row / a.group, hq = h * a.group + row - qi * a.group;
  store_o8(a, static_cast<uint16_t*>(a.out) + int64_t(q0 + qi) * a.o_st + int64_t(hq) * a.o_sh + d, f);
  if (d == 0 && a.lse != nullptr)
    a.lse[int64_t(q0 + qi) * (a.kv_heads * a.group) + hq] =
        l == 0.0f ? -INFINITY : (row_m[r] + kJoinLog2 - kWeightLog2 + log2f(l)) * 0.6931471805599453f;
}

// The same for segments of 128 or 256 rows.  Of those few are split, at most
// one for each boundary between two workers' runs: block y takes the segment
// that worker y's run starts inside of, if no run before does so too.  A
// thread is a row and eight columns.  Blocks behind those write the row tiles
// that see no key: the first ones of a sequence that has fewer keys than queries.
template <int D, int kRows>
__global__ void __launch_bounds__(256) k_attn_join(const __grid_constant__ SplitParams sp, int32_t tok) {
  const AttnParams& a = sp.a;
  const int32_t r = threadIdx.x % kRows, d = (int(blockIdx.x) * (256 / kRows) + int(threadIdx.x) / kRows) * 8;
  auto write = [&](const Cursor& c, const float (&f)[8], float lse) {
    const int32_t row = c.rt * kRows + r;
    if (row >= c.nq * a.group) return;
    const int32_t qi = row / a.group, hq = c.h * a.group + row - qi * a.group;
    store_o8(a, static_cast<uint16_t*>(a.out) + int64_t(c.q0 + qi) * a.o_st + int64_t(hq) * a.o_sh + d, f);
    if (d == 0 && a.lse != nullptr) a.lse[int64_t(c.q0 + qi) * (a.kv_heads * a.group) + hq] = lse;
  };
  grid_wait();
  const int32_t w = blockIdx.y;
  Cursor c;
  if (w >= sp.workers) {
    c.b = w - sp.workers;
    cursor_seq(c, a);
    const float zero[8] = {};
    for (c.rt = 0; c.rt * kRows < c.nq * a.group && row_span(a, c.len, c.nq, c.rt, kRows, tok).n == 0; ++c.rt)
      for (c.h = 0; c.h < a.kv_heads; ++c.h) write(c, zero, -INFINITY);
    return;
  }
  const int64_t total = sp.prefix[a.seqs];
  const int32_t workers = live_workers(sp, total);
  if (w == 0 || w >= workers) return;
  c = sp.start[w];
  const int64_t first = worker_start(total, w, workers) - c.t;  // place of the segment's first tile
  if (c.t == 0 || worker_start(total, w - 1, workers) > first) return;
  const int32_t parts = worker_of(total, first + c.s.n - 1, workers) - (w - 1) + 1;
  const int32_t slot0 = worker_start(total, w - 1, workers) >= first - sp.edge ? 0 : 1;
  auto part_of = [&](int32_t i) { return int64_t(w - 1 + i) * 2 + (i == 0 ? slot0 : 0); };
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
  write(c, f, l == 0.0f ? -INFINITY : (m + kJoinLog2 - kWeightLog2 + log2f(l)) * 0.6931471805599453f);
}

template <int D, int kRows>
nvfp4_status combine_launch(int tok, int row_tiles, const SplitParams& sp, cudaStream_t stream) {
  const bool few = int64_t(sp.a.kv_heads) * row_tiles * sp.a.seqs < 128;
  return launch("launch k_attn_combine", few ? k_attn_combine<D, kRows, 32> : k_attn_combine<D, kRows, 64>,
                dim3(unsigned(sp.a.kv_heads) * (D / (few ? 32 : 64)), unsigned(row_tiles), unsigned(sp.a.seqs)),
                dim3(kCombineThreads), 0, 0, stream, sp, int32_t(tok));
}

template <int D, int kRows>
nvfp4_status join_launch(int tok, const SplitParams& sp, cudaStream_t stream) {
  return launch("launch k_attn_join", k_attn_join<D, kRows>,
                dim3(unsigned(D * kRows / (8 * 256)), unsigned(sp.workers + sp.a.seqs)), dim3(256), 0, 0, stream, sp,
                int32_t(tok));
}

}  // namespace

nvfp4_status attn_join(int dim, int tok, const SplitParams& sp, cudaStream_t stream) {
  if (dim == 64) return join_launch<64, 256>(tok, sp, stream);
  if (dim == 128) return join_launch<128, 256>(tok, sp, stream);
  return join_launch<256, 128>(tok, sp, stream);
}

nvfp4_status attn_combine(int dim, int rows, int tok, int row_tiles, const SplitParams& sp, cudaStream_t stream) {
  if (rows == 8) {
    if (dim == 64) return combine_launch<64, 8>(tok, row_tiles, sp, stream);
    if (dim == 128) return combine_launch<128, 8>(tok, row_tiles, sp, stream);
    return combine_launch<256, 8>(tok, row_tiles, sp, stream);
  }
  if (dim == 64) return combine_launch<64, 16>(tok, row_tiles, sp, stream);
  if (dim == 128) return combine_launch<128, 16>(tok, row_tiles, sp, stream);
  return combine_launch<256, 16>(tok, row_tiles, sp, stream);
}

}  // namespace nvfp4
