// Attention of a few query rows over the paged MXFP4 cache (decoding).
//
// With few rows a key or value is used once, so the cache's bytes are the
// work, and what stands in their way is the decoding of 4-bit codes by the
// ordinary pipes.  Each warp therefore works alone: it streams tiles of kTok
// keys through its own TMA ring and keeps Q, the scores, the softmax state
// and the output of its 16 MMA rows in registers (m16n8k16 f16 MMAs; a tile
// of rows is no work for a 128-row tcgen05 tile).
//
//   codes     E2M1 values are decoded unscaled into FP16 (one cvt for two),
//             which is exact; the E8M0 scales never touch the elements.
//   q k^T     Q is held in FP16 under a power of two per row (exact for BF16
//             and FP16 inputs over 2^-28 of the row's largest element; BF16
//             elements below that lose bits that weigh nothing).  Each 32-wide
//             block of the head is one MMA pair whose FP32 result is
//             multiplied by the key's block scale.
//   softmax   running maximum and sum in FP32, weights p 2^14.
//   p v       a value's block scale varies along the contraction, so it goes
//             onto the weights: p 2^14 2^(E - R) with R the largest E of the
//             block column so far (a running maximum like the softmax's).  The
//             factor 2^14 leaves 28 binades below the largest before FP16
//             loses bits.
//   split     kSplit: up to 8 rows, whose weights go in twice, FP16(p) in MMA
//             rows 0..7 and FP16(p - FP16(p)) in rows 8..15, rows that would
//             be idle: the weights then carry 22 bits.  Otherwise 16 rows and
//             weights of 11 bits (FP16; BF16 would keep 8).
//
// The ldmatrix layouts fit the format: a 16-byte row of an 8x8 matrix is one
// block of one token, so for K a lane gets 8 codes of one block, and with
// .trans for V it gets 4 codes of token t in its low and of token t + 1 in
// its high half, the pairs that the second MMA contracts over.
//
// Work is dealt in equal runs of tiles over all warps of the grid, whatever
// the sequences' lengths: the tiles of all (sequence, row tile, kv head)
// segments in a row, worker w taking [total w / W, total (w+1) / W).  A worker
// writes a segment's output itself if it has all of it, else its partial
// (maximum, sum, unnormalised output) goes to the workspace: at most two a
// worker, its first and its last segment.  k_attn_combine joins them in
// worker order.  The split depends on the lengths alone, so results are
// reproducible.
#include <algorithm>
#include <string>

#include "mx_attn.cuh"

namespace nvfp4 {

nvfp4_status make_map(CUtensorMap* map, CUtensorMapDataType dt, const void* base, int rank, const cuuint64_t* dims,
                      const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle, const char* what);

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxSeqs = 1024;  // sequences of one launch (their tile counts sit in shared memory)

template <int D>
struct Tile {
  static constexpr int C = D / 32;                 // blocks of a row
  static constexpr int kTok = D == 256 ? 32 : 64;  // keys of a tile
  static constexpr int kCodes = kTok * D / 2;      // bytes of K (or V) codes
  static constexpr int kScales = kTok * C;
  static constexpr int kStages = 3;
  static constexpr int kKf = kTok * C * 4;  // K scales as float [token][C]
  static constexpr int kVf = kTok * C * 2;  // V factors as half [C][token]
  static constexpr int kWarpCodes = kStages * 2 * kCodes;
  static constexpr int kWarpRest = kStages * 2 * kScales + kKf + kVf;
  // [warp codes x 4][warp rest x 4][barriers]; the tile counts of the
  // sequences lie where the codes go, before the first load
  static constexpr int kBars = kWarps * kStages * 8;
  static constexpr int kSmem = 1024 + kWarps * (kWarpCodes + kWarpRest) + kBars;
  static_assert((kMaxSeqs + 1) * 8 <= kWarps * kWarpCodes, "tile counts");
  static_assert(kCodes % 1024 == 0, "swizzle atoms");
};

struct StreamParams {
  AttnParams a;
  int32_t workers;
  int32_t rows;      // rows of a row tile: 8 (split) or 16
  float* part_o;     // [2 * workers][rows][D]
  float2* part_ml;   // [2 * workers][rows]  (maximum, sum)
  int64_t* prefix;   // [seqs + 1] tiles before each sequence, written by block 0 for k_attn_combine
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

// Tiles of sequence b over all its row tiles and kv heads.
__device__ __forceinline__ int64_t seq_tiles(const AttnParams& a, int32_t b, int32_t rows, int32_t tok) {
  const int32_t len = a.lens[b], nq = seq_queries(a, b);
  int64_t n = 0;
  for (int32_t rt = 0; rt * rows < nq * a.group; ++rt) n += row_span(a, len, nq, rt, rows, tok).n;
  return n * a.kv_heads;
}

// Workers that get a tile: with fewer tiles than warps, the first ones get one
// each, so that all workers of a segment's range have a partial of it.
__device__ __forceinline__ int32_t live_workers(int64_t total, int32_t workers) {
  return int32_t(min(total, int64_t(workers)));
}
__device__ __forceinline__ int64_t worker_start(int64_t total, int32_t w, int32_t workers) {
  return total * w / workers;
}
// The worker whose run holds tile x: the largest w with worker_start(w) <= x.
__device__ __forceinline__ int32_t worker_of(int64_t total, int64_t x, int32_t workers) {
  return int32_t(((x + 1) * workers - 1) / total);
}

// Position in the list of all tiles.
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

__device__ __forceinline__ void cursor_at(Cursor& c, const AttnParams& a, const int64_t* prefix, int64_t x,
                                          int32_t rows, int32_t tok) {
  int32_t lo = 0, hi = a.seqs;  // prefix[lo] <= x < prefix[hi]
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (prefix[mid] <= x) lo = mid;
    else hi = mid;
  }
  c.b = lo;
  cursor_seq(c, a);
  int64_t rem = x - prefix[lo];
  for (c.rt = 0;; ++c.rt) {
    c.s = row_span(a, c.len, c.nq, c.rt, rows, tok);
    const int64_t n = int64_t(c.s.n) * a.kv_heads;
    if (rem < n) break;
    rem -= n;
  }
  c.h = int32_t(rem / c.s.n);
  c.t = int32_t(rem - int64_t(c.h) * c.s.n);
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

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Byte offset of 16-byte chunk c of row t in a tile whose rows are D/2 bytes,
// as the TMA's swizzle of that width lays it out.
template <int D>
__device__ __forceinline__ uint32_t swz(int t, int c) {
  constexpr int C = D / 32;
  return uint32_t(t * (D / 2) + ((c ^ ((t / (8 / C)) & (C - 1))) << 4));
}

// FP16 2^(e - r) for e <= r (0 once it underflows).
__device__ __forceinline__ uint32_t half_pow2(uint32_t e, uint32_t r) {
  const uint32_t d = r - e;
  return d <= 14u ? (15u - d) << 10 : (d <= 24u ? 1u << (24u - d) : 0u);
}

// Eight consecutive elements of a query row, to binary32.
__device__ __forceinline__ void load_q8(const AttnParams& a, const uint16_t* src, float (&f)[8]) {
  uint32_t w[4];
  if (a.q_vec) {
    const uint4 v = *reinterpret_cast<const uint4*>(src);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = uint32_t(src[2 * i]) | uint32_t(src[2 * i + 1]) << 16;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = a.bf16 ? word_to_f32<__nv_bfloat16>(w[i]) : word_to_f32<__half>(w[i]);
    f[2 * i] = t.x, f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ void store_o8(const AttnParams& a, uint16_t* dst, const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = a.bf16 ? f32_to_word<__nv_bfloat16>(f[2 * i], f[2 * i + 1]) : f32_to_word<__half>(f[2 * i], f[2 * i + 1]);
  if (a.o_vec) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dst[2 * i] = uint16_t(w[i]);
      dst[2 * i + 1] = uint16_t(w[i] >> 16);
    }
  }
}

template <int D, bool kSplit>
__global__ void __launch_bounds__(kThreads, 2)
    k_attn_stream(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                  const __grid_constant__ StreamParams sp) {
  using T = Tile<D>;
  constexpr int C = T::C, kTok = T::kTok, NT = kTok / 8, KK = kTok / 16;
  constexpr int kRows = kSplit ? 8 : 16;
  constexpr int R = kSplit ? 1 : 2;  // real rows of a thread: g, and g + 8
  const AttnParams& a = sp.a;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  uint8_t* codes = base + warp * T::kWarpCodes;
  uint8_t* rest = base + kWarps * T::kWarpCodes + warp * T::kWarpRest;
  float* kf = reinterpret_cast<float*>(rest + T::kStages * 2 * T::kScales);
  uint16_t* vf = reinterpret_cast<uint16_t*>(rest + T::kStages * 2 * T::kScales + T::kKf);
  uint8_t* tail = base + kWarps * (T::kWarpCodes + T::kWarpRest);
  uint64_t* full = reinterpret_cast<uint64_t*>(tail) + warp * T::kStages;
  int64_t* prefix = reinterpret_cast<int64_t*>(base);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kWarps * T::kStages; ++i) mbar_init(reinterpret_cast<uint64_t*>(tail) + i, 1);
    fence_barrier_init();
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  // tiles before each sequence: every thread sums a run of sequences, the
  // first warp scans the runs' sums
  {
    __shared__ int64_t run[kThreads];
    const int per = (a.seqs + kThreads - 1) / kThreads;
    const int b0 = min(int(threadIdx.x) * per, a.seqs), b1 = min(b0 + per, a.seqs);
    int64_t sum = 0;
    for (int b = b0; b < b1; ++b) {
      prefix[b] = sum;
      sum += seq_tiles(a, b, kRows, kTok);
    }
    run[threadIdx.x] = sum;
    __syncthreads();
    if (warp == 0) {
      int64_t v[kThreads / 32], s = 0;
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) {
        v[i] = s;
        s += run[lane * (kThreads / 32) + i];
      }
      int64_t inc = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += u;
      }
      const int64_t before = inc - s;
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) run[lane * (kThreads / 32) + i] = before + v[i];
      if (lane == 31) prefix[a.seqs] = inc;
    }
    __syncthreads();
    for (int b = b0; b < b1; ++b) prefix[b] += run[threadIdx.x];
    __syncthreads();
    if (blockIdx.x == 0)
      for (int b = threadIdx.x; b <= a.seqs; b += kThreads) sp.prefix[b] = prefix[b];
  }

  const int64_t total = prefix[a.seqs];
  // the first workers lie in different blocks: few tiles spread over all SMs
  const int32_t worker = warp * int32_t(gridDim.x) + int32_t(blockIdx.x);
  const int32_t workers = live_workers(total, sp.workers);
  const int64_t x0 = worker < workers ? worker_start(total, worker, workers) : 0;
  const int32_t tiles = worker < workers ? int32_t(worker_start(total, worker + 1, workers) - x0) : 0;
  Cursor ld;
  if (tiles > 0) cursor_at(ld, a, prefix, x0, kRows, kTok);
  fence_proxy_async_smem();  // the counts are read, the TMA may write there
  __syncthreads();
  if (tiles <= 0) return;

  // ---- loads: lane i < boxes takes box i of a tile (a page's share of it)
  const int32_t page = 1 << a.page_shift;
  const int32_t box = min(page, kTok), boxes = kTok / box;
  Cursor cu = ld;
  auto issue = [&](int slot) {
    const int32_t tok0 = ld.s.tile(ld.t) * kTok;
    const int32_t nb = min(boxes, (ld.len - tok0 + box - 1) / box);  // boxes that hold a token
    uint8_t* st = codes + slot * 2 * T::kCodes;
    uint8_t* sc = rest + slot * 2 * T::kScales;
    if (lane == 0) mbar_arrive_expect_tx(&full[slot], uint32_t(nb * box) * (D + 2 * C));
    __syncwarp();
    if (lane < nb) {
      const int32_t tok = tok0 + lane * box;
      const int32_t col = min(int64_t(tok >> a.page_shift), a.table_ld - 1);
      int64_t pg = a.table[int64_t(ld.b) * a.table_ld + col];
      pg = min(max(pg, int64_t(0)), a.pages - 1);
      const int32_t z = int32_t(pg * a.kv_heads + ld.h), off = tok & (page - 1);
      tma_load_3d_plain(st + lane * box * (D / 2), &tmap_k, &full[slot], 0, off, z);
      tma_load_3d_plain(st + T::kCodes + lane * box * (D / 2), &tmap_v, &full[slot], 0, off, z);
      const int64_t srow = ((int64_t(z) << a.page_shift) + off) * C;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv)
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         smem_u32(sc + kv * T::kScales + lane * box * C)),
                     "l"((kv ? a.v_scales : a.k_scales) + srow), "r"(box * C), "r"(smem_u32(&full[slot]))
                     : "memory");
    }
  };
  int32_t issued = 0;
  for (; issued < min(T::kStages, tiles); ++issued) {
    issue(issued);
    if (issued + 1 < tiles) cursor_next(ld, a, kRows, kTok);
  }

  // ---- state of the segment
  uint32_t qa[C][2][2 * R];       // Q fragments: block, MMA of the block
  float qf[R];                    // row factor of the scores (log2 domain)
  int32_t pos[R];                 // position of the row's query
  float o[C][4][4];               // block, column within the lane's four, MMA accumulator
  float m[R], l[R];
  uint32_t rmax[C];               // R of the block columns
  auto begin_segment = [&]() {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int32_t row = cu.rt * kRows + g + 8 * r;
      const bool real = row < cu.nq * a.group;
      const int32_t qi = real ? row / a.group : 0, hq = cu.h * a.group + (real ? row - qi * a.group : 0);
      pos[r] = cu.len - cu.nq + qi;
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + int64_t(cu.q0 + qi) * a.q_st + int64_t(hq) * a.q_sh;
      float f[C][8];
      float am = 0.0f;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        if (real) load_q8(a, src + 32 * j + 8 * tig, f[j]);
        else
#pragma unroll
          for (int i = 0; i < 8; ++i) f[j][i] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) am = max_nan(am, fabsf(f[j][i]));
      }
      am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
      am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
      // the row's largest element goes to [2^13, 2^14); rows of zeros, and
      // rows with an infinity or a NaN, are taken as they are
      const int32_t eb = int32_t(__float_as_uint(am) >> 23) & 0xFF;
      const int32_t up = (eb == 0 || eb == 255) ? 0 : min(126, 140 - eb);
      const float mul = pow2i(up);
      qf[r] = a.scale_log2 * pow2i(-up);
#pragma unroll
      for (int j = 0; j < C; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            qa[j][h][u * R + r] = f32_to_word<__half>(f[j][4 * h + 2 * u] * mul, f[j][4 * h + 2 * u + 1] * mul);
      m[r] = -INFINITY;
      l[r] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
      rmax[j] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][i][e] = 0.0f;
    }
  };
  auto end_segment = [&](bool whole, int slot) {
    const int32_t head_rows = cu.nq * a.group;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
      l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
      const int32_t row = cu.rt * kRows + g + 8 * r;
      const float inv = l[r] > 0.0f ? 1.0f / l[r] : (l[r] == 0.0f ? 0.0f : l[r]);  // a NaN sum stays NaN
      const int32_t qi = row / a.group, hq = cu.h * a.group + row - qi * a.group;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        // the accumulators hold p 2^14 v 2^(127 - R), the sum p 2^14
        const float s = pow2i(int32_t(rmax[j]) - 127) * (whole ? inv : 1.0f);
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (kSplit) {
            f[i] = (o[j][i][0] + o[j][i][2]) * s;
            f[4 + i] = (o[j][i][1] + o[j][i][3]) * s;
          } else {
            f[i] = o[j][i][2 * r] * s;
            f[4 + i] = o[j][i][2 * r + 1] * s;
          }
        }
        if (whole) {
          if (row < head_rows)
            store_o8(a,
                     static_cast<uint16_t*>(a.out) + int64_t(cu.q0 + qi) * a.o_st + int64_t(hq) * a.o_sh + 32 * j +
                         8 * tig,
                     f);
        } else {
          float4* d = reinterpret_cast<float4*>(sp.part_o + ((int64_t(worker) * 2 + slot) * kRows + g + 8 * r) * D +
                                                32 * j + 8 * tig);
          d[0] = make_float4(f[0], f[1], f[2], f[3]);
          d[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
      }
      if (tig == 0) {
        if (!whole) {
          sp.part_ml[(int64_t(worker) * 2 + slot) * kRows + g + 8 * r] = make_float2(m[r], l[r]);
        } else if (a.lse != nullptr && row < head_rows) {
          a.lse[int64_t(cu.q0 + qi) * (a.kv_heads * a.group) + hq] =
              l[r] == 0.0f ? -INFINITY : (m[r] - 14.0f + log2f(l[r])) * 0.6931471805599453f;
        }
      }
    }
  };

  bool timed_out = false;
  bool from_start = cu.t == 0;  // the segment's first tile is ours
  int part_slot = 0;            // workspace slot of a partial: 0 for the run's first segment, 1 for a later one
  begin_segment();
  int slot = 0;
  uint32_t phase = 0;
  for (int32_t n = 0; n < tiles; ++n) {
    if (!timed_out) {
      int ok = 1;
      if (lane == 0) ok = mbar_wait_bounded(&full[slot], phase, a.wait_limit_cycles, nullptr);
      if (__shfl_sync(0xFFFFFFFFu, ok, 0) == 0) {
        timed_out = true;
        if (lane == 0 && a.dev_status != nullptr) atomicExch(a.dev_status, static_cast<uint32_t>(NVFP4_ETIMEOUT));
      }
    }
    __syncwarp();
    if (timed_out) break;
    const uint32_t kc = smem_u32(codes + slot * 2 * T::kCodes), vc = kc + T::kCodes;
    const uint8_t* ks = rest + slot * 2 * T::kScales;
    const uint8_t* vs = ks + T::kScales;
    const int32_t tok0 = cu.s.tile(cu.t) * kTok;
    const int32_t lim = cu.s.hi - tok0;  // keys of the tile that some row may see: those below

    // scales: K as floats; V as FP16 factors against the running maximum
    bool nan_scale = false, new_max = false;
    float vbeta[C];
    {
      uint32_t ve[kTok / 32][C];
#pragma unroll
      for (int u = 0; u < kTok / 32; ++u) {
        const int t = lane + 32 * u;
        if constexpr (C == 2) {
          const uint16_t w = *reinterpret_cast<const uint16_t*>(ks + t * 2);
          *reinterpret_cast<float2*>(kf + t * 2) = make_float2(e8m0_value(w & 0xFF), e8m0_value(w >> 8));
          const uint16_t x = *reinterpret_cast<const uint16_t*>(vs + t * 2);
          ve[u][0] = x & 0xFF, ve[u][1] = x >> 8;
        } else {
#pragma unroll
          for (int h = 0; h < C / 4; ++h) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(ks + t * C + 4 * h);
            *reinterpret_cast<float4*>(kf + t * C + 4 * h) =
                make_float4(e8m0_value(w & 0xFF), e8m0_value((w >> 8) & 0xFF), e8m0_value((w >> 16) & 0xFF),
                            e8m0_value(w >> 24));
            const uint32_t x = *reinterpret_cast<const uint32_t*>(vs + t * C + 4 * h);
#pragma unroll
            for (int i = 0; i < 4; ++i) ve[u][4 * h + i] = (x >> (8 * i)) & 0xFF;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < C; ++j) {
        uint32_t mx = 0;
#pragma unroll
        for (int u = 0; u < kTok / 32; ++u) {
          const bool in = lane + 32 * u < lim;
          if (in && ve[u][j] == 255u) nan_scale = true;
          if (in && ve[u][j] != 255u) mx = max(mx, ve[u][j]);
        }
        mx = max(__reduce_max_sync(0xFFFFFFFFu, mx), rmax[j]);
        vbeta[j] = pow2i(int32_t(rmax[j]) - int32_t(mx));
        new_max = new_max || mx != rmax[j];
        rmax[j] = mx;
#pragma unroll
        for (int u = 0; u < kTok / 32; ++u) {
          const int t = lane + 32 * u;
          // keys that no row sees may hold any byte: factor 0
          vf[j * kTok + t] =
              uint16_t(t >= lim ? 0u : (ve[u][j] == 255u ? 0x7FFFu : half_pow2(ve[u][j], mx)));
        }
      }
      nan_scale = __any_sync(0xFFFFFFFFu, nan_scale);
      __syncwarp();
    }

    // scores
    float s[NT][2 * R];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2 * R; ++e) s[nt][e] = 0.0f;
#pragma unroll
    for (int gi = 0; gi < NT * C / 4; ++gi) {
      uint32_t w[4];
      {
        const int idx = gi * 4 + (lane >> 3);  // matrix (key tile, block) of this lane's row address
        const int t = idx / C * 8 + (lane & 7), c = idx % C;
        ldsm_x4(kc + swz<D>(t, c), w);
      }
      // block scales of this lane's two keys of each key tile of the four matrices
      constexpr int kV = C < 4 ? C : 4;
      float fk[4 / kV][2][kV];
#pragma unroll
      for (int y = 0; y < 4 / kV; ++y) {
        const int idx = gi * 4 + y * kV, nt = idx / C, j = idx % C;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float* src = kf + (nt * 8 + 2 * tig + e) * C + j;
          if constexpr (kV == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            fk[y][e][0] = v.x, fk[y][e][1] = v.y, fk[y][e][2] = v.z, fk[y][e][3] = v.w;
          } else {
            const float2 v = *reinterpret_cast<const float2*>(src);
            fk[y][e][0] = v.x, fk[y][e][1] = v.y;
          }
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int idx = gi * 4 + x, nt = idx / C, j = idx % C;
        uint32_t h[4];
        e2m1x8_to_half(w[x], h);
        float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (kSplit) {
          mma_f16(c, qa[j][0][0], 0u, qa[j][0][1], 0u, h[0], h[1]);
          mma_f16(c, qa[j][1][0], 0u, qa[j][1][1], 0u, h[2], h[3]);
        } else {
          mma_f16(c, qa[j][0][0], qa[j][0][1], qa[j][0][2], qa[j][0][3], h[0], h[1]);
          mma_f16(c, qa[j][1][0], qa[j][1][1], qa[j][1][2], qa[j][1][3], h[2], h[3]);
        }
        const float f0 = fk[x / kV][0][x % kV], f1 = fk[x / kV][1][x % kV];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          s[nt][2 * r] = fmaf(c[2 * r], f0, s[nt][2 * r]);
          s[nt][2 * r + 1] = fmaf(c[2 * r + 1], f1, s[nt][2 * r + 1]);
        }
      }
    }

    // mask, running maximum, weights
    float alpha[R];
    uint32_t ph[NT][R], pl[NT];  // weights in FP16: high parts, and the split's low parts
#pragma unroll
    for (int r = 0; r < R; ++r) {
      // is the whole tile seen by this row?
      const bool all = tok0 + kTok <= cu.len && (!a.causal || tok0 + kTok - 1 <= pos[r]) &&
                       (a.window <= 0 || tok0 > pos[r] - a.window || tok0 + kTok <= a.sinks);
      float mx = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = s[nt][2 * r + e] * qf[r];
          if (!all) {
            const int32_t j = tok0 + nt * 8 + 2 * tig + e;
            if (j >= cu.len || !sees(a, pos[r], j)) v = -INFINITY;
          }
          s[nt][2 * r + e] = v;
          mx = fmaxf(mx, v);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
      const float mn = fmaxf(m[r], mx);
      const float ms = mn == -INFINITY ? 0.0f : mn;  // no key seen yet: every weight is 2^-inf = 0
      alpha[r] = exp2_approx(m[r] - ms);
      m[r] = mn;
      float sum = 0.0f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float p0 = exp2_approx(s[nt][2 * r] - ms + 14.0f), p1 = exp2_approx(s[nt][2 * r + 1] - ms + 14.0f);
        sum += p0 + p1;
        ph[nt][r] = f32_to_word<__half>(p0, p1);
        if constexpr (kSplit) {
          const float2 h = word_to_f32<__half>(ph[nt][r]);
          pl[nt] = f32_to_word<__half>(p0 - h.x, p1 - h.y);
        }
      }
      l[r] = l[r] * alpha[r] + sum;
    }
    bool scaled = new_max;
#pragma unroll
    for (int r = 0; r < R; ++r) scaled = scaled || alpha[r] != 1.0f;
    if (__any_sync(0xFFFFFFFFu, scaled)) {
#pragma unroll
      for (int j = 0; j < C; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][i][e] *= vbeta[j] * alpha[kSplit ? 0 : e >> 1];
    }

    // output
#pragma unroll
    for (int j = 0; j < C; ++j) {
#pragma unroll
      for (int k2 = 0; k2 < KK / 2; ++k2) {
        uint32_t w[4];
        // four groups of eight keys, block j
        ldsm_x4_t(vc + swz<D>(k2 * 32 + lane, j), w);
#pragma unroll
        for (int k1 = 0; k1 < 2; ++k1) {
          const int kk = k2 * 2 + k1;
          const uint32_t fa = *reinterpret_cast<const uint32_t*>(vf + j * kTok + kk * 16 + 2 * tig);
          const uint32_t fb = *reinterpret_cast<const uint32_t*>(vf + j * kTok + kk * 16 + 8 + 2 * tig);
          uint32_t a0, a1, a2, a3;
          if constexpr (kSplit) {
            a0 = hmul2(ph[2 * kk][0], fa), a1 = hmul2(pl[2 * kk], fa);
            a2 = hmul2(ph[2 * kk + 1][0], fb), a3 = hmul2(pl[2 * kk + 1], fb);
          } else {
            a0 = hmul2(ph[2 * kk][0], fa), a1 = hmul2(ph[2 * kk][R - 1], fa);
            a2 = hmul2(ph[2 * kk + 1][0], fb), a3 = hmul2(ph[2 * kk + 1][R - 1], fb);
          }
          if (nan_scale) {
            // a NaN factor (E = 255) reaches only rows that see its key: a
            // zero weight stays zero
            auto keep0 = [](uint32_t v, uint32_t w2) {
              return ((w2 & 0x7FFFu) ? v & 0xFFFFu : 0u) | ((w2 & 0x7FFF0000u) ? v & 0xFFFF0000u : 0u);
            };
            a0 = keep0(a0, ph[2 * kk][0]), a2 = keep0(a2, ph[2 * kk + 1][0]);
            a1 = keep0(a1, kSplit ? pl[2 * kk] : ph[2 * kk][R - 1]);
            a3 = keep0(a3, kSplit ? pl[2 * kk + 1] : ph[2 * kk + 1][R - 1]);
          }
          uint32_t x[4], y[4];
          e2m1x8_to_half(w[2 * k1], x);      // (t, d0 d1) (t, d2 d3) (t+1, d0 d1) (t+1, d2 d3)
          e2m1x8_to_half(w[2 * k1 + 1], y);  // the same eight keys on
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t sel = (i & 1) ? 0x7632u : 0x5410u;
            mma_f16(o[j][i], a0, a1, a2, a3, __byte_perm(x[i >> 1], x[2 + (i >> 1)], sel),
                    __byte_perm(y[i >> 1], y[2 + (i >> 1)], sel));
          }
        }
      }
    }

    // hand the slot back: these generic reads come before the next TMA write
    fence_proxy_async_smem();
    __syncwarp();
    if (issued < tiles) {
      issue(slot);
      if (++issued < tiles) cursor_next(ld, a, kRows, kTok);
    }
    if (++slot == T::kStages) slot = 0, phase ^= 1u;

    const bool seg_end = cu.t + 1 == cu.s.n;
    if (seg_end || n + 1 == tiles) end_segment(from_start && seg_end, part_slot);
    if (n + 1 < tiles) {
      cursor_next(cu, a, kRows, kTok);
      if (seg_end) {
        from_start = true;
        part_slot = 1;
        begin_segment();
      }
    }
  }
}

// Joins the partials of the segments that more than one worker had, and
// writes the rows that see no key at all.
template <int D>
__global__ void __launch_bounds__(128) k_attn_combine(const __grid_constant__ StreamParams sp) {
  const AttnParams& a = sp.a;
  constexpr int kTok = Tile<D>::kTok;
  const int32_t h = blockIdx.x, rt = blockIdx.y, b = blockIdx.z;
  const int32_t rows = sp.rows;
  const int32_t len = a.lens[b], nq = seq_queries(a, b);
  const int32_t q0 = a.q_starts != nullptr ? a.q_starts[b] : b;
  const int32_t live = min(rows, nq * a.group - rt * rows);
  if (live <= 0) return;
  int64_t first = sp.prefix[b];
  for (int32_t r = 0; r < rt; ++r) first += int64_t(row_span(a, len, nq, r, rows, kTok).n) * a.kv_heads;
  const int32_t n = row_span(a, len, nq, rt, rows, kTok).n;
  first += int64_t(h) * n;
  const int64_t total = sp.prefix[a.seqs];
  const int32_t workers = live_workers(total, sp.workers);
  int32_t w0 = 0, w1 = -1, slot0 = 0;
  if (n > 0) {
    w0 = worker_of(total, first, workers), w1 = worker_of(total, first + n - 1, workers);
    if (w0 == w1) return;  // written by its worker
    slot0 = worker_start(total, w0, workers) == first ? 0 : 1;
  }
  for (int32_t i = threadIdx.x; i < live * (D / 8); i += blockDim.x) {
    const int32_t r = i / (D / 8), d = (i - r * (D / 8)) * 8;
    float m = -INFINITY, l = 0.0f;
    float f[8] = {};
    for (int32_t w = w0; w <= w1; ++w) {
      const float2 ml = sp.part_ml[(int64_t(w) * 2 + (w == w0 ? slot0 : 0)) * rows + r];
      if (ml.x == -INFINITY && ml.y == 0.0f) continue;  // this worker's tiles hold no key of the row
      const float mn = fmaxf(m, ml.x);
      const float ms = mn == -INFINITY ? 0.0f : mn;
      const float ca = exp2_approx(m - ms), cb = exp2_approx(ml.x - ms);
      const float4* src =
          reinterpret_cast<const float4*>(sp.part_o + ((int64_t(w) * 2 + (w == w0 ? slot0 : 0)) * rows + r) * D + d);
      const float4 u = src[0], v = src[1];
      const float in[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = f[k] * ca + in[k] * cb;
      l = l * ca + ml.y * cb;
      m = mn;
    }
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] *= inv;
    const int32_t row = rt * rows + r, qi = row / a.group, hq = h * a.group + row - qi * a.group;
    store_o8(a, static_cast<uint16_t*>(a.out) + int64_t(q0 + qi) * a.o_st + int64_t(hq) * a.o_sh + d, f);
    if (d == 0 && a.lse != nullptr)
      a.lse[int64_t(q0 + qi) * (a.kv_heads * a.group) + hq] =
          l == 0.0f ? -INFINITY : (m - 14.0f + log2f(l)) * 0.6931471805599453f;
  }
}

template <int D, bool kSplit>
nvfp4_status stream_launch(const CUtensorMap& tk, const CUtensorMap& tv, const StreamParams& sp, int row_tiles,
                           cudaStream_t stream) {
  using T = Tile<D>;
  auto kern = k_attn_stream<D, kSplit>;
  nvfp4_status st = cuda_check(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem),
                               "cudaFuncSetAttribute(k_attn_stream)");
  if (st != NVFP4_OK) return st;
  kern<<<sp.workers / kWarps, kThreads, T::kSmem, stream>>>(tk, tv, sp);
  if ((st = cuda_check(cudaGetLastError(), "launch k_attn_stream")) != NVFP4_OK) return st;
  k_attn_combine<D><<<dim3(unsigned(sp.a.kv_heads), unsigned(row_tiles), unsigned(sp.a.seqs)), 128, 0, stream>>>(sp);
  return cuda_check(cudaGetLastError(), "launch k_attn_combine");
}

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }
int stream_workers() { return 2 * sm_count() * kWarps; }

}  // namespace

int64_t attn_stream_workspace(int32_t dim) {
  const int64_t slots = 2 * int64_t(stream_workers());
  return align256(slots * 16 * dim * 4) + align256(slots * 16 * 8) + align256((kMaxSeqs + 1) * 8);
}

nvfp4_status attn_stream(const mxfp4_cache* cache, const AttnParams& base, int32_t max_queries, void* workspace,
                         cudaStream_t stream) {
  const int32_t dim = cache->dim;
  CUtensorMap tk, tv;
  const int box = std::min(cache->page_size, dim == 256 ? 32 : 64);
  const cuuint64_t dims[3] = {cuuint64_t(dim / 2), cuuint64_t(cache->page_size),
                              cuuint64_t(cache->pages * cache->kv_heads)};
  const cuuint64_t strides[2] = {cuuint64_t(dim / 2), cuuint64_t(dim / 2) * cuuint64_t(cache->page_size)};
  const cuuint32_t bx[3] = {cuuint32_t(dim / 2), cuuint32_t(box), 1};
  const CUtensorMapSwizzle swz = dim == 64    ? CU_TENSOR_MAP_SWIZZLE_32B
                                 : dim == 128 ? CU_TENSOR_MAP_SWIZZLE_64B
                                              : CU_TENSOR_MAP_SWIZZLE_128B;
  nvfp4_status st = make_map(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, cache->k_codes, 3, dims, strides, bx, swz, "K codes");
  if (st == NVFP4_OK)
    st = make_map(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, cache->v_codes, 3, dims, strides, bx, swz, "V codes");
  if (st != NVFP4_OK) return st;
  StreamParams sp;
  sp.a = base;
  sp.workers = stream_workers();
  const int64_t rows_max = int64_t(max_queries) * base.group;
  const bool split = rows_max <= 8;
  sp.rows = split ? 8 : 16;
  const int64_t slots = 2 * int64_t(sp.workers);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  sp.part_o = reinterpret_cast<float*>(ws);
  sp.part_ml = reinterpret_cast<float2*>(ws + align256(slots * 16 * dim * 4));
  sp.prefix = reinterpret_cast<int64_t*>(ws + align256(slots * 16 * dim * 4) + align256(slots * 16 * 8));
  const int64_t row_tiles = (rows_max + sp.rows - 1) / sp.rows;
  if (row_tiles > 65535) return fail(NVFP4_EUNSUPPORTED, "mxfp4_cache_attention: too many query rows a sequence");
  // kMaxSeqs sequences a launch; the workspace is reused in stream order
  for (int32_t b = 0; b < base.seqs; b += kMaxSeqs) {
    sp.a.seqs = std::min(kMaxSeqs, base.seqs - b);
    sp.a.table = base.table + int64_t(b) * base.table_ld;
    sp.a.lens = base.lens + b;
    if (base.q_starts != nullptr) {
      sp.a.q_starts = base.q_starts + b;
    } else {
      sp.a.q = static_cast<const uint16_t*>(base.q) + int64_t(b) * base.q_st;
      sp.a.out = static_cast<uint16_t*>(base.out) + int64_t(b) * base.o_st;
      if (base.lse != nullptr) sp.a.lse = base.lse + int64_t(b) * base.kv_heads * base.group;
    }
    if (dim == 64) st = split ? stream_launch<64, true>(tk, tv, sp, int(row_tiles), stream)
                              : stream_launch<64, false>(tk, tv, sp, int(row_tiles), stream);
    else if (dim == 128) st = split ? stream_launch<128, true>(tk, tv, sp, int(row_tiles), stream)
                                    : stream_launch<128, false>(tk, tv, sp, int(row_tiles), stream);
    else st = split ? stream_launch<256, true>(tk, tv, sp, int(row_tiles), stream)
                    : stream_launch<256, false>(tk, tv, sp, int(row_tiles), stream);
    if (st != NVFP4_OK) return st;
  }
  return NVFP4_OK;
}

}  // namespace nvfp4
