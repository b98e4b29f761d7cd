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
//   softmax   sum in FP32 against a reference that follows the running
//             maximum once it is 2^5 behind, so that the output is rarely
//             rescaled; weights p 2^10 <= 2^15 rounded to FP16 for the second
//             MMA (11 bits; BF16 would keep 8).
//   p v       a value's block scale varies along the contraction, so it goes
//             onto the weights: p 2^10 2^(E - R) with R the largest E of the
//             block column so far (a running maximum like the softmax's).  The
//             factor 2^10 leaves 24 binades below the reference before FP16
//             loses bits.
//
// The decoding cvt gives two neighbours (d, d + 1) of one token, while an MMA
// contracts over pairs of tokens.  Up to 8 rows (kRows = 8, every decoding
// step of 8 heads a kv head) need no transposition for that: the contraction
// pair is (d, d + 1), MMA row g holds (p, 0) and row g + 8, idle otherwise,
// (0, p), so that rows 0..7 collect the even and rows 8..15 the odd columns.
// In q k^T their rows 8..15 hold the other half of the block, and each of a
// block's two MMAs gives its result in one half of the rows.
// With 16 rows the halves are put together by PRMT, one for each register.
// The ldmatrix layouts fit the format: a 16-byte row of an 8x8 matrix is one
// block of one token, so for K a lane gets 8 codes of one block, and with
// .trans for V it gets 4 codes of token t in its low and of token t + 1 in
// its high half.
//
// Work is dealt over all warps of the grid as SplitParams describes.
//
// What bounds it: latency.  Three warps a scheduler issue in 48% of the cycles, no
// pipe is above 37% and DRAM at 42%; each works through the chain ldmatrix, cvt,
// MMA, FMA, ex2, cvt, MMA of 32 keys at a time, and more warps do not fit beside Q,
// the scores and the output in registers.  32 conversations of 257 to 32,767 keys,
// 8 rows of 8 heads, dim 128 (246 MB): 73 us, 3.4 TB/s; with the join 82 us.  Three
// blocks an SM at 168 registers are 5 to 17% faster than two at 231, although a few
// registers spill.
#include <algorithm>
#include <atomic>
#include <string>

#include "mx_attn.cuh"

namespace nvfp4 {

nvfp4_status make_map(CUtensorMap* map, CUtensorMapDataType dt, const void* base, int rank, const cuuint64_t* dims,
                      const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle, const char* what);

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

// The largest values that only some rows see may be this far above those that
// all see: a row's weights down to 2^-27 are then kept by the FP16 of their factor.
constexpr int kSpreadV = 8;

// A stage of the ring holds kTok keys, worked off kSub at a time.  kSeveral: a
// sequence may have several queries, so that rows may see different keys.
template <int D, int kRows, bool kSeveral>
struct Tile {
  static constexpr int C = D / 32;  // blocks of a row
  static constexpr int kTok = D == 256 ? 32 : (D == 128 ? 64 : 128);
  static constexpr int kSub = 32;  // (dim 64 by 64: 7% slower, registers spill)
  static constexpr int kCodes = kTok * D / 2;  // bytes of K (or V) codes
  static constexpr int kScales = kTok * C;
  static constexpr int kCtas = (kRows == 8 && D <= 128) ? 3 : 2;  // blocks an SM
  static constexpr int kStages = kCtas == 3 ? 2 : 3;
  static constexpr int kKf = kSub * C * 4;  // K scales as float [position][C]
  // V factors: (f, f) [position][C] for 8 rows, f [position pair][C][2] for 16
  static constexpr int kVf = kSub * C * (kRows == 8 ? 4 : 2);
  static constexpr int kWarpCodes = kStages * 2 * kCodes;
  static constexpr int kWarpRest = kStages * 2 * kScales + kKf + kVf;
  // [warp codes x 4][warp rest x 4][barriers]; the tile counts of the
  // sequences lie where the codes go, before the first load
  static constexpr int kBars = kWarps * kStages * 8;
  static constexpr int kSmem = kWarps * (kWarpCodes + kWarpRest + (kSeveral ? int(sizeof(Cursor)) : 0)) + kBars;
  static_assert((kMaxSeqs + 1 + kThreads) * 8 <= kWarps * kWarpCodes, "tile counts");
  static_assert(kCodes % 1024 == 0, "swizzle atoms");
  static_assert(kCtas * (kSmem + 1024) <= 233472, "blocks an SM");
};

constexpr float kLag = 5.0f;          // the softmax reference may lag the maximum by 2^5

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
// The same with a zero accumulator.
__device__ __forceinline__ void mma_f16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A tile lies in shared memory as rows of 128 bytes, P = 256 / D tokens each,
// under the TMA's 128-byte swizzle.  An 8x8 matrix takes the same part of
// eight consecutive rows, which the swizzle spreads over all banks: its
// columns are tokens P apart.  Position pos = 8 nt + column of the MMAs is
// token token_of(pos) of the tile.
template <int D>
__device__ __forceinline__ int token_of(int pos) {
  constexpr int P = 256 / D;
  const int nt = pos >> 3;
  return nt / P * (8 * P) + (pos & 7) * P + nt % P;
}
// Byte offset of 16-byte chunk (block) c of the token at pos.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int pos, int c) {
  constexpr int P = 256 / D, C = D / 32;
  const int nt = pos >> 3, row = nt / P * 8 + (pos & 7);
  return uint32_t(row * 128 + (((nt % P * C + c) ^ (row & 7)) << 4));
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
// Scale word of a block in the high exponent bits: 2^(E-127) for 1 <= E <= 254,
// 0 for E = 0 (a block below 2^-124 has no weight in a score), NaN for 255, where
// the exponent and 1 carry into the sign bit.
__device__ __forceinline__ float e8m0_byte(uint32_t w, int i) {
  const uint32_t v = (i == 0 ? w << 23 : (i == 1 ? w << 15 : (i == 2 ? w << 7 : w >> 1))) & 0x7F800000u;
  return __uint_as_float(v | (v + 0x00800000u) >> 31);
}

// Keys that only some rows see, after a warp's run.  Not inlined: the loops of the
// kernel are not to make room for it.
template <int D, int kRows>
__device__ __noinline__ void check_run(const SplitParams& sp, const Cursor* start, int32_t tiles, int32_t worker) {
  constexpr int kTok = Tile<D, kRows, true>::kTok;
  walk_run<kRows>(sp, *start, tiles, worker, kTok, [&](const Cursor& c, int32_t n, int64_t part) {
    if (too_wide<D, kRows>(sp.a, c, n, kTok, kSpreadV, 0)) wide_segment<D, kRows, false>(sp, c, n, part, kTok, 0, 1);
  });
}

// kFew: up to 32 sequences, which each warp counts for itself.  (A branch instead of a
// variant: the tiles' loop is compiled differently, and 192 sequences take 1 us more.)
// kF32: see store_o8.  16 rows have a variant for each type of the output (a branch: 4
// sequences of 2 queries of 8 heads, dim 128, 16.8 us instead of 15.9, 64 of 8 queries
// 68.8 instead of 65.6); 8 rows branch (variants: up to 2% slower, or the same).
template <int D, int kRows, bool kSeveral, bool kFew, int kF32>
__global__ void __launch_bounds__(kThreads, Tile<D, kRows, kSeveral>::kCtas)
    k_attn_stream(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                  const __grid_constant__ SplitParams sp) {
  using T = Tile<D, kRows, kSeveral>;
  constexpr int C = T::C, kTok = T::kTok, kSub = T::kSub, NT = kSub / 8;
  constexpr int R = kRows / 8;   // rows of a thread: g, and g + 8
  constexpr int Y = 2 * R;       // accumulators of a block: 8 rows hold two columns in each
  constexpr int U = kSub / 32;   // keys of a lane in the scale work
  const AttnParams& a = sp.a;
  extern __shared__ __align__(1024) uint8_t base[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  uint8_t* codes = base + warp * T::kWarpCodes;
  uint8_t* rest = base + kWarps * T::kWarpCodes + warp * T::kWarpRest;
  float* kf = reinterpret_cast<float*>(rest + T::kStages * 2 * T::kScales);
  uint8_t* vf = rest + T::kStages * 2 * T::kScales + T::kKf;
  uint8_t* tail = base + kWarps * (T::kWarpCodes + T::kWarpRest);
  uint64_t* full = reinterpret_cast<uint64_t*>(tail) + warp * T::kStages;
  Cursor* start = reinterpret_cast<Cursor*>(tail + T::kBars) + warp;  // of this warp's run
  int64_t* prefix = reinterpret_cast<int64_t*>(base);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kWarps * T::kStages; ++i) mbar_init(reinterpret_cast<uint64_t*>(tail) + i, 1);
    fence_barrier_init();
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  grid_wait();
  WarpCounts counts;
  int64_t total;
  if constexpr (kFew) {
    counts = warp_counts(sp, kRows, kTok, 1);
    total = all_places(counts);
  } else {
    tile_counts<kThreads>(sp, prefix, kRows, kTok);
    total = prefix[a.seqs];
  }
  // the first workers lie in different blocks: few tiles spread over all SMs
  const int32_t worker = warp * int32_t(gridDim.x) + int32_t(blockIdx.x);
  const int32_t workers = live_workers(sp, total);
  const int64_t x0 = worker < workers ? worker_start(total, worker, workers) : 0;
  const int32_t tiles = worker < workers ? int32_t(worker_start(total, worker + 1, workers) - x0) : 0;
  Cursor cu;
  if constexpr (kFew) {
    if (tiles > 0) cursor_at(cu, a, counts, x0, kRows, kTok, 0);
    if (worker == 0) leave_places(sp, counts);
  } else {
    if (tiles > 0) cursor_at(cu, a, prefix, x0, kRows, kTok, 0);
    fence_proxy_async_smem();  // the counts are read, the TMA may write there
  }
  __syncthreads();
  if (tiles <= 0) return;
  if (kSeveral && lane == 0) *start = cu;
  if (sp.start != nullptr && lane == 0) sp.start[worker] = cu;

  // ---- loads: lane i < boxes takes box i of a tile (a page's share of it);
  // its page is looked up when the tile before is issued
  const int32_t box_shift = min(a.page_shift, kTok == 32 ? 5 : (kTok == 64 ? 6 : 7));
  const int32_t box = 1 << box_shift, boxes = kTok >> box_shift;
  Cursor ld = cu;
  int32_t page;
  auto look_up = [&]() {
    const int32_t tok = ld.s.tile(ld.t) * kTok + (lane << box_shift);
    page = 0;
    if (lane < boxes && tok < ld.len)
      page = a.table[int64_t(ld.b) * a.table_ld + min(tok >> a.page_shift, int32_t(a.table_ld) - 1)];
  };
  auto issue = [&](int slot) {
    const int32_t tok0 = ld.s.tile(ld.t) * kTok;
    const int32_t nb = min(boxes, (ld.len - tok0 + box - 1) >> box_shift);  // boxes that hold a token
    if (lane == 0) mbar_arrive_expect_tx(&full[slot], uint32_t(nb << box_shift) * (D + 2 * C));
    __syncwarp();
    if (lane < nb) {
      uint8_t* st = codes + slot * 2 * T::kCodes + (lane << box_shift) * (D / 2);
      uint8_t* sc = rest + slot * 2 * T::kScales + (lane << box_shift) * C;
      const int32_t pg = min(max(page, 0), int32_t(a.pages) - 1);
      const int32_t z = pg * a.kv_heads + ld.h, off = (tok0 + (lane << box_shift)) & ((1 << a.page_shift) - 1);
      tma_load_3d_plain(st, &tmap_k, &full[slot], 0, off / (256 / D), z);
      tma_load_3d_plain(st + T::kCodes, &tmap_v, &full[slot], 0, off / (256 / D), z);
      const int64_t srow = ((int64_t(z) << a.page_shift) + off) * C;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv)
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         smem_u32(sc + kv * T::kScales)),
                     "l"((kv ? a.v_scales : a.k_scales) + srow), "r"(C << box_shift), "r"(smem_u32(&full[slot]))
                     : "memory");
    }
  };
  int32_t issued = 0;
  look_up();
#pragma unroll 1
  while (issued < min(T::kStages, tiles)) {
    issue(issued);
    if (++issued < tiles) {
      cursor_next(ld, a, kRows, kTok);
      look_up();
    }
  }

  // ---- state of the segment
  uint32_t qa[C][2][2 * R];  // Q fragments: block, MMA of the block
  float qf[R];               // row factor of the scores (log2 domain)
  // the row sees keys j < end with j >= from or j < a.sinks
  int32_t end[R], from[R];
  float o[C][Y][4];  // block, MMA of the block, accumulator
  float m[R], l[R];  // softmax reference; sum of this lane's weights, times 2^10
  int32_t rmax[C];   // R of the block columns
  // kSeveral only
  Common rows;         // keys that all rows see
  Spread spread;       // of block column `lane`
  bool lag = false;    // some are open
  bool check = false;  // of the whole run
  auto begin_segment = [&]() {
    if constexpr (kSeveral) {
      rows = common_of(a, cu.len, cu.nq, cu.rt, kRows);
      spread.reset();
      lag = false;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int32_t row = cu.rt * kRows + g + 8 * r;
      const bool real = row < cu.nq * a.group;
      const int32_t qi = real ? row / a.group : 0, hq = cu.h * a.group + (real ? row - qi * a.group : 0);
      const int32_t pos = cu.len - cu.nq + qi;
      end[r] = a.causal ? min(cu.len, pos + 1) : cu.len;
      from[r] = a.window > 0 ? pos - a.window + 1 : 0;
      const uint16_t* src =
          static_cast<const uint16_t*>(a.q) + query_row(a, cu.q0 + qi) * a.q_st + int64_t(hq) * a.q_sh;
      float am = 0.0f;
#pragma unroll
      for (int pass = 0; pass < 2; ++pass) {  // the row's largest element, then its fragments
        float mul = 1.0f;
        if (pass == 1) {
          am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
          am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
          // the row's largest element goes to [2^13, 2^14); rows of zeros, and
          // rows with an infinity or a NaN, are taken as they are
          const int32_t eb = int32_t(__float_as_uint(am) >> 23) & 0xFF;
          const int32_t up = (eb == 0 || eb == 255) ? 0 : min(126, 140 - eb);
          mul = pow2i(up);
          qf[r] = a.scale_log2 * pow2i(-up);
        }
#pragma unroll
        for (int j = 0; j < C; ++j) {
          float f[8] = {};
          if (real) load_q8(a, src + 32 * j + 8 * tig, f);
          if (pass == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) am = max_nan(am, fabsf(f[i]));
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int u = 0; u < 2; ++u)
                qa[j][h][u * R + r] = f32_to_word<__half>(f[4 * h + 2 * u] * mul, f[4 * h + 2 * u + 1] * mul);
          }
        }
      }
      m[r] = -INFINITY;
      l[r] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
      rmax[j] = 0;
#pragma unroll
      for (int y = 0; y < Y; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][y][e] = 0.0f;
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
      const int32_t pe = part_exponent(l[r]);
      const float fac = whole ? inv : pow2i(-pe);
#pragma unroll
      for (int j = 0; j < C; ++j) {
        // the accumulators hold p 2^10 v 2^(127 - R), the sum p 2^10
        const float s = pow2i(rmax[j] - 127) * fac;
        float f[8];  // columns 32 j + 8 tig + 0 .. 7
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // column n = 2 tig (or 2 tig + 1) of an MMA is code group n of the
          // block: columns 4 n .. 4 n + 3
          f[i] = (kRows == 8 ? o[j][i >> 1][2 * (i & 1)] : o[j][i % Y][2 * r]) * s;
          f[4 + i] = (kRows == 8 ? o[j][i >> 1][2 * (i & 1) + 1] : o[j][i % Y][2 * r + 1]) * s;
        }
        if (whole) {
          if (row < head_rows)
            store_o8<kF32>(a, int64_t(cu.q0 + qi) * a.o_st + int64_t(hq) * a.o_sh + 32 * j + 8 * tig, f);
        } else {
          float4* d = reinterpret_cast<float4*>(sp.part_o + ((int64_t(worker) * 2 + slot) * kRows + g + 8 * r) * D +
                                                32 * j + 8 * tig);
          d[0] = make_float4(f[0], f[1], f[2], f[3]);
          d[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
      }
      if (tig == 0) {
        if (!whole) {
          sp.part_ml[(int64_t(worker) * 2 + slot) * kRows + g + 8 * r] =
              make_float2(m[r] + float(pe), l[r] * pow2i(-pe));
        } else if (a.lse != nullptr && row < head_rows) {
          a.lse[int64_t(cu.q0 + qi) * (a.kv_heads * a.group) + hq] =
              l[r] == 0.0f ? -INFINITY : (m[r] - kWeightLog2 + log2f(l[r])) * 0.6931471805599453f;
        }
      }
    }
  };

  // kSub keys from smem: `sub` of the stage at codes kc, vc, scales ks, vs
  auto work = [&](uint32_t kc, uint32_t vc, const uint8_t* ks, const uint8_t* vs, int32_t tok0) {
    // do all rows see all these keys?
    const bool all = kSeveral ? all_see(a, rows, tok0, kSub)
                              : tok0 + kSub <= end[0] && (tok0 >= from[0] || tok0 + kSub <= a.sinks);
    uint32_t nan_keys[U][C] = {};        // keys whose block holds NaN (E = 255)
    bool nan_scale = false;
    // scales: K as floats; V as FP16 factors against the running maximum
    {
      int32_t e[U][C];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int pos = lane + 32 * u, t = token_of<D>(pos);
        if constexpr (C == 2) {
          const uint32_t kw = *reinterpret_cast<const uint16_t*>(ks + t * 2);
          uint32_t vw = *reinterpret_cast<const uint16_t*>(vs + t * 2);
          if (!cu.s.has(a, tok0 + t)) vw = 0;  // no row sees it: no factor, no reference, no NaN
          *reinterpret_cast<float2*>(kf + pos * 2) = make_float2(e8m0_byte(kw, 0), e8m0_byte(kw, 1));
          e[u][0] = vw & 0xFF, e[u][1] = vw >> 8;
        } else {
#pragma unroll
          for (int h = 0; h < C / 4; ++h) {
            const uint32_t kw = *reinterpret_cast<const uint32_t*>(ks + t * C + 4 * h);
            uint32_t vw = *reinterpret_cast<const uint32_t*>(vs + t * C + 4 * h);
            if (!cu.s.has(a, tok0 + t)) vw = 0;
            *reinterpret_cast<float4*>(kf + pos * C + 4 * h) =
                make_float4(e8m0_byte(kw, 0), e8m0_byte(kw, 1), e8m0_byte(kw, 2), e8m0_byte(kw, 3));
#pragma unroll
            for (int i = 0; i < 4; ++i) e[u][(4 * h + i) % C] = (vw >> (8 * i)) & 0xFF;
          }
        }
      }
      if (kSeveral && (!all || lag) && !rows.one) {
        int32_t top = 0, low = 255, old = 0;
#pragma unroll
        for (int j = 0; j < C; ++j) {
          int32_t hi = 0, lo = 255;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            hi = max(hi, e[u][j] == 255 ? 0 : e[u][j]);
            if (e[u][j] > 0) lo = min(lo, e[u][j]);
          }
          hi = __reduce_max_sync(0xFFFFFFFFu, hi), lo = __reduce_min_sync(0xFFFFFFFFu, lo);
          if (lane == j) top = hi, low = lo, old = rmax[j];
        }
        const bool fine = all ? spread.all_see(old, top, kSpreadV) : spread.some_see(old, top, low, kSpreadV);
        check = check || __any_sync(0xFFFFFFFFu, !fine);
        lag = __any_sync(0xFFFFFFFFu, spread.open());
      }
      bool up = false;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < C; ++j) up = up || e[u][j] > rmax[j];
      if (__any_sync(0xFFFFFFFFu, up)) {
#pragma unroll
        for (int j = 0; j < C; ++j) {
          int32_t mx = 0;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            nan_keys[u][j] = __ballot_sync(0xFFFFFFFFu, e[u][j] == 255);
            nan_scale = nan_scale || nan_keys[u][j] != 0;
            if (e[u][j] == 255) e[u][j] = 0;
            mx = max(mx, e[u][j]);
          }
          mx = max(__reduce_max_sync(0xFFFFFFFFu, mx), rmax[j]);
          const float beta = pow2i(rmax[j] - mx);
          rmax[j] = mx;
#pragma unroll
          for (int y = 0; y < Y; ++y)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[j][y][i] *= beta;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int pos = lane + 32 * u;
        uint32_t w[C];
#pragma unroll
        for (int j = 0; j < C; ++j) {
          // 2^(E - R) through binary32, rounded (to a subnormal, to zero) by the conversion
          const float f = __uint_as_float(uint32_t(max(e[u][j] - rmax[j] + 127, 0)) << 23);
          w[j] = f32_to_word<__half>(f, f);
          if constexpr (kRows == 16) reinterpret_cast<uint16_t*>(vf)[(pos / 2 * C + j) * 2 + pos % 2] = uint16_t(w[j]);
        }
        if constexpr (kRows == 8) {
          if constexpr (C == 2) {
            *reinterpret_cast<uint2*>(vf + pos * 8) = make_uint2(w[0], w[1]);
          } else {
#pragma unroll
            for (int h = 0; h < C / 4; ++h)
              *reinterpret_cast<uint4*>(vf + pos * C * 4 + h * 16) =
                  make_uint4(w[(4 * h) % C], w[(4 * h + 1) % C], w[(4 * h + 2) % C], w[(4 * h + 3) % C]);
          }
        }
      }
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
        const int idx = gi * 4 + (lane >> 3);  // matrix (key group, block) of this lane's row address
        ldsm_x4(kc + chunk_at<D>(idx / C * 8 + (lane & 7), idx % C), w);
      }
      // block scales of this lane's two keys of each key group of the four matrices
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
        const float f0 = fk[x / kV][0][x % kV], f1 = fk[x / kV][1][x % kV];
        float c[4];
        if constexpr (kRows == 8) {
          // rows 0..7 hold the block's first, rows 8..15 its second half
          float d[4];
          mma_f16_zero(c, qa[j][0][0], qa[j][1][0], qa[j][0][1], qa[j][1][1], h[0], h[1]);
          mma_f16_zero(d, qa[j][0][0], qa[j][1][0], qa[j][0][1], qa[j][1][1], h[2], h[3]);
          s[nt][0] = fmaf(c[0], f0, s[nt][0]);
          s[nt][1] = fmaf(c[1], f1, s[nt][1]);
          s[nt][0] = fmaf(d[2], f0, s[nt][0]);
          s[nt][1] = fmaf(d[3], f1, s[nt][1]);
        } else {
          mma_f16_zero(c, qa[j][0][0], qa[j][0][1], qa[j][0][2 % (2 * R)], qa[j][0][3 % (2 * R)], h[0], h[1]);
          mma_f16(c, qa[j][1][0], qa[j][1][1], qa[j][1][2 % (2 * R)], qa[j][1][3 % (2 * R)], h[2], h[3]);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            s[nt][2 * r] = fmaf(c[2 * r], f0, s[nt][2 * r]);
            s[nt][2 * r + 1] = fmaf(c[2 * r + 1], f1, s[nt][2 * r + 1]);
          }
        }
      }
    }

    // mask, reference, weights
    // 8 rows: words (p, 0) of the lane's two keys; 16 rows: pairs of the two keys
    uint32_t pw[NT][2];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) s[nt][2 * r + e] *= qf[r];
    if (!all) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int32_t j = tok0 + token_of<D>(nt * 8 + 2 * tig + e);
            if (j >= end[r] || (j < from[r] && j >= a.sinks)) s[nt][2 * r + e] = -INFINITY;
          }
    }
    float mx[R];
    bool raise = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mx[r] = fmaxf(s[0][2 * r], s[0][2 * r + 1]);
#pragma unroll
      for (int nt = 1; nt < NT; ++nt) mx[r] = fmaxf(mx[r], fmaxf(s[nt][2 * r], s[nt][2 * r + 1]));
      raise = raise || mx[r] > m[r] + kLag;
    }
    if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xFFFFFFFFu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xFFFFFFFFu, mx[r], 2));
        mx[r] = fmaxf(mx[r], m[r]);
        const float alpha = exp2_approx(m[r] - (mx[r] == -INFINITY ? 0.0f : mx[r]));
        m[r] = mx[r];
        l[r] *= alpha;
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
          for (int y = 0; y < Y; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (kRows == 8 || (e >> 1) == r) o[j][y][e] *= alpha;
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float ms = (m[r] == -INFINITY ? 0.0f : m[r]) - kWeightLog2;  // no key seen yet: every weight is 2^-inf = 0
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float p0 = exp2_approx(s[nt][2 * r] - ms), p1 = exp2_approx(s[nt][2 * r + 1] - ms);
        l[r] += p0 + p1;
        if constexpr (kRows == 8) {
          pw[nt][0] = f32_to_word<__half>(p0, 0.0f);
          pw[nt][1] = f32_to_word<__half>(p1, 0.0f);
        } else {
          pw[nt][r] = f32_to_word<__half>(p0, p1);
        }
      }
    }

    // a block of NaN reaches the rows that see its key, whatever its weight (0 times
    // NaN), and only those
    if (nan_scale) {
#pragma unroll
      for (int j = 0; j < C; ++j) {
        bool hit[R] = {};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bool bad = (nan_keys[nt / 4][j] >> ((nt % 4) * 8 + 2 * tig + e)) & 1u;
            const int32_t key = tok0 + token_of<D>(nt * 8 + 2 * tig + e);
#pragma unroll
            for (int r = 0; r < R; ++r)
              hit[r] = hit[r] || (bad && key < end[r] && (key >= from[r] || key < a.sinks));
          }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const uint32_t row_hits = __ballot_sync(0xFFFFFFFFu, hit[r]) >> (lane & ~3) & 0xFu;
          if (row_hits != 0) {
#pragma unroll
            for (int y = 0; y < Y; ++y)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (kRows == 8 || (e >> 1) == r) o[j][y][e] = __uint_as_float(0x7FFFFFFFu);
          }
        }
      }
      __syncwarp();  // the MMAs are by the whole warp
    }

    // output
    if constexpr (kRows == 8) {
#pragma unroll
      for (int gi = 0; gi < NT * C / 4; ++gi) {
        uint32_t w[4];
        {
          const int idx = gi * 4 + (lane >> 3);
          ldsm_x4_t(vc + chunk_at<D>(idx / C * 8 + (lane & 7), idx % C), w);
        }
        constexpr int kV = C < 4 ? C : 4;
        uint32_t f[4 / kV][2][kV];  // factors of the lane's two keys
#pragma unroll
        for (int y = 0; y < 4 / kV; ++y) {
          const int idx = gi * 4 + y * kV, nt = idx / C, j = idx % C;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint8_t* src = vf + ((nt * 8 + 2 * tig + e) * C + j) * 4;
            if constexpr (kV == 4) {
              const uint4 v = *reinterpret_cast<const uint4*>(src);
              f[y][e][0] = v.x, f[y][e][1] = v.y, f[y][e][2] = v.z, f[y][e][3] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(src);
              f[y][e][0] = v.x, f[y][e][1] = v.y;
            }
          }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int idx = gi * 4 + x, nt = idx / C, j = idx % C;
          const uint32_t f0 = f[x / kV][0][x % kV], f1 = f[x / kV][1][x % kV];
          const uint32_t a0 = hmul2(pw[nt][0], f0), a1 = hmul2(pw[nt][0] << 16, f0);
          const uint32_t a2 = hmul2(pw[nt][1], f1), a3 = hmul2(pw[nt][1] << 16, f1);
          uint32_t v[4];
          e2m1x8_to_half(w[x], v);  // (t, d0 d1) (t, d2 d3) (t', d0 d1) (t', d2 d3)
          mma_f16(o[j][0], a0, a1, a2, a3, v[0], v[2]);
          mma_f16(o[j][1], a0, a1, a2, a3, v[1], v[3]);
        }
      }
    } else {
#pragma unroll
      for (int n2 = 0; n2 < NT / 2; ++n2) {  // sixteen keys: groups 2 n2 and 2 n2 + 1
#pragma unroll
        for (int j2 = 0; j2 < C / 2; ++j2) {  // two blocks
          uint32_t w[4];  // (group, block): (0, 0) (1, 0) (0, 1) (1, 1)
          ldsm_x4_t(vc + chunk_at<D>((n2 * 2 + ((lane >> 3) & 1)) * 8 + (lane & 7), j2 * 2 + (lane >> 4)), w);
#pragma unroll
          for (int jj = 0; jj < 2; ++jj) {
            const int j = j2 * 2 + jj, nt = n2 * 2;
            const uint32_t fa = *reinterpret_cast<const uint32_t*>(vf + 4 * ((nt * 4 + tig) * C + j));
            const uint32_t fb = *reinterpret_cast<const uint32_t*>(vf + 4 * ((nt * 4 + 4 + tig) * C + j));
            const uint32_t a0 = hmul2(pw[nt][0], fa), a1 = hmul2(pw[nt][1], fa);
            const uint32_t a2 = hmul2(pw[nt + 1][0], fb), a3 = hmul2(pw[nt + 1][1], fb);
            uint32_t x[4], y[4];
            e2m1x8_to_half(w[2 * jj], x);
            e2m1x8_to_half(w[2 * jj + 1], y);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t sel = (i & 1) ? 0x7632u : 0x5410u;
              mma_f16(o[j][i % Y], a0, a1, a2, a3, __byte_perm(x[i >> 1], x[2 + (i >> 1)], sel),
                      __byte_perm(y[i >> 1], y[2 + (i >> 1)], sel));
            }
          }
        }
      }
    }
    __syncwarp();  // before the factors are overwritten
  };

  bool from_start = cu.t == 0;  // the segment's first tile is ours
  int part_slot = 0;            // workspace slot of a partial: 0 for the run's first segment, 1 for a later one
  bool fresh = true;
  int slot = 0;
  uint32_t phase = 0;
#pragma unroll 1
  for (int32_t n = 0; n < tiles; ++n) {
    if (fresh) begin_segment();
    {
      int ok = 1;
      if (lane == 0) ok = mbar_wait_bounded(&full[slot], phase, a.wait_limit_cycles, nullptr);
      if (__shfl_sync(0xFFFFFFFFu, ok, 0) == 0) {
        if (lane == 0 && a.dev_status != nullptr) atomicExch(a.dev_status, static_cast<uint32_t>(NVFP4_ETIMEOUT));
        // the warp's later copies may still land in the block's shared memory
        for (++n; n < issued; ++n) {
          if (++slot == T::kStages) slot = 0, phase ^= 1u;
          mbar_wait_bounded(&full[slot], phase, a.wait_limit_cycles, nullptr);
        }
        return;
      }
    }
    {
      uint32_t kc = smem_u32(codes + slot * 2 * T::kCodes);
      const uint8_t* ks = rest + slot * 2 * T::kScales;
      const int32_t first = cu.s.tile(cu.t) * kTok;
      const int32_t last = min(first + kTok, cu.s.hi);
#pragma unroll 1
      for (int32_t tok0 = first; tok0 < last; tok0 += T::kSub) {
        work(kc, kc + T::kCodes, ks, ks + T::kScales, tok0);
        kc += T::kSub * (D / 2);
        ks += T::kSub * C;
      }
    }
    // hand the slot back: these generic reads come before the next TMA write
    fence_proxy_async_smem();
    __syncwarp();
    if (issued < tiles) {
      issue(slot);
      if (++issued < tiles) {
        cursor_next(ld, a, kRows, kTok);
        look_up();
      }
    }
    if (++slot == T::kStages) slot = 0, phase ^= 1u;

    fresh = cu.t + 1 == cu.s.n;
    if (fresh || n + 1 == tiles) end_segment(from_start && fresh, part_slot);
    if (n + 1 < tiles) {
      cursor_next(cu, a, kRows, kTok);
      if (fresh) from_start = true, part_slot = 1;
    }
  }
  if (kSeveral && check) {
    __syncwarp();
    check_run<D, kRows>(sp, start, tiles, worker);
  }
}

// From so many segments on (sequences times kv heads times row tiles) partials are joined
// by boundaries between runs (k_attn_combine_boundaries), below by segments: 1,024 of 8
// rows, and twice as many of 16, which have twice the rows to join.  8 heads of 128,
// sequences of 32 to 1,025 keys, by boundaries / segments: 32 of them 20.5 / 20.3 us,
// 128 36.7 / 41.0, 512 110 / 131; with one of 20,000 keys among them 34.0 / 29.7,
// 50.0 / 50.4, 110 / 131: a long one has many partials, for which a block is better.
// 4 heads, 16 rows: 256 of them 73.0 / 71.7, 512 122 / 124.
constexpr int64_t kManySegments = 1024;

template <int D, int kRows, bool kSeveral, bool kFew = false, int kF32 = -1>
nvfp4_status stream_launch(const CUtensorMap& tk, const CUtensorMap& tv, Pending& w, cudaStream_t stream) {
  using T = Tile<D, kRows, kSeveral>;
  auto kern = k_attn_stream<D, kRows, kSeveral, kFew, kF32>;
  static std::atomic<uint64_t> ready{0};  // devices whose attribute is set
  nvfp4_status st = allow_smem(reinterpret_cast<const void*>(kern), T::kSmem, ready);
  if (st != NVFP4_OK) return st;
  SplitParams& p = w.sp;
  w.tok = T::kTok;
  p.workers = T::kCtas * sm_count() * kWarps;
  if (int64_t(p.a.kv_heads) * w.row_tiles * p.a.seqs < kManySegments * (kRows / 8)) p.start = nullptr;
  p.least = 1, p.edge = 0, p.even = 4;  // 16,000 keys, 8 heads, dim 128: 24.2 us, without 29.0
  return launch("launch k_attn_stream", kern, dim3(unsigned(p.workers / kWarps)), dim3(kThreads), T::kSmem, 0, stream, tk,
                tv, p);
}

template <int D>
nvfp4_status launch_of(const CUtensorMap& tk, const CUtensorMap& tv, Pending& w, cudaStream_t stream) {
  const SplitParams& sp = w.sp;
  if (w.rows == 8) {
    auto f = sp.several ? stream_launch<D, 8, true>
                        : (sp.a.seqs <= 32 ? stream_launch<D, 8, false, true> : stream_launch<D, 8, false>);
    return f(tk, tv, w, stream);
  }
  auto f = sp.a.o_f32 ? (sp.several ? stream_launch<D, 16, true, false, 1> : stream_launch<D, 16, false, false, 1>)
                      : (sp.several ? stream_launch<D, 16, true, false, 0> : stream_launch<D, 16, false, false, 0>);
  return f(tk, tv, w, stream);
}

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }
// Rows of partials: two a worker, the most of any variant (16 rows of 2 blocks
// an SM; 8 rows of 3 have fewer).
int64_t partial_rows() { return 2 * int64_t(sm_count()) * kWarps * 32; }
int64_t most_workers() { return 3 * int64_t(sm_count()) * kWarps; }

}  // namespace

int64_t attn_stream_workspace(int32_t dim) {
  return align256(partial_rows() * dim * 4) + align256(partial_rows() * 8) + align256((kMaxSeqs + 1) * 8) +
         align256(most_workers() * int64_t(sizeof(Cursor)));
}

nvfp4_status attn_stream(const mxfp4_cache* cache, const AttnParams& base, int32_t b, int32_t max_queries,
                         void* workspace, cudaStream_t stream, Pending& w) {
  const int32_t dim = cache->dim;
  CUtensorMap tk, tv;
  const int box = std::min(cache->page_size, dim == 64 ? 128 : (dim == 128 ? 64 : 32));
  // rows of 128 bytes: 256 / dim tokens of one head and page
  const int per_row = 256 / dim;
  const cuuint64_t dims[3] = {128, cuuint64_t(cache->page_size / per_row), cuuint64_t(cache->pages * cache->kv_heads)};
  const cuuint64_t strides[2] = {128, cuuint64_t(dim / 2) * cuuint64_t(cache->page_size)};
  const cuuint32_t bx[3] = {128, cuuint32_t(box / per_row), 1};
  const CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B;
  nvfp4_status st = make_map(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, cache->k_codes, 3, dims, strides, bx, swz, "K codes");
  if (st == NVFP4_OK)
    st = make_map(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, cache->v_codes, 3, dims, strides, bx, swz, "V codes");
  if (st != NVFP4_OK) return st;
  SplitParams& sp = w.sp;
  sp.a = base;
  sp.several = max_queries > 1;
  const int64_t rows_max = int64_t(max_queries) * base.group;
  const int32_t rows = rows_max <= 8 ? 8 : 16;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  sp.part_o = reinterpret_cast<float*>(ws);
  sp.part_ml = reinterpret_cast<float2*>(ws + align256(partial_rows() * dim * 4));
  sp.prefix =
      reinterpret_cast<int64_t*>(ws + align256(partial_rows() * dim * 4) + align256(partial_rows() * 8));
  sp.start = reinterpret_cast<Cursor*>(reinterpret_cast<uint8_t*>(sp.prefix) + align256((kMaxSeqs + 1) * 8));
  const int64_t row_tiles = (rows_max + rows - 1) / rows;
  if (row_tiles > 65535) return fail(NVFP4_EUNSUPPORTED, "mxfp4_cache_attention: too many query rows a sequence");
  w.rows = rows, w.row_tiles = int32_t(row_tiles), w.many = false;
  sp.a.seqs = std::min(kMaxSeqs, base.seqs - b);
  sp.a.table = base.table + int64_t(b) * base.table_ld;
  sp.a.lens = base.lens + b;
  split_queries(sp.a, base, b);
  auto launch = dim == 64 ? launch_of<64> : (dim == 128 ? launch_of<128> : launch_of<256>);
  return launch(tk, tv, w, stream);
}

}  // namespace nvfp4
