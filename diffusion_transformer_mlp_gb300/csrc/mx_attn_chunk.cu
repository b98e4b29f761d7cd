// Attention of many query rows over the paged MXFP4 cache (taking in a
// prompt by chunks) on tcgen05.
//
// A row is a (query, head of the group) pair: the heads that share a kv head
// are rows of one tile, so the cache is decoded once for all of them.  A
// segment is kNQ tiles of 128 rows of one (sequence, kv head) with the keys
// that they see in tiles of kTK; one CTA an SM works through an equal run of
// all segments' tiles (SplitParams).  Its warps walk the run each for itself,
// so the decoders are in the next segment while the softmax finishes this one:
//
//   warps 0-3, 4-7  softmax of row tile 0, 1: a thread is a row.  Scores come
//                   from tensor memory, the weights go back there as FP16 over
//                   the scores they came from (the A operand of p v)
//   4 or 8 warps    decode the tile's keys and values to FP16 in shared memory:
//                   a thread takes one token (of kTK), loads its codes and
//                   scales one tile ahead, and writes its rows under the
//                   128-byte swizzle
//   one warp        goes ahead of them over the scales: the references of each
//                   tile (below) and its NaN blocks
//   last warps      one a row tile, issue its MMAs: S = Q K^T (both from
//                   shared memory, K-major), O += P V (P from tensor memory, V
//                   MN-major)
//
// Every row tile has two score buffers: Q K^T of the next keys is under way
// while the softmax of these runs, so that neither waits for the other's
// latency (128 keys and one buffer took 4,300 cycles for 128 keys of both row
// tiles, this 3,400; the MMAs alone 2,050).
//
// What bounds it: the issue slots and latencies of the softmax and decoding
// warps (57% of the slots used, tensor pipe 50%).  Two prompts' chunks of 2,048
// queries on 4,099 and 8,192 keys, 32 / 8 heads, dim 128: 266 us, 1.2 PFLOP/s.
// Five kinds of warps run at once, so the loops are kept short enough for the
// instruction caches (fully unrolled: 430 us).
//
// FP16 operands are exact: a code times 2^(E - R + 13), R the tile's largest
// key scale (its power of two goes onto the scores), is exact for E >= R - 36,
// and a code times 2^(E - R + 5), R a running reference of the value scales of
// its block column (its power of two goes onto the output's columns), for E >=
// R - 28.  Q is scaled by a power of two per row.  Weights are held times 2^10
// against a reference that lags the running maximum by up to 2^5, so that the
// output is rarely rescaled (an 11-bit rounding; sums and statistics in FP32).
#include <algorithm>
#include <atomic>
#include <string>
#include <type_traits>

#include "mx_attn.cuh"

namespace nvfp4 {
namespace {

constexpr float kLag = 5.0f;
constexpr int kLeast = 4;      // tiles of a run at least
// Tiles that a new segment costs: its queries, its outputs, the pipeline's
// restart (2 chunks of 2,048 queries, 32 / 8 heads, dim 128: 294 us without, 270 with).
constexpr int kEdge = 8;
constexpr int kMeta = 8;       // tiles whose references are kept: the decoders are up to 6 ahead of the softmax
constexpr int kTK = 64;        // keys of a tile
constexpr int kHeadroom = 8;   // value scales may exceed their reference by 2^8 before it is raised
constexpr int kLiftK = 13, kLiftV = 5;  // largest elements: 6 * 2^13
// Where rows see different keys (see too_wide): keys down to 2^-36 of the tile's
// largest are exact, and values down to 2^-28 of their reference, which may be 2^16
// above the largest that a row sees: a row keeps those down to 2^-12 of its own.
// (2^8, as with few rows, would work more of the first rows of prompts anew, which
// see little but a first token whose values may be small.)
constexpr int kSpreadK = 23 + kLiftK, kSpreadV = 16;

template <int D>
struct Chunk {
  static constexpr int C = D / 32;
  static constexpr int kNQ = D == 256 ? 1 : 2;
  static constexpr int kSlots = D == 256 ? 2 : 4;     // decoded tiles
  // Keys and values of a tile handed on apart, so that with two slots the next
  // keys need not wait for this tile's p v (2 x 2,048 queries on 8,192 keys,
  // dim 256: 1,336 -> 984 us, 1,021 with the check for what rows see; with four
  // slots it only costs, dim 128: 366 -> 409).
  static constexpr bool kApart = kSlots == 2;
  static constexpr int kQBytes = 128 * D * 2;         // one row tile
  static constexpr int kKvBytes = kTK * D * 2;        // one decoded tile of K or V
  // one row tile leaves registers for eight decoding warps (dim 256)
  static constexpr int kDecoders = kNQ == 1 ? 8 : 4;
  static constexpr int kWarpD = kNQ * 4, kWarpR = kWarpD + kDecoders, kWarpMma = kWarpR + 1;
  static constexpr int kThreads = (kWarpMma + kNQ) * 32;
  static constexpr int kPart = D * kTK / (32 * kDecoders);  // elements of K (and V) of a decoding thread
  static constexpr int kStage = 32 * 64;              // a softmax warp's outputs on their way, 32 columns at a time
  static constexpr int kSmem = kNQ * kQBytes + 2 * kSlots * kKvBytes + kWarpD * kStage + 4096;
  static constexpr uint32_t kS = 0, kO = kNQ * 2 * kTK;  // tensor-memory columns: scores, outputs
  static constexpr uint32_t kTmem = 512;
  static_assert(kNQ * (2 * kTK + D) <= 512, "tensor memory");
  static_assert(kSmem <= 232448, "shared memory");
};

// A warp's place in the run of its block: a segment, of which the n tiles from
// seg.t on belong to the run, after g tiles of it; `left` places with these to go.
struct Walk {
  Cursor seg;
  int32_t left, n, g;
};

// Small shared state behind the operands.
struct Shared {
  uint64_t done;
  uint64_t q_full[2], o_empty[2];                 // by row tile: Q of a segment is there; its outputs are read
  // by slot: references; decoded keys (with the values, unless kApart) and
  // values; both row tiles' scores, and p v, complete
  uint64_t ref_full[4], k_full[4], v_full[4], k_empty[4], v_empty[4];
  uint64_t s_full[2][2], p_full[2][2];            // by row tile and score buffer
  uint64_t pv_done[2], o_full[2];                 // by row tile: p v of a tile, of a segment's last tile is complete
  uint32_t tmem;
  int abort_flag;
  Cursor first;                // of the run
  int32_t places;              // from there to its end
  Walk walk[16][2];            // by warp; kept here, as registers are short
  int32_t rk[kMeta];           // reference of the keys' scales
  int32_t rv[kMeta][8];        // of the values' scales by block, as the outputs have it from this tile on
  float vfac[kMeta][8];        // factor onto the outputs before this tile (2^(old - new reference))
  uint32_t raised[kMeta];      // the factors are not all 1
  uint32_t nan_any[kMeta];     // a block of values holds NaN
  uint32_t nan_bits[kMeta][8][kTK / 32];  // [block][32 tokens]
  int check;                   // the run may have segments to work anew
  uint32_t wide[32];           // those: a bit each, shared by those 1,024 apart
};
static_assert(sizeof(Shared) <= 4096, "shared state");

// Shared-memory descriptors, 128-byte swizzle, descriptor version 1.  The high
// word is the same for both forms (8-row groups 1,024 bytes apart); the low
// word is the address and the leading offset, so a step along the operand is
// one 32-bit addition.
//   K-major: rows of 128 bytes; the leading offset is not used
//   MN-major: 64 elements x 8 rows of the contraction an atom, the next 64
//   elements atom_bytes on
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lead_bytes) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lead_bytes >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(uint32_t(accumulate))
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(uint32_t(accumulate))
      : "memory");
}
// 32 columns of this warp's lanes, complete on return.
__device__ __forceinline__ void tmem_load32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Eight 16-bit elements without the alignment of one load.
__device__ __noinline__ uint4 load_8x16(const uint16_t* e) {
  return make_uint4(uint32_t(e[0]) | uint32_t(e[1]) << 16, uint32_t(e[2]) | uint32_t(e[3]) << 16,
                    uint32_t(e[4]) | uint32_t(e[5]) << 16, uint32_t(e[6]) | uint32_t(e[7]) << 16);
}

// After the run, by all warps: which segments have to be worked anew (a warp each),
// and those over what was written.  Not inlined: the loops of the kernel are not to
// make room for it.
template <int D>
__device__ __noinline__ void check_run(const SplitParams& sp, Shared& sh, int32_t places) {
  using T = Chunk<D>;
  constexpr int kRows = 128 * T::kNQ, kWarps = T::kThreads / 32;
  const int warp = threadIdx.x >> 5;
  for (int pass = 0; pass < 2; ++pass) {
    int seg = 0;
    walk_run<kRows>(sp, sh.first, places, int32_t(blockIdx.x), kTK, [&](const Cursor& c, int32_t n, int64_t part) {
      const uint32_t bit = 1u << (seg / 32 & 31);
      if (pass == 0 && seg % kWarps == warp && too_wide<D, kRows>(sp.a, c, n, kTK, kSpreadV, kSpreadK))
        atomicOr(&sh.wide[seg & 31], bit);
      if (pass == 1 && (sh.wide[seg & 31] & bit)) wide_segment<D, kRows, true>(sp, c, n, part, kTK, warp, kWarps);
      ++seg;
    });
    __syncthreads();
    if (!__any_sync(0xFFFFFFFFu, sh.wide[threadIdx.x & 31] != 0)) return;
  }
}

template <int D>
__global__ void __launch_bounds__(Chunk<D>::kThreads, 1)
    k_attn_chunk(const uint8_t* __restrict__ k_codes, const uint8_t* __restrict__ v_codes,
                 const __grid_constant__ SplitParams sp) {
  using T = Chunk<D>;
  constexpr int C = T::C, kNQ = T::kNQ, kSlots = T::kSlots, kRows = 128 * kNQ;
  const AttnParams& a = sp.a;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sq = smem;                          // [row tile][atom][128 rows][128 bytes]
  uint8_t* sk = sq + kNQ * T::kQBytes;         // [slot][atom][token][128 bytes]
  uint8_t* sv = sk + kSlots * T::kKvBytes;
  uint8_t* staging = sv + kSlots * T::kKvBytes;
  Shared& sh = *reinterpret_cast<Shared*>(staging + T::kWarpD * T::kStage);
  const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 32) {
    mbar_init(&sh.done, kNQ);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh.ref_full[i], 1);
      mbar_init(&sh.k_full[i], T::kDecoders);
      mbar_init(&sh.v_full[i], T::kDecoders);
      mbar_init(&sh.k_empty[i], kNQ);
      mbar_init(&sh.v_empty[i], kNQ);
      mbar_init(&sh.s_full[i >> 1][i & 1], 2);
      mbar_init(&sh.p_full[i >> 1][i & 1], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 4);
      mbar_init(&sh.pv_done[i], 1);
      mbar_init(&sh.o_full[i], 1);
      mbar_init(&sh.o_empty[i], 4);
    }
    sh.abort_flag = 0;
    for (uint32_t& w : sh.wide) w = 0;
    sh.check = 0;
    fence_barrier_init();
  }
  grid_wait();
  if (warp == T::kWarpMma) tmem_alloc(&sh.tmem, T::kTmem);

  // this block's run of tiles: up to 32 sequences are counted by the first warp alone
  auto begin_at = [&](int64_t total, const auto& counts) {
    const int32_t workers = live_workers(sp, total), w = int32_t(blockIdx.x);
    int32_t places = 0;
    if (w < workers) {
      const int64_t x0 = worker_start(total, w, workers);
      Cursor first;
      const int32_t skip = cursor_at(first, a, counts, x0, kRows, kTK, sp.edge);
      places = int32_t(worker_start(total, w + 1, workers) - x0) - skip;
      if (lane == 0) sh.first = first, sp.start[w] = first;
    }
    if (lane == 0) sh.places = places;
  };
  if (a.seqs <= 32) {
    if (warp == 0) {
      int share = 1;
      while (a.seqs * share * 2 <= 32) share *= 2;
      const WarpCounts counts = warp_counts(sp, kRows, kTK, share);
      if (blockIdx.x == 0) leave_places(sp, counts);
      begin_at(all_places(counts), counts);
    }
  } else {
    int64_t* prefix = reinterpret_cast<int64_t*>(smem);
    tile_counts<T::kThreads>(sp, prefix, kRows, kTK);
    if (warp == 0) begin_at(prefix[a.seqs], prefix);
  }
  tc_fence_before();
  __syncthreads();  // the counts are read, the first tile is known
  tc_fence_after();
  const int32_t tiles = sh.places;
  if (tiles <= 0) {  // no worker, or nothing but the room before a segment
    if (warp == T::kWarpMma) tmem_dealloc(sh.tmem, T::kTmem);
    return;
  }
  const uint32_t tmem = sh.tmem;
  const volatile int* abort_flag = &sh.abort_flag;
  // Every warp walks the segments of the run for itself.
  auto next_segment = [&](const Walk& from, Walk& to) {
    Walk w = from;
    w.left -= w.n;
    w.g += w.n;
    const bool next = w.n > 0;
    if (next) w.left -= sp.edge;
    if (w.left > 0) {
      if (next) {
        w.seg.t += w.n - 1;
        cursor_next(w.seg, a, kRows, kTK);
      }
      w.n = min(w.seg.s.n - w.seg.t, w.left);
    } else {
      w.n = 0;
    }
    to = w;
  };
  // false at the end of the run
  auto advance = [&](const Walk& from, Walk& to) -> bool {
    __syncwarp();
    if (lane == 0) next_segment(from, to);
    __syncwarp();
    return to.n > 0;
  };
  Walk& wk = sh.walk[warp][0];
  if (lane == 0) wk.seg = sh.first, wk.left = tiles, wk.n = wk.g = 0;
  // false once a bounded wait anywhere ran out, for the whole warp alike
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    const bool ok = mbar_wait_bounded(bar, parity, a.wait_limit_cycles, abort_flag);
    if (__all_sync(0xFFFFFFFFu, ok)) return true;
    sh.abort_flag = 1;
    return false;
  };

  if (warp < T::kWarpD) {
    // ------------------------------------------------------------ softmax
    const int qt = warp >> 2, q = warp & 3;
    const int r = q * 32 + lane;  // row of the tile, lane of tensor memory
    const uint32_t t_lane = tmem + (uint32_t(q * 32) << 16);
    const uint32_t t_o = t_lane + T::kO + qt * D;
    // The warp's queries into shared memory, a row's largest element going to
    // [2^13, 2^14) and the sign of the softmax scale onto the elements.  D / 8
    // lanes load a row, so that the loads are of whole rows (a thread that
    // loads its own row: 13,000 cycles for all rows), by asynchronous copies
    // (through registers, 16 of them under way: the two prompts 272 us instead of
    // 266); then a thread scales its own row in place.  Returns the factor of this
    // thread's scores.
    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kAhead = D == 64 ? 4 : 2;
    auto load_q = [&](const Cursor& c) -> float {
      const int32_t row = c.rt * kRows + qt * 128 + r;
      int64_t off = -1;
      if (row < c.nq * a.group) {
        const int32_t qi = row / a.group;
        off = int64_t(c.q0 + qi) * a.q_st + int64_t(c.h * a.group + row - qi * a.group) * a.q_sh;
      }
      const int col = lane % kLanes;
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + 8 * col;
      uint8_t* dst = sq + qt * T::kQBytes;
      // chunk `ch` of eight elements of the row rq
      auto place = [&](int rq, int ch) {
        return reinterpret_cast<uint4*>(dst + (ch / 8) * (128 * 128) + rq * 128 + (((ch & 7) ^ (rq & 7)) << 4));
      };
      // small loops, as straight-line code that runs once is slow to fetch
      if (a.q_vec) {
#pragma unroll 2
        for (int i = 0; i < kLanes; ++i) {
          const int64_t o = __shfl_sync(0xFFFFFFFFu, off, i * kAtOnce + lane / kLanes);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           smem_u32(place(q * 32 + i * kAtOnce + lane / kLanes, col))),
                       "l"(src + max(o, int64_t(0))), "r"(o >= 0 ? 16 : 0)
                       : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
      } else {
#pragma unroll 1
        for (int i = 0; i < kLanes; ++i) {
          const int64_t o = __shfl_sync(0xFFFFFFFFu, off, i * kAtOnce + lane / kLanes);
          uint4 v = make_uint4(0, 0, 0, 0);
          if (o >= 0) v = load_8x16(src + o);
          *place(q * 32 + i * kAtOnce + lane / kLanes, col) = v;
        }
      }
      __syncwarp();
      // magnitudes of 16-bit floats are in the order of their bits (NaN above all)
      uint32_t top = 0;
#pragma unroll kAhead
      for (int i = 0; i < kLanes; ++i) {
        const uint4 v = *place(r, i);
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                     __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
      }
      top = max(top & 0xFFFFu, top >> 16);
      auto value = [&](uint32_t x) { return a.bf16 ? word_to_f32<__nv_bfloat16>(x) : word_to_f32<__half>(x); };
      const int32_t eb = int32_t(__float_as_uint(value(top).x) >> 23) & 0xFF;
      const int32_t up = (eb == 0 || eb == 255) ? 0 : min(126, 140 - eb);
      const float mul = a.scale_log2 < 0.0f ? -pow2i(up) : pow2i(up);
#pragma unroll kAhead
      for (int i = 0; i < kLanes; ++i) {
        const uint4 v = *place(r, i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t h[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float2 t = value(w[x]);
          h[x] = f32_to_word<__half>(t.x * mul, t.y * mul);
        }
        *place(r, i) = make_uint4(h[0], h[1], h[2], h[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full[qt]);
      return fabsf(a.scale_log2) * pow2i(-up);
    };
    auto live_rows = [&](const Cursor& c) { return c.rt * kRows + qt * 128 + q * 32 < c.nq * a.group; };
    advance(wk, wk);
    float qf = load_q(wk.seg);
    bool ok = true;
    for (int seg = 0; ok; ++seg) {
      const Walk& w = sh.walk[warp][seg & 1];
      const Cursor& cu = w.seg;
      const int32_t n = w.n, g = w.g, sink_tiles = cu.s.sink_tiles - cu.t, first_tile = cu.t,
                    lo_tile = cu.s.lo_tile - sink_tiles;
      // A warp behind the segment's last row: the barriers go on, and nothing is worked
      // out, which would be masked throughout (rows of 64 to a kv head: 1.45 us a tile,
      // so 0.8).  Whatever is in its lanes of tensor memory stays in them.
      if (!live_rows(cu)) {
        for (int j = 0; ok && j < n; ++j) {
          const int x = g + j;
          ok = wait(&sh.s_full[qt][x & 1], (x >> 1) & 1);
          if (lane == 0 && ok) mbar_arrive(&sh.p_full[qt][x & 1]);
        }
        if (!ok) break;
        Walk& next = sh.walk[warp][(seg + 1) & 1];
        const bool more = advance(w, next);
        if (more) qf = load_q(next.seg);
        ok = wait(&sh.o_full[qt], seg & 1);
        if (lane == 0 && ok) mbar_arrive(&sh.o_empty[qt]);
        if (!ok || !more) break;
        continue;
      }
      const int32_t row = cu.rt * kRows + qt * 128 + r;
      const bool real = row < cu.nq * a.group;
      const int32_t pos = cu.len - cu.nq + (real ? row / a.group : 0);
      // the row sees keys j < end with j >= from or j < sinks
      const int32_t end = !real ? 0 : (a.causal ? min(cu.len, pos + 1) : cu.len);
      const int32_t from = a.window > 0 ? pos - a.window + 1 : 0;
      float m = -INFINITY;
      float2 l2 = make_float2(0.0f, 0.0f);
      uint32_t nan_cols = 0;  // blocks of the output that are NaN
      int last_meta = 0;
      for (int j = 0; j < n; ++j) {
        const int x = g + j;  // of the run's tiles
        const uint32_t t_s = t_lane + T::kS + (qt * 2 + (x & 1)) * kTK;
        if (!wait(&sh.s_full[qt][x & 1], (x >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int ms_ = x & (kMeta - 1);
        const int32_t tok0 = (j < sink_tiles ? j + first_tile : j + lo_tile) * kTK;
        const float c1 = qf * pow2i(sh.rk[ms_] - 127 - kLiftK);
        last_meta = ms_;
        const bool all = tok0 + kTK <= end && (tok0 >= from || tok0 + kTK <= a.sinks);
        const bool plain = __all_sync(0xFFFFFFFFu, all);
        // keys of the tile that the row sees: [lo, hi) and [0, sk_)
        const int32_t hi = end - tok0, lo = from - tok0, sk_ = a.sinks - tok0;
        // Weights against the reference as it stands, in registers; where a
        // row's maximum is too far ahead of it, it is raised and the weights are
        // formed again (the scores are still there).
        const uint64_t c1p = pair_const(c1);
        bool raised = sh.raised[ms_] != 0;
        float alpha = 1.0f;
        // one pass; true if the weights are in place
        auto weights = [&](auto masked) -> bool {
          const float sub = kWeightLog2 - (m == -INFINITY ? 0.0f : m);
          const uint64_t subp = pair_const(sub);
          uint64_t sum = 0;
          float top = -INFINITY;
          uint32_t w[kTK / 32][16];
#pragma unroll
          for (int c = 0; c < kTK / 32; ++c) {
            uint32_t v[32];
            tmem_load32(t_s + 32 * c, v);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float2 t = unpair(fma2(pair_of(v[i], v[i + 1]), c1p, subp));
              if constexpr (decltype(masked)::value) {
                const int y = 32 * c + i;
                if (y >= hi || (y < lo && y >= sk_)) t.x = -INFINITY;
                if (y + 1 >= hi || (y + 1 < lo && y + 1 >= sk_)) t.y = -INFINITY;
              }
              top = fmaxf(top, fmaxf(t.x, t.y));
              t.x = exp2_approx(t.x), t.y = exp2_approx(t.y);
              sum = add2(sum, pair_of(__float_as_uint(t.x), __float_as_uint(t.y)));
              w[c][i / 2] = f32_to_word<__half>(t.x, t.y);
            }
          }
          top -= sub;  // back to the score's logarithm
          const bool raise = top > m + kLag;
          if (__any_sync(0xFFFFFFFFu, raise)) {
            if (raise) {
              // not below the maximum by its rounding either, however large it is
              const float ref = fmaf(fabsf(top), 0x1p-22f, top);
              alpha *= exp2_approx(m - ref);
              m = ref;
            }
            __syncwarp();
            raised = true;
            return false;
          }
          l2.x = l2.x * alpha + unpair(sum).x, l2.y = l2.y * alpha + unpair(sum).y;
          if (j > 0 && raised) {
            // The p v of the tile before has to be complete.  Parities mean one
            // phase here: the slot is not filled again before this tile's
            // weights, and p v of two tiles ago is complete (this tile's scores
            // were issued behind it), but if keys and values go apart only that
            // of this row tile.
            if (T::kApart ? !wait(&sh.pv_done[qt], (x - 1) & 1)
                          : !wait(&sh.v_empty[(x - 1) % kSlots], ((x - 1) / kSlots) & 1))
              return true;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              const float f = alpha * sh.vfac[ms_][c / 32];
              uint32_t v[32];
              tmem_load32(t_o + c, v);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
              tmem_st_32x32b_x32(t_o + c, v);
            }
          }
#pragma unroll
          for (int c = 0; c < kTK / 32; ++c) tmem_st_x16(t_s + 16 * c, w[c]);
          return true;
        };
        // the second pass finds every maximum in reach of its reference
#pragma unroll 1
        for (int attempt = 0; attempt < 3; ++attempt)
          if (plain ? weights(std::false_type{}) : weights(std::true_type{})) break;
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[qt][x & 1]);
        if (sh.nan_any[ms_]) {
          // a block of NaN among the values reaches the rows that see its key
          for (int blk = 0; blk < C; ++blk)
            for (int w = 0; w < kTK / 32; ++w) {
              uint32_t bits = sh.nan_bits[ms_][blk][w];
              while (bits != 0) {
                const int32_t t = w * 32 + __ffs(bits) - 1;
                bits &= bits - 1;
                if (t < hi && (t >= lo || t < sk_)) nan_cols |= 1u << blk;
              }
            }
        }
      }
      if (!ok) break;
      // the next segment's queries first: the MMAs that read this segment's are
      // complete, and the next ones can start while the outputs are written
      Walk& next = sh.walk[warp][(seg + 1) & 1];
      const bool more = advance(w, next);
      if (more) qf = load_q(next.seg);
      // ---- output
      ok = wait(&sh.o_full[qt], seg & 1);
      tc_fence_after();
      if (!ok) break;
      const bool whole = cu.t == 0 && w.n == cu.s.n;
      const int32_t qi = real ? row / a.group : 0, hq = cu.h * a.group + (real ? row - qi * a.group : 0);
      const float l = l2.x + l2.y;
      const int32_t pe = part_exponent(l);
      const float inv = !whole ? pow2i(-pe) : (l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l));
      const int64_t part = int64_t(blockIdx.x) * 2 + (seg > 0 ? 1 : 0);
      const int64_t off = real ? int64_t(cu.q0 + qi) * a.o_st + int64_t(hq) * a.o_sh : -1;
      uint8_t* stage = staging + warp * T::kStage;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t v[32];
        __syncwarp();  // rows with and without NaN
        tmem_load32(t_o + c, v);
        if (c + 32 == D) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.o_empty[qt]);
        }
        // c / 32 is a reference's block, and its factor the same for all rows
        const float fac = pow2i(sh.rv[last_meta][c / 32] - 127 - kLiftV) * inv;
        if ((nan_cols >> (c / 32)) & 1u) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0x7FFFFFFFu;
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * fac);
        }
        if (!whole) {
          // [D / 4][rows] of four columns: a warp writes 512 bytes at a time
          uint4* d = reinterpret_cast<uint4*>(sp.part_o) + (part * (D / 4) + c / 4) * kRows + qt * 128 + r;
          if (real) {
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i * kRows] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
          continue;
        }
        if (a.o_f32) {
          if (off >= 0) {
            uint4* d = reinterpret_cast<uint4*>(static_cast<float*>(a.out) + off + c);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
          continue;
        }
        // through shared memory, so that four lanes write 64 bytes of a row
        // (a thread that writes its own row: 4,400 to 10,000 cycles)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t h[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float f0 = __uint_as_float(v[8 * i + 2 * x]), f1 = __uint_as_float(v[8 * i + 2 * x + 1]);
            h[x] = a.bf16 ? f32_to_word<__nv_bfloat16>(f0, f1) : f32_to_word<__half>(f0, f1);
          }
          *reinterpret_cast<uint4*>(stage + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) =
              make_uint4(h[0], h[1], h[2], h[3]);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = i * 8 + lane / 4;
          const uint4 h = *reinterpret_cast<const uint4*>(stage + rr * 64 + (((lane & 3) ^ ((rr >> 1) & 3)) << 4));
          const int64_t o = __shfl_sync(0xFFFFFFFFu, off, rr);
          if (o >= 0) store_o8_words(a, static_cast<uint16_t*>(a.out) + o + c + (lane & 3) * 8, h);
        }
        __syncwarp();
      }
      if (!whole)
        sp.part_ml[part * kRows + qt * 128 + r] = make_float2(m + float(pe), l * pow2i(-pe));
      else if (real && a.lse != nullptr)
        a.lse[int64_t(cu.q0 + qi) * (a.kv_heads * a.group) + hq] =
            l == 0.0f ? -INFINITY : (m - kWeightLog2 + log2f(l)) * 0.6931471805599453f;
      if (!more) break;
    }
  } else if (warp < T::kWarpR) {
    // ------------------------------------------------------------ decoding
    const int t = int(threadIdx.x) - T::kWarpD * 32;
    const int tok = t % kTK, part = t / kTK;  // the token, and the thread's share of its rows
    constexpr int kWords = T::kPart / 32;     // blocks of a share
    bool ok = true;
    while (ok && advance(wk, wk)) {
      const Cursor cu = wk.seg;
      const int32_t n = wk.n, g = wk.g;
      const int32_t* table = a.table + int64_t(cu.b) * a.table_ld;
      auto page_of = [&](int j) -> int32_t {
        const int32_t at = cu.s.tile(cu.t + j) * kTK + tok;
        // -1: a key that no row sees, which counts as zeros
        return j < n && cu.s.has(a, at) ? max(table[min(at >> a.page_shift, int32_t(a.table_ld) - 1)], 0) : -1;
      };
      uint4 raw[2][kWords];  // codes of K and V
      uint32_t sc[2] = {0, 0};
      auto fetch = [&](int j, int32_t page) {
        const int32_t at = cu.s.tile(cu.t + j) * kTK + tok;
        const bool in = page >= 0;
        const int32_t z = min(page, int32_t(a.pages) - 1) * a.kv_heads + cu.h;
        const int64_t rowi = (int64_t(z) << a.page_shift) + (at & ((1 << a.page_shift) - 1));
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const uint8_t* src = (kv ? v_codes : k_codes) + rowi * (D / 2) + part * (T::kPart / 2);
          const uint8_t* s = (kv ? a.v_scales : a.k_scales) + rowi * C + part * kWords;
#pragma unroll
          for (int i = 0; i < kWords; ++i)
            raw[kv][i] = in ? *reinterpret_cast<const uint4*>(src + 16 * i) : make_uint4(0, 0, 0, 0);
          sc[kv] = 0;
          if (in) {
            if constexpr (kWords == 1) sc[kv] = *s;
            else if constexpr (kWords == 2) sc[kv] = *reinterpret_cast<const uint16_t*>(s);
            else sc[kv] = *reinterpret_cast<const uint32_t*>(s);
          }
        }
      };
      int32_t page = page_of(0);
      fetch(0, page);
      page = page_of(1);
      for (int j = 0; j < n; ++j) {
        const int x0 = g + j, slot = x0 % kSlots, meta = x0 & (kMeta - 1);
        const uint32_t ph = (x0 / kSlots) & 1;
        // this tile's codes make room for the next tile's, whose loads take as
        // long as the decoding
        uint4 cur[2][kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) cur[0][i] = raw[0][i], cur[1][i] = raw[1][i];
        const uint32_t scale[2] = {sc[0], sc[1]};
        fetch(j + 1, page);
        page = page_of(j + 2);
        // the references come after their writer has seen the slot empty
        ok = wait(&sh.ref_full[slot], ph) && (T::kApart || wait(&sh.v_empty[slot], ph ^ 1));
        if (!ok) break;
        const int32_t rk = sh.rk[meta] - kLiftK;
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          // a slot of keys is free once its scores are there, one of values
          // only after p v: the next keys do not wait for that
          if constexpr (T::kApart) {
            ok = wait(kv ? &sh.v_empty[slot] : &sh.k_empty[slot], ph ^ 1);
            if (!ok) break;
          }
          uint8_t* dst = (kv ? sv : sk) + slot * T::kKvBytes + tok * 128;
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            const int32_t e = ((kv ? scale[1] : scale[0]) >> (8 * i)) & 0xFF;
            const int32_t ref = kv ? sh.rv[meta][part * kWords + i] - kLiftV : rk;
            const float f = __uint_as_float(uint32_t(max(e - ref + 127, 0)) << 23);
            uint32_t fw = f32_to_word<__half>(f, f);
            if (e == 255) fw = kv ? 0u : 0x7FFF7FFFu;
            const uint32_t w[4] = {kv ? cur[1][i].x : cur[0][i].x, kv ? cur[1][i].y : cur[0][i].y,
                                   kv ? cur[1][i].z : cur[0][i].z, kv ? cur[1][i].w : cur[0][i].w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t h[4];
              e2m1x8_to_half(w[x], h);
              const int d = part * T::kPart + i * 32 + x * 8;
              *reinterpret_cast<uint4*>(dst + (d / 64) * (kTK * 128) + ((((d % 64) / 8) ^ (tok & 7)) << 4)) =
                  make_uint4(hmul2(h[0], fw), hmul2(h[1], fw), hmul2(h[2], fw), hmul2(h[3], fw));
            }
          }
          if constexpr (T::kApart) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(kv ? &sh.v_full[slot] : &sh.k_full[slot]);
          }
        }
        if (!ok) break;
        if constexpr (!T::kApart) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.k_full[slot]);
        }
      }
    }
  } else if (warp == T::kWarpR) {
    // ------------------------------------------------------------ references
    // a lane takes kTK / 32 tokens of each tile; scales are loaded a tile ahead,
    // their pages looked up a tile before that
    constexpr int kPer = kTK / 32, kW = (C + 3) / 4;
    bool ok = true;
    while (ok && advance(wk, wk)) {
      const Cursor cu = wk.seg;
      const int32_t n = wk.n, g = wk.g;
      const int32_t* table = a.table + int64_t(cu.b) * a.table_ld;
      uint32_t kw[kPer][kW], vw[kPer][kW];
      int32_t pages[kPer];
      auto look_up = [&](int j) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int32_t at = cu.s.tile(cu.t + j) * kTK + i * 32 + lane;
          pages[i] = j < n && cu.s.has(a, at) ? max(table[min(at >> a.page_shift, int32_t(a.table_ld) - 1)], 0) : -1;
        }
      };
      auto fetch = [&](int j) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int32_t at = cu.s.tile(cu.t + j) * kTK + i * 32 + lane;
          const int32_t z = min(pages[i], int32_t(a.pages) - 1) * a.kv_heads + cu.h;
          const int64_t at_s = ((int64_t(z) << a.page_shift) + (at & ((1 << a.page_shift) - 1))) * C;
#pragma unroll
          for (int y = 0; y < kW; ++y) {
            kw[i][y] = vw[i][y] = 0;
            if (pages[i] >= 0) {
              if constexpr (C == 2) {
                kw[i][0] = *reinterpret_cast<const uint16_t*>(a.k_scales + at_s);
                vw[i][0] = *reinterpret_cast<const uint16_t*>(a.v_scales + at_s);
              } else {
                kw[i][y] = *reinterpret_cast<const uint32_t*>(a.k_scales + at_s + 4 * y);
                vw[i][y] = *reinterpret_cast<const uint32_t*>(a.v_scales + at_s + 4 * y);
              }
            }
          }
        }
      };
      int32_t rv = -1;  // of block `lane`
      // largest scale of the values that all rows see, smallest but 0 (less 1) of
      // all blocks of the others' tiles
      const Common rows = common_of(a, cu.len, cu.nq, cu.rt, kRows);
      int32_t common = 0;
      uint32_t least = 254;
      bool check = false;
      look_up(0);
      fetch(0);
      look_up(1);
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        int32_t mk = 0, mv[C];
        uint32_t nan[C][kPer], any = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          mv[c] = 0;
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int32_t ek = (kw[i][c / 4] >> (8 * (c % 4))) & 0xFF;
            const int32_t ev = (vw[i][c / 4] >> (8 * (c % 4))) & 0xFF;
            mk = max(mk, ek == 255 ? 0 : ek);
            mv[c] = max(mv[c], ev == 255 ? 0 : ev);
            nan[c][i] = __ballot_sync(0xFFFFFFFFu, ev == 255);
            any |= nan[c][i];
          }
        }
        mk = __reduce_max_sync(0xFFFFFFFFu, mk);
        const bool all = rows.one || all_see(a, rows, cu.s.tile(cu.t + j) * kTK, kTK);
        if (!all) {
          uint32_t lk = 254, lv = 254;
#pragma unroll 1
          for (int b = 0; b < 32; b += 8)
#pragma unroll
            for (int i = 0; i < kPer * kW; ++i) {
              lk = min(lk, ((kw[i / kW][i % kW] >> b) & 0xFF) - 1);
              lv = min(lv, ((vw[i / kW][i % kW] >> b) & 0xFF) - 1);
            }
          least = min(least, __reduce_min_sync(0xFFFFFFFFu, lv));
          check = check || int32_t(__reduce_min_sync(0xFFFFFFFFu, lk)) + 1 < mk - kSpreadK;
        }
        fetch(j + 1);
        look_up(j + 2);
        const int slot = (g + j) % kSlots, meta = (g + j) & (kMeta - 1);
        // lane c takes block c from here
        int32_t top = 0;
        uint32_t bits[kPer];
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int32_t t = __reduce_max_sync(0xFFFFFFFFu, mv[c]);
          if (lane == c) {
            top = t;
#pragma unroll
            for (int i = 0; i < kPer; ++i) bits[i] = nan[c][i];
          }
        }
        // values: running references, raised only when the headroom is used up
        float fac = 1.0f;
        const bool up = rv >= 0 && top > rv + kHeadroom;
        if (up) fac = pow2i(rv - top);
        if (up || rv < 0) rv = top;
        if (all) common = max(common, top);
        const bool raised = __any_sync(0xFFFFFFFFu, lane < C && up);
        // whoever used this place kMeta tiles ago is done once the scores of
        // kSlots tiles ago are there
        ok = wait(T::kApart ? &sh.k_empty[slot] : &sh.v_empty[slot], (((g + j) / kSlots) & 1) ^ 1);
        if (!ok) break;
        if (lane < C) {
          sh.rv[meta][lane] = rv;
          sh.vfac[meta][lane] = fac;
#pragma unroll
          for (int i = 0; i < kPer; ++i) sh.nan_bits[meta][lane][i] = bits[i];
        }
        if (lane == 0) {
          sh.rk[meta] = mk;
          sh.raised[meta] = raised;
          sh.nan_any[meta] = any;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.ref_full[slot]);
      }
      if (lane < C && !rows.one && (check || rv > (common > 0 ? common : int32_t(least) + 1) + kSpreadV)) sh.check = 1;
    }
  } else {
    // ------------------------------------------------------------ MMA issue
    // The whole warp runs this and one thread is elected where it issues: the
    // descriptors then stay in uniform registers (issued under lane == 0, an
    // MMA took 25 instructions and the issuing warp was the bottleneck: 336
    // against 279 us).
    constexpr uint32_t kIdS = (1u << 4) | (uint32_t(kTK >> 3) << 17) | (8u << 24);               // M = 128, N = kTK
    constexpr uint32_t kIdO = (1u << 4) | (1u << 16) | (uint32_t(D >> 3) << 17) | (8u << 24);    // N = D, B MN-major
    const int qt = warp - T::kWarpMma;
    const uint32_t q_lo = desc_lo(smem_u32(sq + qt * T::kQBytes), 16), k_lo = desc_lo(smem_u32(sk), 16),
                   v_lo = desc_lo(smem_u32(sv), kTK * 128);
    const uint32_t t_q = tmem + T::kS + qt * 2 * kTK, t_o = tmem + T::kO + qt * D;
    bool live = true;  // the row tile has rows in this segment; a second one of few rows has none
    auto scores = [&](int x) -> bool {
      const int slot = x % kSlots;
      if (!wait(&sh.k_full[slot], (x / kSlots) & 1)) return false;
      tc_fence_after();
      const uint32_t kb = k_lo + uint32_t(slot) * (T::kKvBytes >> 4), t_s = t_q + (x & 1) * kTK;
      if (elect_one()) {
        if (live) {
#pragma unroll
          for (int d = 0; d < D; d += 16)
            mma_ss(t_s, q_lo + (d / 64) * (128 * 128 >> 4) + (d % 64) / 8,
                   kb + (d / 64) * (kTK * 128 >> 4) + (d % 64) / 8, kIdS, d > 0);
        }
        tc_commit(&sh.s_full[qt][x & 1]);
        if constexpr (T::kApart) tc_commit(&sh.k_empty[slot]);
        mbar_arrive(&sh.s_full[qt][x & 1]);  // hands on what the decoders wrote for the softmax
      }
      __syncwarp();
      return true;
    };
    bool ok = true;
    for (int seg = 0; ok && advance(wk, wk); ++seg) {
      const int32_t n = __shfl_sync(0xFFFFFFFFu, wk.n, 0), g = __shfl_sync(0xFFFFFFFFu, wk.g, 0);
      live = kNQ == 1 || __shfl_sync(0xFFFFFFFFu, wk.seg.rt * kRows + qt * 128 < wk.seg.nq * a.group, 0);
      ok = wait(&sh.q_full[qt], seg & 1) && scores(g) && (n == 1 || scores(g + 1));
      for (int j = 0; j < n && ok; ++j) {
        const int x = g + j;
        ok = wait(&sh.p_full[qt][x & 1], (x >> 1) & 1) &&
             (!T::kApart || wait(&sh.v_full[x % kSlots], (x / kSlots) & 1)) &&
             (j > 0 || seg == 0 || wait(&sh.o_empty[qt], (seg - 1) & 1));  // the outputs before are read
        if (!ok) break;
        tc_fence_after();
        const uint32_t vb = v_lo + uint32_t(x % kSlots) * (T::kKvBytes >> 4), t_p = t_q + (x & 1) * kTK;
        if (elect_one()) {
          if (live) {
#pragma unroll
            for (int t = 0; t < kTK; t += 16) mma_ts(t_o, t_p + t / 2, vb + t * 8, kIdO, j > 0 || t > 0);
          }
          tc_commit(&sh.v_empty[x % kSlots]);
          if constexpr (T::kApart) tc_commit(&sh.pv_done[qt]);
          if (j + 1 == n) tc_commit(&sh.o_full[qt]);
        }
        __syncwarp();
        if (j + 2 < n) ok = scores(x + 2);  // into the buffer that p v has read
      }
    }
    if (elect_one()) tc_commit(&sh.done);
    __syncwarp();
    if (!mbar_wait_bounded(&sh.done, 0, a.wait_limit_cycles, nullptr)) sh.abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && sh.abort_flag && a.dev_status != nullptr)
    atomicExch(a.dev_status, static_cast<uint32_t>(NVFP4_ETIMEOUT));
  if (sh.check) check_run<D>(sp, sh, tiles);
  if (warp == T::kWarpMma) {
    __syncwarp();
    tmem_dealloc(tmem, T::kTmem);
  }
}

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }
int64_t partial_rows(int32_t dim) { return 2 * int64_t(sm_count()) * (dim == 256 ? 128 : 256); }

template <int D>
nvfp4_status chunk_launch(const mxfp4_cache* cache, const SplitParams& p, cudaStream_t stream) {
  using T = Chunk<D>;
  auto kern = k_attn_chunk<D>;
  static std::atomic<uint64_t> ready{0};
  nvfp4_status st = allow_smem(reinterpret_cast<const void*>(kern), T::kSmem, ready);
  if (st != NVFP4_OK) return st;
  return launch("launch k_attn_chunk", kern, dim3(unsigned(p.workers)), dim3(T::kThreads), T::kSmem, 0, stream,
                static_cast<const uint8_t*>(cache->k_codes), static_cast<const uint8_t*>(cache->v_codes), p);
}

}  // namespace

int64_t attn_chunk_workspace(int32_t dim) {
  return align256(partial_rows(dim) * dim * 4) + align256(partial_rows(dim) * 8) + align256((kMaxSeqs + 1) * 8) +
         align256(sm_count() * int64_t(sizeof(Cursor)));
}

nvfp4_status attn_chunk(const mxfp4_cache* cache, const AttnParams& base, int32_t b, int32_t max_queries,
                        void* workspace, cudaStream_t stream, Pending& pending) {
  const int32_t dim = cache->dim;
  pending.tok = kTK, pending.many = true;
  SplitParams& sp = pending.sp;
  sp.a = base;
  sp.workers = sm_count();
  sp.several = max_queries > 1;
  sp.least = kLeast, sp.even = 0, sp.edge = kEdge;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  sp.part_o = reinterpret_cast<float*>(ws);
  sp.part_ml = reinterpret_cast<float2*>(ws + align256(partial_rows(dim) * dim * 4));
  sp.prefix = reinterpret_cast<int64_t*>(ws + align256(partial_rows(dim) * dim * 4) + align256(partial_rows(dim) * 8));
  sp.start = reinterpret_cast<Cursor*>(reinterpret_cast<uint8_t*>(sp.prefix) + align256((kMaxSeqs + 1) * 8));
  sp.a.seqs = std::min(kMaxSeqs, base.seqs - b);
  sp.a.table = base.table + int64_t(b) * base.table_ld;
  sp.a.lens = base.lens + b;
  split_queries(sp.a, base, b);
  if (dim == 64) return chunk_launch<64>(cache, sp, stream);
  return dim == 128 ? chunk_launch<128>(cache, sp, stream) : chunk_launch<256>(cache, sp, stream);
}

}  // namespace nvfp4
