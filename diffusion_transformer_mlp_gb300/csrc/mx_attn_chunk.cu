// Attention of many query rows over the paged MXFP4 cache (taking in a
// prompt by chunks) on tcgen05.
//
// A row is a (query, head of the group) pair: the heads that share a kv head
// are rows of one tile, so the cache is decoded once for all of them.  A CTA
// takes kNQ tiles of 128 rows of one (sequence, kv head) and walks the keys
// that they see in tiles of kTK:
//
//   warps 0-3, 4-7  softmax of row tile 0, 1: a thread is a row.  Scores come
//                   from tensor memory, the weights go back there as FP16 over
//                   the scores they came from (the A operand of p v)
//   four warps      decode the tile's keys and values to FP16 in shared memory:
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
// latency (128 keys and one buffer: 4,300 cycles for 128 keys of both row
// tiles; one issuing thread for both was slower still).
//
// FP16 operands are exact: a code times 2^(E - R + 13), R the tile's largest
// key scale (its power of two goes onto the scores), is exact for E >= R - 36,
// and a code times 2^(E - R + 5), R a running reference of the value scales of
// its block column (its power of two goes onto the output's columns), for E >=
// R - 28.  Q is scaled by a power of two per row.  Weights are held times 2^10 against a reference that lags the
// running maximum by up to 2^5, so that the output is rarely rescaled (an
// 11-bit rounding; sums and statistics in FP32).
#include <algorithm>
#include <atomic>
#include <string>
#include <type_traits>

#include "mx_attn.cuh"

namespace nvfp4 {
namespace {

constexpr float kWeightLog2 = 10.0f;
constexpr float kLag = 5.0f;
constexpr int kMeta = 8;       // tiles whose references are kept: the decoders are up to 6 ahead of the softmax
constexpr int kTK = 64;        // keys of a tile
constexpr int kHeadroom = 8;   // value scales may exceed their reference by 2^8 before it is raised
constexpr int kLiftK = 13, kLiftV = 5;  // largest elements: 6 * 2^13

template <int D>
struct Chunk {
  static constexpr int C = D / 32;
  static constexpr int kNQ = D == 256 ? 1 : 2;
  static constexpr int kSlots = D == 256 ? 2 : 4;     // decoded tiles
  static constexpr int kQBytes = 128 * D * 2;         // one row tile
  static constexpr int kKvBytes = kTK * D * 2;        // one decoded tile of K or V
  static constexpr int kWarpD = kNQ * 4, kWarpR = kWarpD + 4, kWarpMma = kWarpR + 1;
  static constexpr int kThreads = (kWarpMma + kNQ) * 32;
  static constexpr int kPart = D * kTK / 128;         // elements of a decoding thread
  static constexpr int kSmem = kNQ * kQBytes + 2 * kSlots * kKvBytes + 4096;
  static constexpr uint32_t kS = 0, kO = kNQ * 2 * kTK;  // tensor-memory columns: scores, outputs
  static constexpr uint32_t kTmem = 512;
  static_assert(kNQ * (2 * kTK + D) <= 512, "tensor memory");
  static_assert(kSmem <= 232448, "shared memory");
};

// Small shared state behind the operands.
struct Shared {
  uint64_t q_full, done;
  uint64_t ref_full[4], kv_full[4], kv_empty[4];  // by slot: references, decoded tile, both row tiles' p v complete
  uint64_t s_full[2][2], p_full[2][2];            // by row tile and score buffer
  uint64_t o_full[2];                             // p v of the last tile is complete
  uint32_t tmem;
  int abort_flag;
  int32_t rk[kMeta];           // reference of the keys' scales
  int32_t rv[kMeta][8];        // of the values' scales by block, as the outputs have it from this tile on
  float vfac[kMeta][8];        // factor onto the outputs before this tile (2^(old - new reference))
  uint32_t raised[kMeta];      // the factors are not all 1
  uint32_t nan_any[kMeta];     // a block of values holds NaN
  uint32_t nan_bits[kMeta][8][kTK / 32];  // [block][32 tokens]
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
// Pairs of binary32 in 64 bits.  A pair of equal constants is made once, by a
// volatile move: left to the compiler it is made again at every use.
__device__ __forceinline__ uint64_t pair_const(float v) {
  uint64_t r;
  asm volatile("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ uint64_t pair_of(uint32_t x, uint32_t y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <int D>
__global__ void __launch_bounds__(Chunk<D>::kThreads, 1)
    k_attn_chunk(const uint8_t* __restrict__ k_codes, const uint8_t* __restrict__ v_codes,
                 const __grid_constant__ AttnParams a) {
  using T = Chunk<D>;
  constexpr int C = T::C, kNQ = T::kNQ, kSlots = T::kSlots;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sq = smem;                          // [row tile][atom][128 rows][128 bytes]
  uint8_t* sk = sq + kNQ * T::kQBytes;         // [slot][atom][token][128 bytes]
  uint8_t* sv = sk + kSlots * T::kKvBytes;
  Shared& sh = *reinterpret_cast<Shared*>(sv + kSlots * T::kKvBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_wait();

  const int b = blockIdx.z, head = blockIdx.y;
  const int32_t len = a.lens[b];
  const int32_t q0 = a.q_starts != nullptr ? a.q_starts[b] : b;
  const int32_t nq = a.q_starts != nullptr ? a.q_starts[b + 1] - q0 : 1;
  const int32_t rows = nq * a.group;
  // the last rows see the most keys: they come first
  const int32_t pairs = (rows + 128 * kNQ - 1) / (128 * kNQ);
  const int32_t pair = pairs - 1 - int32_t(blockIdx.x);
  if (pair < 0) return;
  const int32_t row0 = pair * 128 * kNQ;
  const int32_t last = min(row0 + 128 * kNQ, rows) - 1;
  const Span span = span_of(a, len, nq, row0 / a.group, last / a.group, kTK);

  if (threadIdx.x == 0) {
    mbar_init(&sh.q_full, kNQ * 4);
    mbar_init(&sh.done, kNQ);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh.ref_full[i], 1);
      mbar_init(&sh.kv_full[i], 4);
      mbar_init(&sh.kv_empty[i], kNQ);
      mbar_init(&sh.s_full[i >> 1][i & 1], 2);
      mbar_init(&sh.p_full[i >> 1][i & 1], 4);
    }
    mbar_init(&sh.o_full[0], 1);
    mbar_init(&sh.o_full[1], 1);
    sh.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == T::kWarpMma) tmem_alloc(&sh.tmem, T::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const volatile int* abort_flag = &sh.abort_flag;
  const int n = span.n;
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
    const int32_t row = row0 + qt * 128 + r;
    const bool real = row < rows;
    const int32_t qi = real ? row / a.group : 0, hq = head * a.group + (real ? row - qi * a.group : 0);
    const int32_t pos = len - nq + qi;
    // the row sees keys j < end with j >= from or j < sinks
    const int32_t end = !real ? 0 : (a.causal ? min(len, pos + 1) : len);
    const int32_t from = a.window > 0 ? pos - a.window + 1 : 0;
    const uint32_t t_lane = tmem + (uint32_t(q * 32) << 16);
    const uint32_t t_o = t_lane + T::kO + qt * D;
    // Q: the row's largest element goes to [2^13, 2^14), the sign of the
    // softmax scale onto the elements
    float qf;
    {
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + int64_t(q0 + qi) * a.q_st + int64_t(hq) * a.q_sh;
      // up to 128 elements at a time, their loads all in flight; the row twice,
      // for its largest element and for the conversion, unless it fits
      constexpr int kRound = D < 128 ? D : 128;
      uint32_t w[kRound / 2];
      auto load = [&](int d0) {
#pragma unroll
        for (int i = 0; i < kRound / 8; ++i) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (real) {
            const uint16_t* e = src + d0 + 8 * i;
            if (a.q_vec) {
              v = *reinterpret_cast<const uint4*>(e);
            } else {
              v.x = uint32_t(e[0]) | uint32_t(e[1]) << 16, v.y = uint32_t(e[2]) | uint32_t(e[3]) << 16;
              v.z = uint32_t(e[4]) | uint32_t(e[5]) << 16, v.w = uint32_t(e[6]) | uint32_t(e[7]) << 16;
            }
          }
          w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
      };
      auto value = [&](uint32_t x) { return a.bf16 ? word_to_f32<__nv_bfloat16>(x) : word_to_f32<__half>(x); };
      float am = 0.0f;
#pragma unroll 1
      for (int d0 = 0; d0 < D; d0 += kRound) {
        load(d0);
#pragma unroll
        for (int i = 0; i < kRound / 2; ++i) {
          const float2 t = value(w[i]);
          am = max_nan(am, max_nan(fabsf(t.x), fabsf(t.y)));
        }
      }
      const int32_t eb = int32_t(__float_as_uint(am) >> 23) & 0xFF;
      const int32_t up = (eb == 0 || eb == 255) ? 0 : min(126, 140 - eb);
      const float mul = a.scale_log2 < 0.0f ? -pow2i(up) : pow2i(up);
      qf = fabsf(a.scale_log2) * pow2i(-up);
      uint8_t* dst = sq + qt * T::kQBytes + r * 128;
#pragma unroll 1
      for (int d0 = 0; d0 < D; d0 += kRound) {
        if (kRound < D) load(d0);
#pragma unroll
        for (int i = 0; i < kRound / 8; ++i) {
          uint32_t h[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float2 t = value(w[4 * i + x]);
            h[x] = f32_to_word<__half>(t.x * mul, t.y * mul);
          }
          const int d = d0 + 8 * i;
          *reinterpret_cast<uint4*>(dst + (d / 64) * (128 * 128) + ((((d % 64) / 8) ^ (r & 7)) << 4)) =
              make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full);
    }

    float m = -INFINITY;
    float2 l2 = make_float2(0.0f, 0.0f);
    uint32_t nan_cols = 0;  // blocks of the output that are NaN
    int last_meta = 0;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const uint32_t t_s = t_lane + T::kS + (qt * 2 + (j & 1)) * kTK;
      if (!wait(&sh.s_full[qt][j & 1], (j >> 1) & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int ms_ = j & (kMeta - 1);
      const int32_t tok0 = span.tile(j) * kTK;
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
              const int x = 32 * c + i;
              if (x >= hi || (x < lo && x >= sk_)) t.x = -INFINITY;
              if (x + 1 >= hi || (x + 1 < lo && x + 1 >= sk_)) t.y = -INFINITY;
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
          raised = true;
          return false;
        }
        l2.x = l2.x * alpha + unpair(sum).x, l2.y = l2.y * alpha + unpair(sum).y;
        if (j > 0 && raised) {
          // The p v of the tile before has to be complete (its slot is filled
          // again only after the weights of this tile).
          if (!wait(&sh.kv_empty[(j - 1) % kSlots], ((j - 1) / kSlots) & 1)) return true;
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
      if (lane == 0) mbar_arrive(&sh.p_full[qt][j & 1]);
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
    // ---- output
    if (ok && n > 0) ok = wait(&sh.o_full[qt], 0);
    tc_fence_after();
    const float l = l2.x + l2.y;
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
    if (ok) {
      uint16_t* dst = static_cast<uint16_t*>(a.out) + int64_t(q0 + qi) * a.o_st + int64_t(hq) * a.o_sh;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t v[32];
        tmem_load32(t_o + c, v);
        const bool nan = (nan_cols >> (c / 32)) & 1u;
        const float fac = l == 0.0f ? 0.0f : pow2i(sh.rv[last_meta][c / 32] - 127 - kLiftV) * inv;
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          uint32_t w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            // nothing seen: tensor memory may hold anything
            float e0 = l == 0.0f ? 0.0f : __uint_as_float(v[i + 2 * x]) * fac;
            float e1 = l == 0.0f ? 0.0f : __uint_as_float(v[i + 2 * x + 1]) * fac;
            if (nan) e0 = e1 = __uint_as_float(0x7FFFFFFFu);
            w[x] = a.bf16 ? f32_to_word<__nv_bfloat16>(e0, e1) : f32_to_word<__half>(e0, e1);
          }
          if (real) {
            if (a.o_vec) {
              *reinterpret_cast<uint4*>(dst + c + i) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                dst[c + i + 2 * x] = uint16_t(w[x]);
                dst[c + i + 2 * x + 1] = uint16_t(w[x] >> 16);
              }
            }
          }
        }
      }
      if (real && a.lse != nullptr)
        a.lse[int64_t(q0 + qi) * (a.kv_heads * a.group) + hq] =
            l == 0.0f ? -INFINITY : (m - kWeightLog2 + log2f(l)) * 0.6931471805599453f;
    }
    tc_fence_before();
  } else if (warp < T::kWarpR) {
    // ------------------------------------------------------------ decoding
    const int t = int(threadIdx.x) - T::kWarpD * 32;
    const int tok = t % kTK, part = t / kTK;  // the token, and the thread's share of its rows
    constexpr int kWords = T::kPart / 32;     // blocks of a share
    const int32_t* table = a.table + int64_t(b) * a.table_ld;
    auto page_of = [&](int j) -> int32_t {
      const int32_t at = span.tile(j) * kTK + tok;
      return j < n && at < span.hi ? table[min(at >> a.page_shift, int32_t(a.table_ld) - 1)] : 0;
    };
    uint4 raw[2][kWords];  // codes of K and V
    uint32_t sc[2] = {0, 0};
    auto fetch = [&](int j, int32_t page) {
      const int32_t at = span.tile(j) * kTK + tok;
      const bool in = j < n && at < span.hi;
      const int32_t z = min(max(page, 0), int32_t(a.pages) - 1) * a.kv_heads + head;
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
      const int slot = j % kSlots, meta = j & (kMeta - 1);
      const uint32_t ph = (j / kSlots) & 1;
      // this tile's codes make room for the next tile's, whose loads take as
      // long as the decoding
      uint4 cur[2][kWords];
#pragma unroll
      for (int i = 0; i < kWords; ++i) cur[0][i] = raw[0][i], cur[1][i] = raw[1][i];
      const uint32_t scale[2] = {sc[0], sc[1]};
      fetch(j + 1, page);
      page = page_of(j + 2);
      // the references come after their writer has seen the slot empty
      if (!wait(&sh.ref_full[slot], ph) || !wait(&sh.kv_empty[slot], ph ^ 1)) break;
      const int32_t rk = sh.rk[meta] - kLiftK;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        uint8_t* dst = (kv ? sv : sk) + slot * T::kKvBytes + tok * 128;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          const int32_t e = (scale[kv] >> (8 * i)) & 0xFF;
          const int32_t ref = kv ? sh.rv[meta][part * kWords + i] - kLiftV : rk;
          const float f = __uint_as_float(uint32_t(max(e - ref + 127, 0)) << 23);
          uint32_t fw = f32_to_word<__half>(f, f);
          if (e == 255) fw = kv ? 0u : 0x7FFF7FFFu;
          const uint32_t w[4] = {cur[kv][i].x, cur[kv][i].y, cur[kv][i].z, cur[kv][i].w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t h[4];
            e2m1x8_to_half(w[x], h);
            const int d = part * T::kPart + i * 32 + x * 8;
            *reinterpret_cast<uint4*>(dst + (d / 64) * (kTK * 128) + ((((d % 64) / 8) ^ (tok & 7)) << 4)) =
                make_uint4(hmul2(h[0], fw), hmul2(h[1], fw), hmul2(h[2], fw), hmul2(h[3], fw));
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.kv_full[slot]);
    }
  } else if (warp == T::kWarpR) {
    // ------------------------------------------------------------ references
    // a lane takes kTK / 32 tokens of each tile; the loads of kBatch tiles are
    // in flight together, ahead of the batch that is worked off, and the pages
    // are looked up a batch before that
    constexpr int kPer = kTK / 32, kW = (C + 3) / 4, kBatch = 4;
    const int32_t* table = a.table + int64_t(b) * a.table_ld;
    uint32_t kw[kBatch][kPer][kW], vw[kBatch][kPer][kW];
    int32_t pages[kBatch][kPer];
    auto look_up = [&](int j0) {
#pragma unroll
      for (int x = 0; x < kBatch; ++x)
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int32_t at = span.tile(j0 + x) * kTK + i * 32 + lane;
          pages[x][i] =
              j0 + x < n && at < span.hi ? table[min(at >> a.page_shift, int32_t(a.table_ld) - 1)] : 0;
        }
    };
    auto fetch = [&](int j0) {
#pragma unroll
      for (int x = 0; x < kBatch; ++x)
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int32_t at = span.tile(j0 + x) * kTK + i * 32 + lane;
          const bool in = j0 + x < n && at < span.hi;
          const int32_t z = min(max(pages[x][i], 0), int32_t(a.pages) - 1) * a.kv_heads + head;
          const int64_t at_s = ((int64_t(z) << a.page_shift) + (at & ((1 << a.page_shift) - 1))) * C;
#pragma unroll
          for (int y = 0; y < kW; ++y) {
            kw[x][i][y] = vw[x][i][y] = 0;
            if (in) {
              if constexpr (C == 2) {
                kw[x][i][0] = *reinterpret_cast<const uint16_t*>(a.k_scales + at_s);
                vw[x][i][0] = *reinterpret_cast<const uint16_t*>(a.v_scales + at_s);
              } else {
                kw[x][i][y] = *reinterpret_cast<const uint32_t*>(a.k_scales + at_s + 4 * y);
                vw[x][i][y] = *reinterpret_cast<const uint32_t*>(a.v_scales + at_s + 4 * y);
              }
            }
          }
        }
    };
    int32_t rv[C];
#pragma unroll
    for (int c = 0; c < C; ++c) rv[c] = -1;
    look_up(0);
    fetch(0);
    look_up(kBatch);
    bool ok = true;
    for (int j0 = 0; j0 < n && ok; j0 += kBatch) {
      int32_t mk[kBatch], mv[kBatch][C];
      uint32_t nan[kBatch][C][kPer];
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        mk[x] = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          mv[x][c] = 0;
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int32_t ek = (kw[x][i][c / 4] >> (8 * (c % 4))) & 0xFF;
            const int32_t ev = (vw[x][i][c / 4] >> (8 * (c % 4))) & 0xFF;
            mk[x] = max(mk[x], ek == 255 ? 0 : ek);
            mv[x][c] = max(mv[x][c], ev == 255 ? 0 : ev);
            nan[x][c][i] = __ballot_sync(0xFFFFFFFFu, ev == 255);
          }
        }
      }
      fetch(j0 + kBatch);
      look_up(j0 + 2 * kBatch);
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        const int j = j0 + x;
        if (j >= n || !ok) break;
        const int slot = j % kSlots, meta = j & (kMeta - 1);
        const int32_t top_k = __reduce_max_sync(0xFFFFFFFFu, mk[x]);
        uint32_t up = 0, any = 0;
        float fac[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
          // values: running references, raised only when the headroom is used up
          const int32_t top_v = __reduce_max_sync(0xFFFFFFFFu, mv[x][c]);
          fac[c] = 1.0f;
          if (rv[c] < 0) {
            rv[c] = top_v;
          } else if (top_v > rv[c] + kHeadroom) {
            fac[c] = pow2i(rv[c] - top_v);
            rv[c] = top_v;
            up = 1;
          }
#pragma unroll
          for (int i = 0; i < kPer; ++i) any |= nan[x][c][i];
        }
        // whoever used this place kMeta tiles ago is done once the slot is empty
        ok = wait(&sh.kv_empty[slot], ((j / kSlots) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) {
          sh.rk[meta] = top_k;
          sh.raised[meta] = up;
          sh.nan_any[meta] = any;
#pragma unroll
          for (int c = 0; c < C; ++c) {
            sh.rv[meta][c] = rv[c];
            sh.vfac[meta][c] = fac[c];
#pragma unroll
            for (int i = 0; i < kPer; ++i) sh.nan_bits[meta][c][i] = nan[x][c][i];
          }
          mbar_arrive(&sh.ref_full[slot]);
        }
        __syncwarp();
      }
    }
  } else if (lane == 0) {
    // ------------------------------------------------------------ MMA issue
    constexpr uint32_t kIdS = (1u << 4) | (uint32_t(kTK >> 3) << 17) | (8u << 24);               // M = 128, N = kTK
    constexpr uint32_t kIdO = (1u << 4) | (1u << 16) | (uint32_t(D >> 3) << 17) | (8u << 24);    // N = D, B MN-major
    const int qt = warp - T::kWarpMma;
    auto wait1 = [&](uint64_t* bar, uint32_t parity) -> bool {
      if (mbar_wait_bounded(bar, parity, a.wait_limit_cycles, abort_flag)) return true;
      sh.abort_flag = 1;
      return false;
    };
    const uint32_t q_lo = desc_lo(smem_u32(sq + qt * T::kQBytes), 16), k_lo = desc_lo(smem_u32(sk), 16),
                   v_lo = desc_lo(smem_u32(sv), kTK * 128);
    const uint32_t t_q = tmem + T::kS + qt * 2 * kTK, t_o = tmem + T::kO + qt * D;
    auto scores = [&](int j) -> bool {
      const int slot = j % kSlots;
      if (!wait1(&sh.kv_full[slot], (j / kSlots) & 1)) return false;
      tc_fence_after();
      const uint32_t kb = k_lo + uint32_t(slot) * (T::kKvBytes >> 4), t_s = t_q + (j & 1) * kTK;
#pragma unroll
      for (int d = 0; d < D; d += 16)
        mma_ss(t_s, q_lo + (d / 64) * (128 * 128 >> 4) + (d % 64) / 8, kb + (d / 64) * (kTK * 128 >> 4) + (d % 64) / 8,
               kIdS, d > 0);
      tc_commit(&sh.s_full[qt][j & 1]);
      mbar_arrive(&sh.s_full[qt][j & 1]);  // hands on what the decoders wrote for the softmax
      return true;
    };
    bool ok = n > 0 && wait1(&sh.q_full, 0) && scores(0) && (n == 1 || scores(1));
    for (int j = 0; j < n && ok; ++j) {
      if (!(ok = wait1(&sh.p_full[qt][j & 1], (j >> 1) & 1))) break;
      tc_fence_after();
      const uint32_t vb = v_lo + uint32_t(j % kSlots) * (T::kKvBytes >> 4), t_p = t_q + (j & 1) * kTK;
#pragma unroll
      for (int t = 0; t < kTK; t += 16) mma_ts(t_o, t_p + t / 2, vb + t * 8, kIdO, j > 0 || t > 0);
      tc_commit(&sh.kv_empty[j % kSlots]);
      if (j + 1 == n) tc_commit(&sh.o_full[qt]);
      if (j + 2 < n) ok = scores(j + 2);  // into the buffer that p v has read
    }
    tc_commit(&sh.done);
    if (!mbar_wait_bounded(&sh.done, 0, a.wait_limit_cycles, nullptr)) sh.abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && sh.abort_flag && a.dev_status != nullptr)
    atomicExch(a.dev_status, static_cast<uint32_t>(NVFP4_ETIMEOUT));
  if (warp == T::kWarpMma) {
    __syncwarp();
    tmem_dealloc(tmem, T::kTmem);
  }
}

template <int D>
nvfp4_status chunk_launch(const mxfp4_cache* cache, const AttnParams& p, int32_t max_queries, cudaStream_t stream) {
  using T = Chunk<D>;
  auto kern = k_attn_chunk<D>;
  static std::atomic<uint64_t> ready{0};
  nvfp4_status st = allow_smem(reinterpret_cast<const void*>(kern), T::kSmem, ready);
  if (st != NVFP4_OK) return st;
  const int64_t pairs = (int64_t(max_queries) * p.group + 128 * T::kNQ - 1) / (128 * T::kNQ);
  AttnParams q = p;
  for (int32_t b = 0; b < p.seqs; b += 65535) {  // the grid's z
    q.seqs = std::min(65535, p.seqs - b);
    q.table = p.table + int64_t(b) * p.table_ld;
    q.lens = p.lens + b;
    if (p.q_starts != nullptr) q.q_starts = p.q_starts + b;
    st = launch("launch k_attn_chunk", kern, dim3(unsigned(pairs), unsigned(p.kv_heads), unsigned(q.seqs)),
                dim3(T::kThreads), T::kSmem, 0, stream, static_cast<const uint8_t*>(cache->k_codes),
                static_cast<const uint8_t*>(cache->v_codes), q);
    if (st != NVFP4_OK) return st;
  }
  return NVFP4_OK;
}

}  // namespace

nvfp4_status attn_chunk(const mxfp4_cache* cache, const AttnParams& p, int32_t max_queries, cudaStream_t stream) {
  if (cache->dim == 64) return chunk_launch<64>(cache, p, max_queries, stream);
  if (cache->dim == 128) return chunk_launch<128>(cache, p, max_queries, stream);
  return chunk_launch<256>(cache, p, max_queries, stream);
}

}  // namespace nvfp4
