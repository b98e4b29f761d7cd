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
//   last warp       issues the MMAs: S = Q K^T (both from shared memory,
//                   K-major), O += P V (P from tensor memory, V MN-major)
//
// The tensor pipe alternates between the row tiles: P V and the next Q K^T of
// one run while the softmax of the other does.
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
constexpr int kMeta = 4;       // tiles whose references are kept
constexpr int kHeadroom = 8;   // value scales may exceed their reference by 2^8 before it is raised
constexpr int kLiftK = 13, kLiftV = 5;  // largest elements: 6 * 2^13

template <int D>
struct Chunk {
  static constexpr int C = D / 32;
  static constexpr int kNQ = D == 256 ? 1 : 2;
  static constexpr int kTK = D == 256 ? 64 : 128;
  static constexpr int kQBytes = 128 * D * 2;         // one row tile
  static constexpr int kKvBytes = kTK * D * 2;        // one decoded tile of K or V
  static constexpr int kWarpD = kNQ * 4, kWarpMma = kWarpD + 4;
  static constexpr int kThreads = (kWarpMma + 1) * 32;
  static constexpr int kPart = D * kTK / 128;         // elements of a decoding thread
  static constexpr int kSmem = kNQ * kQBytes + 4 * kKvBytes + 2048;
  static constexpr uint32_t kS = 0, kO = kNQ * kTK;   // tensor-memory columns: scores, outputs
  static constexpr uint32_t kTmem = 512;
  static_assert(kNQ * (kTK + D) <= 512, "tensor memory");
  static_assert(kSmem <= 232448, "shared memory");
};

// Small shared state behind the operands.
struct Shared {
  uint64_t q_full, done;
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint32_t tmem;
  int abort_flag;
  int32_t rk[kMeta];           // reference of the keys' scales
  int32_t rv[kMeta][8];        // of the values' scales by block, as the outputs have it from this tile on
  float vfac[kMeta][8];        // factor onto the outputs before this tile (2^(old - new reference))
  uint32_t raised[kMeta];      // warps whose factors are not all 1
  int32_t red[2][2][4][4];     // [parity][K, V][warp][block of the thread]: largest scale codes
  uint32_t nan_any[kMeta];     // a block of values holds NaN: the warps that met one
  uint32_t nan_bits[kMeta][8][4];  // [block][32 tokens]
};
static_assert(sizeof(Shared) <= 2048, "shared state");

__device__ __forceinline__ uint64_t desc_mn128(uint32_t saddr, uint32_t atom_bytes) {
  // MN-major, 128-byte swizzle: 64 elements x 8 rows of the contraction an
  // atom; next 64 elements atom_bytes on, next 8 rows 1,024 bytes on
  return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(atom_bytes >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
__device__ __forceinline__ uint64_t desc_k128(uint32_t saddr) {
  return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
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
  constexpr int C = T::C, kNQ = T::kNQ, kTK = T::kTK;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sq = smem;                          // [row tile][atom][128 rows][128 bytes]
  uint8_t* sk = sq + kNQ * T::kQBytes;         // [slot][atom][token][128 bytes]
  uint8_t* sv = sk + 2 * T::kKvBytes;
  Shared& sh = *reinterpret_cast<Shared*>(sv + 2 * T::kKvBytes);
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
    mbar_init(&sh.done, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.k_full[i], 4);
      mbar_init(&sh.k_empty[i], 1);
      mbar_init(&sh.v_full[i], 4);
      mbar_init(&sh.v_empty[i], 1);
      mbar_init(&sh.s_full[i], 2);
      mbar_init(&sh.p_full[i], 4);
      mbar_init(&sh.o_full[i], 1);
    }
    sh.abort_flag = 0;
    for (int i = 0; i < kMeta; ++i) sh.nan_any[i] = sh.raised[i] = 0;
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
    const uint32_t t_s = t_lane + T::kS + qt * kTK, t_o = t_lane + T::kO + qt * D;
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
      if (!wait(&sh.s_full[qt], j & 1)) {
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
      uint32_t w[kTK / 2];
      uint64_t sum;
      float top;
      const uint64_t c1p = pair_const(c1);
      auto weights = [&](auto masked) {
        const float sub = kWeightLog2 - (m == -INFINITY ? 0.0f : m);
        const uint64_t subp = pair_const(sub);
        sum = 0;
        top = -INFINITY;
#pragma unroll
        for (int c = 0; c < kTK; c += 32) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(t_s + c, v);
          tc_wait_ld();
          tmem_ld_fence_regs<32>(v);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float2 t = unpair(fma2(pair_of(v[i], v[i + 1]), c1p, subp));
            if constexpr (decltype(masked)::value) {
              if (c + i >= hi || (c + i < lo && c + i >= sk_)) t.x = -INFINITY;
              if (c + i + 1 >= hi || (c + i + 1 < lo && c + i + 1 >= sk_)) t.y = -INFINITY;
            }
            top = fmaxf(top, fmaxf(t.x, t.y));
            t.x = exp2_approx(t.x), t.y = exp2_approx(t.y);
            sum = add2(sum, pair_of(__float_as_uint(t.x), __float_as_uint(t.y)));
            w[(c + i) / 2] = f32_to_word<__half>(t.x, t.y);
          }
        }
        top -= sub;  // back to the score's logarithm
      };
      float alpha = 1.0f;
      bool raised = sh.raised[ms_] != 0;
#pragma unroll 1
      for (int attempt = 0; attempt < 2; ++attempt) {
        if (plain) weights(std::false_type{});
        else weights(std::true_type{});
        const bool raise = top > m + kLag;
        if (!__any_sync(0xFFFFFFFFu, raise) || attempt == 1) break;
        if (raise) {
          alpha = exp2_approx(m - top);
          l2.x *= alpha, l2.y *= alpha;
          m = top;
        }
        raised = true;
      }
      l2.x += unpair(sum).x, l2.y += unpair(sum).y;
      // s_full also says that the p v of the tile before is complete
      if (j > 0 && raised) {
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t v[16];
          asm volatile(
              "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
              : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
              : "r"(t_o + c)
              : "memory");
          tc_wait_ld();
          tmem_ld_fence_regs<16>(v);
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * (alpha * sh.vfac[ms_][c / 32]));
          tmem_st_x16(t_o + c, v);
        }
      }
#pragma unroll
      for (int c = 0; c < kTK / 2; c += 16) tmem_st_x16(t_s + c, reinterpret_cast<const uint32_t(&)[16]>(w[c]));
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_full[qt]);
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
        tmem_ld_32x32b_x32(t_o + c, v);
        tc_wait_ld();
        tmem_ld_fence_regs<32>(v);
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
  } else if (warp < T::kWarpMma) {
    // ------------------------------------------------------------ decoding
    const int t = int(threadIdx.x) - T::kWarpD * 32, dw = t >> 5;
    const int tok = t % kTK, part = t / kTK;        // the token, and the thread's share of its rows
    constexpr int kWords = T::kPart / 32;           // blocks of a share
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
      const int64_t pg = min(max(page, 0), int32_t(a.pages) - 1);
      const int64_t rowi = ((pg * a.kv_heads + head) << a.page_shift) + (at & ((1 << a.page_shift) - 1));
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint8_t* src = (kv ? v_codes : k_codes) + rowi * (D / 2) + part * (T::kPart / 2);
        const uint8_t* s = (kv ? a.v_scales : a.k_scales) + rowi * C + part * kWords;
#pragma unroll
        for (int i = 0; i < kWords; ++i)
          raw[kv][i] = in ? *reinterpret_cast<const uint4*>(src + 16 * i) : make_uint4(0, 0, 0, 0);
        sc[kv] = 0;
        if (in) {
          if constexpr (kWords == 2) sc[kv] = *reinterpret_cast<const uint16_t*>(s);
          else sc[kv] = *reinterpret_cast<const uint32_t*>(s);
        }
      }
    };
    int32_t page = page_of(0);
    int32_t rv[kWords];  // the references of the thread's value blocks
#pragma unroll
    for (int i = 0; i < kWords; ++i) rv[i] = -1;
    bool dead = false;  // a wait ran out: the loop goes on, for the barrier of the group, without its work
    fetch(0, page);
    page = page_of(1);
    for (int j = 0; j < n; ++j) {
      const int slot = j & 1, meta = j & (kMeta - 1);
      // this tile's codes make room for the next tile's, whose loads take as
      // long as the decoding
      uint4 cur[2][kWords];
#pragma unroll
      for (int i = 0; i < kWords; ++i) cur[0][i] = raw[0][i], cur[1][i] = raw[1][i];
      // the largest finite scales of the tile, by block
      int32_t ref[2][kWords];
      const uint32_t scale[2] = {sc[0], sc[1]};
      fetch(j + 1, page);
      page = page_of(j + 2);
      bool nan = false;
#pragma unroll
      for (int i = 0; i < kWords; ++i)
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int32_t e = (scale[kv] >> (8 * i)) & 0xFF;
          nan = nan || (kv == 1 && e == 255);
          const int32_t mx = __reduce_max_sync(0xFFFFFFFFu, e == 255 ? 0 : e);
          if (lane == 0) sh.red[slot][kv][dw][i] = mx;
          ref[kv][i] = mx;
        }
      asm volatile("bar.sync 1, 128;" ::: "memory");
      // values: running references, raised only when the headroom is used up
      bool up = false;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        // the warps that hold the same share of the rows
#pragma unroll
        for (int w = 0; w < 4; ++w)
          if (w / (kTK / 32) == part) ref[1][i] = max(ref[1][i], sh.red[slot][1][w][i]);
        float fac = 1.0f;
        if (rv[i] < 0) {
          rv[i] = ref[1][i];
        } else if (ref[1][i] > rv[i] + kHeadroom) {
          fac = pow2i(rv[i] - ref[1][i]);
          rv[i] = ref[1][i];
          up = true;
        }
        ref[1][i] = rv[i] - kLiftV;
        if (tok == 0) {
          sh.vfac[meta][part * kWords + i] = fac;
          sh.rv[meta][part * kWords + i] = rv[i];
        }
        const uint32_t bits = __ballot_sync(0xFFFFFFFFu, ((scale[1] >> (8 * i)) & 0xFF) == 255u);
        if (lane == 0) sh.nan_bits[meta][part * kWords + i][tok / 32] = bits;
      }
      const bool any = __any_sync(0xFFFFFFFFu, nan);
      if (lane == 0) {
        // a bit a warp: no warp waits for another here
        const uint32_t bit = 1u << dw;
        if (any) atomicOr(&sh.nan_any[meta], bit);
        else atomicAnd(&sh.nan_any[meta], ~bit);
        if (up) atomicOr(&sh.raised[meta], bit);
        else atomicAnd(&sh.raised[meta], ~bit);
      }
      {
        int32_t mx = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int i = 0; i < kWords; ++i) mx = max(mx, sh.red[slot][0][w][i]);
        if (t == 0) sh.rk[meta] = mx;
#pragma unroll
        for (int i = 0; i < kWords; ++i) ref[0][i] = mx - kLiftK;
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if (!dead && !wait(kv ? &sh.v_empty[slot] : &sh.k_empty[slot], ((j >> 1) & 1) ^ 1)) dead = true;
        if (!dead) {
          uint8_t* dst = (kv ? sv : sk) + slot * T::kKvBytes + tok * 128;
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            const int32_t e = (scale[kv] >> (8 * i)) & 0xFF;
            const float f = __uint_as_float(uint32_t(max(e - ref[kv][i] + 127, 0)) << 23);
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
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(kv ? &sh.v_full[slot] : &sh.k_full[slot]);
        }
      }
    }
  } else if (lane == 0) {
    // ------------------------------------------------------------ MMA issue
    constexpr uint32_t kIdS = (1u << 4) | (uint32_t(kTK >> 3) << 17) | (8u << 24);               // M = 128, N = kTK
    constexpr uint32_t kIdO = (1u << 4) | (1u << 16) | (uint32_t(D >> 3) << 17) | (8u << 24);    // N = D, B MN-major
    auto wait1 = [&](uint64_t* bar, uint32_t parity) -> bool {
      if (mbar_wait_bounded(bar, parity, a.wait_limit_cycles, abort_flag)) return true;
      sh.abort_flag = 1;
      return false;
    };
    auto scores = [&](int qt, int j) {
      const uint32_t qa = smem_u32(sq + qt * T::kQBytes), kb = smem_u32(sk + (j & 1) * T::kKvBytes);
#pragma unroll
      for (int d = 0; d < D; d += 16)
        mma_ss(tmem + T::kS + qt * kTK, desc_k128(qa + (d / 64) * (128 * 128)) + (d % 64) / 8,
               desc_k128(kb + (d / 64) * (kTK * 128)) + (d % 64) / 8, kIdS, d > 0);
      tc_commit(&sh.s_full[qt]);
      mbar_arrive(&sh.s_full[qt]);  // hands on what the decoders wrote for the softmax
    };
    bool ok = n > 0 && wait1(&sh.q_full, 0) && wait1(&sh.k_full[0], 0) && wait1(&sh.v_full[0], 0);
    tc_fence_after();
    if (ok) {
      for (int qt = 0; qt < kNQ; ++qt) scores(qt, 0);
      tc_commit(&sh.k_empty[0]);
    }
    for (int j = 0; j < n && ok; ++j) {
      const uint32_t vb = smem_u32(sv + (j & 1) * T::kKvBytes);
      for (int qt = 0; qt < kNQ && ok; ++qt) {
        if (!(ok = wait1(&sh.p_full[qt], j & 1))) break;
        tc_fence_after();
#pragma unroll
        for (int t = 0; t < kTK; t += 16)
          mma_ts(tmem + T::kO + qt * D, tmem + T::kS + qt * kTK + t / 2, desc_mn128(vb, kTK * 128) + t * 8, kIdO,
                 (j > 0 || t > 0) ? 1u : 0u);
        if (qt == kNQ - 1) tc_commit(&sh.v_empty[j & 1]);
        if (j + 1 < n) {
          if (qt == 0) {
            const uint32_t ph = ((j + 1) >> 1) & 1;
            if (!(ok = wait1(&sh.k_full[(j + 1) & 1], ph) && wait1(&sh.v_full[(j + 1) & 1], ph))) break;
            tc_fence_after();
          }
          scores(qt, j + 1);
          if (qt == kNQ - 1) tc_commit(&sh.k_empty[(j + 1) & 1]);
        } else {
          tc_commit(&sh.o_full[qt]);
        }
      }
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
