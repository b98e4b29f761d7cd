// MXFP4 product for few rows: out [m, n] = A [m, k] W [n, k]^T on tcgen05.
//
// With few rows the weight's bytes are the work (17/32 byte an element), so
// the weight is the tensor core's M operand: a CTA takes 128 weight rows and
// up to 128 activation rows (the MMA's N: 16, 32, 64 or 128), streams its
// weight rows through a TMA ring and accumulates D[weight row][activation
// row] in tensor memory with kind::mxf4 MMAs (block 32, E8M0 scales), which
// read the 4-bit codes and the scales as stored: nothing is decoded.
//
//   warp 0      TMA producer: a k-tile of 256 elements is a 128-byte swizzled
//               box of each operand and one 1 KB piece of each scale array
//               (two 512-byte tiles of 128 rows x 4 scale columns)
//   warp 1      MMA issuer: per k-tile four tcgen05.cp (the scale tiles into
//               tensor memory) and four MMAs of K = 64
//   warps 2-5   epilogue: a lane is one weight row, so stores run along n
//
// For up to 32 rows mxfp4_linear hands over x itself: warps 2-5 quantise each
// k-tile of it into the ring (a block of 32 a lane), which costs less than a
// kernel of its own and its launch.
//
// One weight tile per 128 rows fills few SMs (42 tiles at n = 5,376), so k is
// split over the CTAs of a cluster: each leaves its float32 partial in its
// shared memory and sums the columns it owns over the cluster in rank order.
// The split depends on the shape alone, so results are reproducible.  Bound by
// the weight's bytes and, at these sizes, by latency: 5,376 x 14,336 (41 MB) in
// 10.2 us for 8 rows, 4.0 TB/s, and in 11.7 us for 64 rows.
#include <algorithm>
#include <atomic>
#include <string>

#include "mx_gemm.cuh"

namespace nvfp4 {
namespace {

constexpr int kThreads = 192;
constexpr int kWRows = 128;
constexpr int kWBytes = kWRows * 128;  // one k-tile of the weight
constexpr int kSfBytes = 1024;         // one k-tile of one scale array
constexpr int kMaxSplit = 8;           // portable cluster size
constexpr uint32_t kSfSlots = 2;       // scale columns alternate between two places
constexpr uint32_t kSfCols = 16;       // of one k-tile: 2 x 4 columns for W, 2 x 4 for A

template <int NT>
struct Shape {
  static constexpr int kABytes = NT * 128;
  static constexpr int kStage = kWBytes + kABytes + 2 * kSfBytes;
  // two CTAs an SM: 5 x 20, 5 x 22, 4 x 26 and 3 x 34 KB
  static constexpr int kStages = NT <= 32 ? 5 : (NT == 64 ? 4 : 3);
  static constexpr int kSmem = 1024 + kStages * kStage + 256;
  static constexpr uint32_t kTmem = NT <= 32 ? 64u : (NT == 64 ? 128u : 256u);
  static_assert(NT + kSfSlots * kSfCols <= kTmem, "tensor memory");
  static_assert(NT * 512 <= kStages * kStage, "the partial sums reuse the ring");
  static_assert(2 * (kSmem + 1024) <= 233472, "two CTAs an SM");
};

struct RowsParams {
  const uint8_t* a_s;
  const uint8_t* w_s;
  void* out;
  int64_t ldo;
  int32_t m, n, dtype;
  int32_t groups;   // 128-element groups of k
  int32_t split;    // CTAs of the cluster along k
  // kX only: the activation [m, k] before quantisation
  const void* x;
  int64_t ldx;
  int32_t k, x_vec;  // x_vec: rows are 16-byte aligned
  int32_t out_vec;   // four outputs of a row are one aligned store
  int32_t w_once;    // the weight is read by one row of CTAs only
  uint32_t* dev_status;
  uint64_t wait_limit_cycles;
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ uint64_t l2_policy_evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}

__device__ __forceinline__ void tma_load_2d_plain(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t x,
                                                  int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}

// Scale tile (32 lanes x 16 bytes, unswizzled) into 4 tensor-memory columns of
// all four lane quarters.
__device__ __forceinline__ void tc_cp_scales(uint32_t taddr, uint32_t saddr) {
  const uint64_t desc = uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(128 >> 4) << 32) |
                        (uint64_t(1) << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ void tc_mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void store_out(const RowsParams& p, int64_t row, int32_t col, float v) {
  const int64_t at = row * p.ldo + col;
  if (p.dtype == MXFP4_BF16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
  else if (p.dtype == MXFP4_FP16) static_cast<__half*>(p.out)[at] = __float2half_rn(v);
  else static_cast<float*>(p.out)[at] = v;
}

// Four consecutive outputs of a row.
__device__ __forceinline__ void store_out4(const RowsParams& p, int64_t row, int32_t col, float4 v) {
  if (p.out_vec && col + 4 <= p.n) {
    const int64_t at = row * p.ldo + col;
    if (p.dtype == MXFP4_FP32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = v;
    } else {
      const uint2 w = p.dtype == MXFP4_BF16
                          ? make_uint2(f32_to_word<__nv_bfloat16>(v.x, v.y), f32_to_word<__nv_bfloat16>(v.z, v.w))
                          : make_uint2(f32_to_word<__half>(v.x, v.y), f32_to_word<__half>(v.z, v.w));
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = w;
    }
    return;
  }
  const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (col + i < p.n) store_out(p, row, col + i, f[i]);
}

// 32 consecutive elements of a row of x, zeros past column k.
template <typename X>
struct RawBlock {
  static constexpr int kWords = 32 * sizeof(X) / 16;
  uint4 w[kWords];
  __device__ __forceinline__ void load(const RowsParams& p, int row, int col) {
    const X* src = static_cast<const X*>(p.x) + int64_t(row) * p.ldx + col;
    if (p.x_vec && col + 32 <= p.k) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint4*>(src)[i];
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < int(16 / sizeof(X)); ++e) {
          const int c = i * int(16 / sizeof(X)) + e;
          if (col + c < p.k) {
            if constexpr (sizeof(X) == 4) v[e] = reinterpret_cast<const uint32_t*>(src)[c];
            else v[e / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(src)[c]) << (16 * (e % 2));
          }
        }
        w[i] = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
  }
  __device__ __forceinline__ void values(float (&f)[32]) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(X) == 4) {
          f[4 * i + e] = __uint_as_float(v[e]);
        } else {
          const float2 t = word_to_f32<X>(v[e]);
          f[8 * i + 2 * e] = t.x, f[8 * i + 2 * e + 1] = t.y;
        }
      }
    }
  }
};

// kX: X is the element type of p.x, which warps 2-5 quantise; else X is
// ignored and the activation comes quantised through tmap_a and p.a_s.
template <int NT, bool kX, typename X>
__global__ void __launch_bounds__(kThreads, 2)
    k_mx_rows(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_w,
              const RowsParams p) {
  using S = Shape<NT>;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + S::kStages * S::kStage);
  uint64_t* empty = full + S::kStages;
  uint64_t* done = empty + S::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? int(cluster_ctarank()) : 0;
  const int w_row = (int(blockIdx.x) / p.split) * kWRows;
  const int a_row = int(blockIdx.y) * NT;
  const int tiles = (p.groups + 1) / 2;
  const int kt0 = int(int64_t(tiles) * rank / p.split), kt1 = int(int64_t(tiles) * (rank + 1) / p.split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], kX ? 5 : 1);  // the TMA's arrival, and one of each quantising warp
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    if constexpr (!kX) prefetch_tmap(&tmap_a);
    prefetch_tmap(&tmap_w);
  }
  if (warp == 1) tmem_alloc(tmem_slot, S::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_wait();

  if (warp == 0 && lane == 0) {
    const uint64_t once = l2_policy_evict_first();
    int slot = 0;
    uint32_t phase = 0;
    for (int kt = kt0; kt < kt1; ++kt) {
      if (!mbar_wait_bounded(&empty[slot], phase ^ 1u, p.wait_limit_cycles, const_cast<const int*>(abort_flag))) {
        *abort_flag = 1;
        // the copies under way: the phase of each stage that was filled last
        for (int i = 0; i < min(kt - kt0, S::kStages); ++i) {
          if (--slot < 0) slot = S::kStages - 1, phase ^= 1u;
          mbar_wait_bounded(&full[slot], phase, p.wait_limit_cycles, nullptr);
        }
        break;
      }
      uint8_t* st = ring + slot * S::kStage;
      // the last k-tile may hold one 128-element group only: the boxes are
      // zero-filled past the operand, the scale pieces are half as long
      const uint32_t sf = (2 * kt + 1 < p.groups) ? kSfBytes : kSfBytes / 2;
      mbar_arrive_expect_tx(&full[slot], kX ? kWBytes + sf : kWBytes + S::kABytes + 2 * sf);
      // a weight that streams through once leaves what else is in L2 there
      if (p.w_once) tma_load_2d(st, &tmap_w, &full[slot], kt * 128, w_row, once);
      else tma_load_2d_plain(st, &tmap_w, &full[slot], kt * 128, w_row);
      bulk_load(st + kWBytes + S::kABytes, p.w_s + (int64_t(w_row >> 7) * p.groups + 2 * kt) * 512, sf, &full[slot]);
      if constexpr (!kX) {
        tma_load_2d_plain(st + kWBytes, &tmap_a, &full[slot], kt * 128, a_row);
        bulk_load(st + kWBytes + S::kABytes + kSfBytes, p.a_s + (int64_t(a_row >> 7) * p.groups + 2 * kt) * 512, sf,
                  &full[slot]);
      }
      if (++slot == S::kStages) slot = 0, phase ^= 1u;
    }
  } else if (warp == 1) {
    // M = 128 weight rows, N = NT activation rows, both E2M1 and K-major
    constexpr uint32_t kIdesc =
        (1u << 7) | (1u << 10) | (uint32_t(NT >> 3) << 17) | kIdescE8m0 | (uint32_t(kWRows >> 4) << 24);
    int slot = 0;
    uint32_t phase = 0, sf_slot = 0;
    bool ok = true;
    for (int kt = kt0; kt < kt1; ++kt) {
      ok = mbar_wait_bounded(&full[slot], phase, p.wait_limit_cycles, const_cast<const int*>(abort_flag));
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t st = smem_u32(ring + slot * S::kStage);
      const uint32_t sfw = tmem + NT + sf_slot * kSfCols, sfa = sfw + 8;
      const uint64_t dw = desc_k128(st), da = desc_k128(st + kWBytes);
      const int ng = 2 * kt + 1 < p.groups ? 2 : 1;
      // elected: the descriptors stay in uniform registers (under lane == 0,
      // 8 x 14,336 x 5,376: 12.5 us, now 10.2)
      if (elect_one()) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (g >= ng) break;
          tc_cp_scales(sfw + 4 * g, st + kWBytes + S::kABytes + 512 * g);
          tc_cp_scales(sfa + 4 * g, st + kWBytes + S::kABytes + kSfBytes + 512 * g);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // K = 64 step: 32 bytes further along the row; its two scales are
            // bytes 2h, 2h + 1 of the group's scale word
            const uint32_t id = kIdesc | (uint32_t(2 * h) << 4) | (uint32_t(2 * h) << 29);
            tc_mma_mxf4(tmem, dw + 4 * g + 2 * h, da + 4 * g + 2 * h, id, sfw + 4 * g, sfa + 4 * g,
                        (kt > kt0 || g > 0 || h > 0) ? 1u : 0u);
          }
        }
        tc_commit(&empty[slot]);
      }
      __syncwarp();
      sf_slot ^= 1u;
      if (++slot == S::kStages) slot = 0, phase ^= 1u;
    }
    if (!ok) *abort_flag = 1;
    if (elect_one()) tc_commit(done);
  }

  // Quantised activation: thread t of warps 2..5 takes block t % 8 of row
  // t / 8 (and of row 16 + t / 8) of every k-tile.  Rows past m stay as they
  // are: they only reach accumulator columns that nobody stores.
  if constexpr (kX) {
    if (warp >= 2) {
      constexpr int kPer = NT / 16;
      const int t = int(threadIdx.x) - 64, c = t & 7;
      const int valid = min(NT, p.m - a_row);
      RawBlock<X> next[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i * 16 + (t >> 3) < valid && kt0 < kt1) next[i].load(p, a_row + i * 16 + (t >> 3), kt0 * 256 + c * 32);
      int slot = 0;
      uint32_t phase = 0;
      for (int kt = kt0; kt < kt1; ++kt) {
        RawBlock<X> cur[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          cur[i] = next[i];
          if (i * 16 + (t >> 3) < valid && kt + 1 < kt1)
            next[i].load(p, a_row + i * 16 + (t >> 3), (kt + 1) * 256 + c * 32);
        }
        int ok = 1;
        if (lane == 0)
          ok = mbar_wait_bounded(&empty[slot], phase ^ 1u, p.wait_limit_cycles, const_cast<const int*>(abort_flag));
        if (__shfl_sync(0xFFFFFFFFu, ok, 0) == 0) {
          *abort_flag = 1;
          break;
        }
        uint8_t* tile = ring + slot * S::kStage + kWBytes;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int r = i * 16 + (t >> 3);
          if (r < valid) {
            float f[32];
            cur[i].values(f);
            uint32_t e;
            const uint4 q = mx_encode_block(f, e);
            *reinterpret_cast<uint4*>(tile + r * 128 + ((c ^ (r & 7)) << 4)) = q;
            tile[S::kABytes + kSfBytes + (c >> 2) * 512 + r * 16 + (c & 3)] = uint8_t(e);
          }
        }
        fence_proxy_async_smem();  // the generic-proxy writes, then the MMA's and the copy's reads
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[slot]);
        if (++slot == S::kStages) slot = 0, phase ^= 1u;
      }
    }
  }

  // The accumulators: warps 2..5, lane quarter warp % 4.
  const bool epi = warp >= 2;
  const int q = warp & 3;
  const int valid = min(NT, p.m - a_row);
  const int col = w_row + q * 32 + lane;
  float* part = reinterpret_cast<float*>(ring);  // [NT][128], the ring is idle once `done` completes
  if (epi) {
    int ok = 1;
    if (lane == 0) ok = mbar_wait_bounded(done, 0, p.wait_limit_cycles, nullptr);
    ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
    if (lane == 0 && (!ok || *abort_flag) && p.dev_status != nullptr)
      atomicExch(p.dev_status, static_cast<uint32_t>(NVFP4_ETIMEOUT));
    tc_fence_after();
#pragma unroll 1
    for (int c = 0; c < NT; c += 16) {
      if (c >= valid) break;
      uint32_t r[16];
      __syncwarp();  // lanes past n have stored nothing
      tmem_ld_32x32b_x16(tmem + (uint32_t(q * 32) << 16) + c, r);
      tc_wait_ld();
      tmem_ld_fence_regs<16>(r);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (p.split == 1) {
          if (c + i < valid && col < p.n) store_out(p, a_row + c + i, col, __uint_as_float(r[i]));
        } else {
          part[(c + i) * 128 + q * 32 + lane] = __uint_as_float(r[i]);
        }
      }
    }
    tc_fence_before();
  }
  if (p.split > 1) {
    cluster_sync();  // every CTA's partial is in its shared memory
    if (epi) {
      // a warp takes an activation row, a lane four weight rows of it
      const uint32_t mine = smem_u32(part) + uint32_t(lane) * 16u;
#pragma unroll 1
      for (int c = rank + q * p.split; c < valid; c += 4 * p.split) {
        float4 v[kMaxSplit];
#pragma unroll
        for (int s = 0; s < kMaxSplit; ++s)
          v[s] = s < p.split ? ld_cluster_f32x4(mapa_shared(mine + uint32_t(c) * 512u, uint32_t(s)))
                             : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float4 sum = v[0];
#pragma unroll
        for (int s = 1; s < kMaxSplit; ++s) {
          sum.x += v[s].x, sum.y += v[s].y, sum.z += v[s].z, sum.w += v[s].w;
        }
        store_out4(p, a_row + c, w_row + lane * 4, sum);
      }
    }
    cluster_sync();  // nobody leaves while its partial is read
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, S::kTmem);
  }
}

// Clusters of c CTAs of `kernel` that are resident at once on the current device.
template <class K>
nvfp4_status resident_clusters(K kernel, int smem, int c, int32_t* most) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(c) * 1024);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = size_t(smem);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(c);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  const nvfp4_status st =
      cuda_check(cudaOccupancyMaxActiveClusters(&n, kernel, &cfg), "cudaOccupancyMaxActiveClusters(k_mx_rows)");
  *most = n < 1 ? 1 : n;
  return st;
}

template <int NT, bool kX, typename X>
nvfp4_status rows_launch(const void* a_q, const void* w_q, int64_t m, int64_t n, int64_t k, RowsParams& p,
                         cudaStream_t stream) {
  using S = Shape<NT>;
  CUtensorMap ta = {}, tw;
  nvfp4_status st = NVFP4_OK;
  if (!kX) st = mx_operand_map(&ta, a_q, m, k, NT, "A");
  if (st == NVFP4_OK) st = mx_operand_map(&tw, w_q, n, k, kWRows, "W");
  if (st != NVFP4_OK) return st;
  const int64_t w_tiles = (n + kWRows - 1) / kWRows, a_tiles = (m + NT - 1) / NT;
  const int tiles = (p.groups + 1) / 2;
  auto kernel = k_mx_rows<NT, kX, X>;
  static std::atomic<uint64_t> ready{0};  // devices whose attribute is set
  st = allow_smem(reinterpret_cast<const void*>(kernel), S::kSmem, ready);
  if (st != NVFP4_OK) return st;
  // The largest split that leaves every CTA a k-tile and whose clusters run all at
  // once by the runtime's count, which is of one CTA an SM: 46, 36, 28, 23 and 15
  // clusters of 3, 4, 5, 6 and 7.  (Two CTAs fit, but more than one draw little
  // more; what costs is a second wave.)  1 x 5376 x 14336 (42 tiles, split 3):
  // split 1 to 8 take 23.2, 13.9, 10.9, 10.8, 11.1, 10.7, 14.6 and 13.9 us.
  // 61 x 21504 x 5376 (168 tiles, split 1): 15.6, 23.2, 21.3, 25.6, 26.1 us.
  static std::atomic<int32_t> fit[64][kMaxSplit] = {};  // asked once for each device
  int dev = 0;
  if ((st = cuda_check(cudaGetDevice(&dev), "cudaGetDevice")) != NVFP4_OK) return st;
  int64_t split = 1;
  for (int c = std::min(tiles, kMaxSplit); c > 1; --c) {
    if (w_tiles * a_tiles * c > 2 * int64_t(sm_count())) continue;
    int32_t most = dev < 64 ? fit[dev][c - 1].load(std::memory_order_relaxed) : 0;
    if (most == 0) {
      st = resident_clusters(kernel, S::kSmem, c, &most);
      if (st != NVFP4_OK) return st;
      if (dev < 64) fit[dev][c - 1].store(most, std::memory_order_relaxed);
    }
    if (w_tiles * a_tiles <= most) {
      split = c;
      break;
    }
  }
  p.split = int32_t(split);
  p.w_once = a_tiles == 1;
  return launch("launch k_mx_rows", kernel, dim3(unsigned(w_tiles * split), unsigned(a_tiles)), dim3(kThreads), S::kSmem,
                int(split), stream, ta, tw, p);
}

RowsParams rows_params(const void* w_s, int64_t m, int64_t n, int64_t k, void* out, int32_t dtype, int64_t ldo,
                       uint32_t* dev_status) {
  RowsParams p = {};
  p.w_s = static_cast<const uint8_t*>(w_s);
  p.out = out;
  p.ldo = ldo;
  p.m = int32_t(m), p.n = int32_t(n), p.k = int32_t(k), p.dtype = dtype;
  p.groups = int32_t(mxfp4_padded_cols(k) / 128);
  p.out_vec = aligned16(out) && ldo % 4 == 0;
  p.dev_status = dev_status;
  p.wait_limit_cycles = kMxWaitLimitCycles;
  return p;
}

template <typename X>
nvfp4_status rows_x(const void* w_q, int64_t m, int64_t n, int64_t k, RowsParams& p, cudaStream_t stream) {
  if (m <= 16) return rows_launch<16, true, X>(nullptr, w_q, m, n, k, p, stream);
  return rows_launch<32, true, X>(nullptr, w_q, m, n, k, p, stream);
}

}  // namespace

nvfp4_status mx_rows(const void* a_q, const void* a_s, const void* w_q, const void* w_s, int64_t m, int64_t n,
                     int64_t k, void* out, int32_t dtype, int64_t ldo, uint32_t* dev_status, cudaStream_t stream) {
  RowsParams p = rows_params(w_s, m, n, k, out, dtype, ldo, dev_status);
  p.a_s = static_cast<const uint8_t*>(a_s);
  if (m <= 16) return rows_launch<16, false, float>(a_q, w_q, m, n, k, p, stream);
  if (m <= 32) return rows_launch<32, false, float>(a_q, w_q, m, n, k, p, stream);
  if (m <= 64) return rows_launch<64, false, float>(a_q, w_q, m, n, k, p, stream);
  return rows_launch<128, false, float>(a_q, w_q, m, n, k, p, stream);
}

nvfp4_status mx_rows_x(const void* x, int32_t x_dtype, int64_t ldx, const void* w_q, const void* w_s, int64_t m,
                       int64_t n, int64_t k, void* out, int32_t dtype, int64_t ldo, uint32_t* dev_status,
                       cudaStream_t stream) {
  RowsParams p = rows_params(w_s, m, n, k, out, dtype, ldo, dev_status);
  p.x = x;
  p.ldx = ldx;
  p.x_vec = aligned16(x) && ldx * mx_elem_bytes(x_dtype) % 16 == 0;
  if (x_dtype == MXFP4_BF16) return rows_x<__nv_bfloat16>(w_q, m, n, k, p, stream);
  if (x_dtype == MXFP4_FP16) return rows_x<__half>(w_q, m, n, k, p, stream);
  return rows_x<float>(w_q, m, n, k, p, stream);
}

}  // namespace nvfp4
