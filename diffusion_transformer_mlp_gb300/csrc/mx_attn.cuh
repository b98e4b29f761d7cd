// What the attention kernels over the MXFP4 cache share: parameters, the
// masks' geometry, small PTX helpers.
#pragma once

#include "mx_common.cuh"

namespace nvfp4 {

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
// `tok` keys: tiles [0, sink_tiles) and [lo_tile, hi_tile).
struct Span {
  int32_t hi;          // keys >= hi are seen by none of the rows
  int32_t lo_tile, sink_tiles, n;
  __device__ __forceinline__ int32_t tile(int32_t s) const { return s < sink_tiles ? s : s - sink_tiles + lo_tile; }
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
  s.hi = hi;
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

}  // namespace nvfp4
