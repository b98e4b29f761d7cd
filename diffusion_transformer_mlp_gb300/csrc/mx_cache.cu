// The paged KV cache in MXFP4: quantising k and v as they are written, and
// reading whole sequences back.
//
// A page holds [kv_heads][page_size][dim / 2] code bytes and [kv_heads]
// [page_size][dim / 32] scale bytes, so the tokens of a page that one head
// reads are contiguous.  A lane takes 16 elements of one (token, head) row:
// dim / 16 lanes a row, 8 code bytes a lane, and the row's scale bytes in one
// or two stores from its first lane(s).  Bound by HBM like the quantiser:
// 24,000 tokens of 8 heads of 128 (123 MB) written in 23.5 us, 5.2 TB/s, read
// back in 23 us, 5.3 TB/s.
#include <string>

#include "mx_common.cuh"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kReadTokens = 32;  // most tokens of one block of k_mx_cache_read

struct CacheDims {
  int64_t pages;
  int32_t page_shift, heads, dim;
};

// Row of (page, head, offset) in units of one token's codes.
__device__ __forceinline__ int64_t cache_row(const CacheDims& c, int64_t page, int32_t head, int32_t off) {
  return ((page * c.heads + head) << c.page_shift) + off;
}

template <typename T, bool kAligned>
__global__ void __launch_bounds__(kThreads)
    k_mx_cache_write(const T* __restrict__ k, const T* __restrict__ v, int64_t k_st, int64_t k_sh, int64_t v_st,
                     int64_t v_sh, const int64_t* __restrict__ slots, int64_t tokens, uint8_t* __restrict__ kc,
                     uint8_t* __restrict__ ks, uint8_t* __restrict__ vc, uint8_t* __restrict__ vs, const CacheDims c) {
  grid_wait();
  const bool is_v = blockIdx.y != 0;
  const T* x = is_v ? v : k;
  const int64_t st = is_v ? v_st : k_st, sh = is_v ? v_sh : k_sh;
  uint8_t* codes = is_v ? vc : kc;
  uint8_t* scales = is_v ? vs : ks;
  const int32_t lane_bits = c.dim == 64 ? 2 : (c.dim == 128 ? 3 : 4);  // a row never leaves its warp
  const int64_t items = (tokens * c.heads) << lane_bits;
  // the whole warp stays in the loop for the shuffles
  for (int64_t i0 = int64_t(blockIdx.x) * kThreads + (threadIdx.x & ~31); i0 < items;
       i0 += int64_t(gridDim.x) * kThreads) {
    const int64_t i = i0 + (threadIdx.x & 31);
    const int64_t rowi = i >> lane_bits;
    const int32_t s = int32_t(i - (rowi << lane_bits));
    const int64_t tok = items <= 0x7FFFFFFF ? int64_t(uint32_t(rowi) / uint32_t(c.heads)) : rowi / c.heads;
    const int32_t head = int32_t(rowi - tok * c.heads);
    const bool in = i < items;
    const int64_t slot = in ? slots[tok] : -1;
    const bool live = slot >= 0 && slot < (c.pages << c.page_shift);
    float f[16];
    if (live) {
      const T* src = x + tok * st + head * sh + s * 16;
      if constexpr (kAligned) {
        load16(src, f);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) f[j] = to_f32(src[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] = 0.0f;
    }
    uint32_t e;
    const uint2 q = mx_encode_half(f, e);
    const uint32_t e1 = __shfl_down_sync(0xFFFFFFFFu, e, 2), e2 = __shfl_down_sync(0xFFFFFFFFu, e, 4),
                   e3 = __shfl_down_sync(0xFFFFFFFFu, e, 6);
    if (live) {
      const int64_t row = cache_row(c, slot >> c.page_shift, head, int32_t(slot & ((1 << c.page_shift) - 1)));
      *reinterpret_cast<uint2*>(codes + row * (c.dim / 2) + s * 8) = q;
      uint8_t* d = scales + row * (c.dim / 32);
      if (c.dim == 64) {
        if (s == 0) *reinterpret_cast<uint16_t*>(d) = uint16_t(e | e1 << 8);
      } else if ((s & 7) == 0) {
        *reinterpret_cast<uint32_t*>(d + s / 2) = e | e1 << 8 | e2 << 16 | e3 << 24;
      }
    }
  }
}

// One block takes `chunk` tokens: a thread a token finds its sequence (binary
// search of starts) and page, then all threads walk the tokens' rows of k and v.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_mx_cache_read(const int32_t* __restrict__ table, int64_t table_ld, int32_t seqs,
                    const int32_t* __restrict__ starts, int64_t total, int32_t chunk, T* __restrict__ k,
                    T* __restrict__ v, const uint8_t* __restrict__ kc, const uint8_t* __restrict__ ks,
                    const uint8_t* __restrict__ vc, const uint8_t* __restrict__ vs, const CacheDims c) {
  __shared__ int64_t base[kReadTokens];  // row of (page, head 0, offset)
  grid_wait();
  const int64_t t0 = int64_t(blockIdx.x) * chunk;
  const int32_t n = int32_t(total - t0 < chunk ? total - t0 : chunk);
  if (threadIdx.x < n) {
    const int64_t t = t0 + threadIdx.x;
    int32_t lo = 0, hi = seqs;  // starts[lo] <= t < starts[hi]
    while (hi - lo > 1) {
      const int32_t mid = (lo + hi) >> 1;
      if (starts[mid] <= t) lo = mid;
      else hi = mid;
    }
    int64_t pos = t - starts[lo];
    int64_t col = pos >> c.page_shift;
    if (col < 0) col = 0;
    if (col >= table_ld) col = table_ld - 1;
    int64_t page = table[int64_t(lo) * table_ld + col];
    if (page < 0) page = 0;
    if (page >= c.pages) page = c.pages - 1;
    base[threadIdx.x] = cache_row(c, page, 0, int32_t(pos & ((1 << c.page_shift) - 1)));
  }
  __syncthreads();
  const int32_t lane_bits = c.dim == 64 ? 2 : (c.dim == 128 ? 3 : 4);
  const int32_t per_tok = c.heads << lane_bits;
  const int32_t items = n * per_tok;
  for (int32_t i = threadIdx.x; i < 2 * items; i += kThreads) {
    const bool is_v = i >= items;
    const int32_t r = is_v ? i - items : i;
    const int32_t tok = int32_t(uint32_t(r) / uint32_t(per_tok));
    const int32_t hs = r - tok * per_tok;
    const int32_t head = hs >> lane_bits, s = hs - (head << lane_bits);
    const int64_t row = base[tok] + (int64_t(head) << c.page_shift);
    const uint2 q = *reinterpret_cast<const uint2*>((is_v ? vc : kc) + row * (c.dim / 2) + s * 8);
    float f[16];
    mx_decode16(q, (is_v ? vs : ks)[row * (c.dim / 32) + s / 2], f);
    store16((is_v ? v : k) + ((t0 + tok) * c.heads + head) * c.dim + s * 16, f);
  }
}

}  // namespace

// Checks a cache description; on success page_shift is its log2 page size.
nvfp4_status check_cache(const mxfp4_cache* cache, int* page_shift, const std::string& nm) {
  if (!cache || !cache->k_codes || !cache->k_scales || !cache->v_codes || !cache->v_scales)
    return fail(NVFP4_EINVAL, nm + ": null pointer");
  if (cache->pages < 1 || cache->kv_heads < 1 || cache->page_size < 1)
    return fail(NVFP4_EINVAL, nm + ": pages, kv_heads and page_size must be positive");
  int sh = 0;
  while ((1 << sh) < cache->page_size) ++sh;
  if ((1 << sh) != cache->page_size || cache->page_size < 16 || cache->page_size > 256)
    return fail(NVFP4_EUNSUPPORTED, nm + ": page_size must be 16, 32, 64, 128 or 256");
  if (cache->dim != 64 && cache->dim != 128 && cache->dim != 256)
    return fail(NVFP4_EUNSUPPORTED, nm + ": dim must be 64, 128 or 256");
  if (cache->kv_heads > 65535 || cache->pages > 0x7FFFFFFF / cache->kv_heads)
    return fail(NVFP4_EUNSUPPORTED, nm + ": cache too large");
  if (!aligned16(cache->k_codes) || !aligned16(cache->k_scales) || !aligned16(cache->v_codes) ||
      !aligned16(cache->v_scales))
    return fail(NVFP4_EALIGN, nm + ": cache pointers must be 16-byte aligned");
  *page_shift = sh;
  return NVFP4_OK;
}

namespace {

template <typename T>
nvfp4_status write_launch(const mxfp4_cache* cache, const CacheDims& c, const void* k, const void* v, int64_t tokens,
                  int64_t k_st, int64_t k_sh, int64_t v_st, int64_t v_sh, const int64_t* slots, cudaStream_t s) {
  constexpr int64_t el = 16 / sizeof(T);
  const bool vec = aligned16(k) && aligned16(v) && k_st % el == 0 && k_sh % el == 0 && v_st % el == 0 && v_sh % el == 0;
  const int64_t items = tokens * c.heads * (c.dim / 16);
  const int64_t blocks = (items + kThreads - 1) / kThreads, most = int64_t(sm_count()) * 8;
  const dim3 grid(unsigned(blocks < most ? blocks : most), 2);
  auto kern = vec ? k_mx_cache_write<T, true> : k_mx_cache_write<T, false>;
  return launch("launch k_mx_cache_write", kern, grid, dim3(kThreads), 0, 0, s, static_cast<const T*>(k),
                static_cast<const T*>(v), k_st, k_sh, v_st, v_sh, slots, tokens,
                static_cast<uint8_t*>(cache->k_codes), static_cast<uint8_t*>(cache->k_scales),
                static_cast<uint8_t*>(cache->v_codes), static_cast<uint8_t*>(cache->v_scales), c);
}

template <typename T>
nvfp4_status read_launch(const mxfp4_cache* cache, const CacheDims& c, const int32_t* table, int64_t table_ld, int64_t seqs,
                 const int32_t* starts, int64_t total, void* k, void* v, cudaStream_t s) {
  int64_t chunk = total / (int64_t(sm_count()) * 8);
  chunk = chunk < 1 ? 1 : (chunk > kReadTokens ? kReadTokens : chunk);
  const int64_t blocks = (total + chunk - 1) / chunk;
  return launch("launch k_mx_cache_read", k_mx_cache_read<T>, dim3(unsigned(blocks)), dim3(kThreads), 0, 0, s, table,
                table_ld, int32_t(seqs), starts, total, int32_t(chunk), static_cast<T*>(k), static_cast<T*>(v),
                static_cast<const uint8_t*>(cache->k_codes), static_cast<const uint8_t*>(cache->k_scales),
                static_cast<const uint8_t*>(cache->v_codes), static_cast<const uint8_t*>(cache->v_scales), c);
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status mxfp4_cache_write(const mxfp4_cache* cache, const void* k, const void* v, int32_t dtype,
                                          int64_t tokens, int64_t k_st, int64_t k_sh, int64_t v_st, int64_t v_sh,
                                          const int64_t* slots, nvfp4_stream_t stream) {
  const std::string nm("mxfp4_cache_write");
  int sh = 0;
  const nvfp4_status st = check_cache(cache, &sh, nm);
  if (st != NVFP4_OK) return st;
  if (!mx_dtype_ok(dtype)) return fail(NVFP4_EINVAL, nm + ": unknown element type");
  if (tokens < 0) return fail(NVFP4_EINVAL, nm + ": tokens must not be negative");
  if (tokens == 0) return NVFP4_OK;
  if (!k || !v || !slots) return fail(NVFP4_EINVAL, nm + ": null pointer");
  if (tokens > 0x7FFFFFFF) return fail(NVFP4_EUNSUPPORTED, nm + ": too many tokens");
  const uintptr_t es = uintptr_t(mx_elem_bytes(dtype));
  if (reinterpret_cast<uintptr_t>(k) % es != 0 || reinterpret_cast<uintptr_t>(v) % es != 0 ||
      reinterpret_cast<uintptr_t>(slots) % 8 != 0)
    return fail(NVFP4_EALIGN, nm + ": k, v and slots must be aligned to their elements");
  const CacheDims c{cache->pages, sh, cache->kv_heads, cache->dim};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == MXFP4_BF16) return write_launch<__nv_bfloat16>(cache, c, k, v, tokens, k_st, k_sh, v_st, v_sh, slots, s);
  if (dtype == MXFP4_FP16) return write_launch<__half>(cache, c, k, v, tokens, k_st, k_sh, v_st, v_sh, slots, s);
  return write_launch<float>(cache, c, k, v, tokens, k_st, k_sh, v_st, v_sh, slots, s);
}

extern "C" nvfp4_status mxfp4_cache_read(const mxfp4_cache* cache, const int32_t* table, int64_t table_ld,
                                         int64_t seqs, const int32_t* starts, int64_t total, void* k, void* v,
                                         int32_t dtype, nvfp4_stream_t stream) {
  const std::string nm("mxfp4_cache_read");
  int sh = 0;
  const nvfp4_status st = check_cache(cache, &sh, nm);
  if (st != NVFP4_OK) return st;
  if (!mx_dtype_ok(dtype)) return fail(NVFP4_EINVAL, nm + ": unknown element type");
  if (total < 0 || seqs < 0) return fail(NVFP4_EINVAL, nm + ": negative size");
  if (total == 0 || seqs == 0) return NVFP4_OK;
  if (!table || !starts || !k || !v) return fail(NVFP4_EINVAL, nm + ": null pointer");
  if (table_ld < 1) return fail(NVFP4_EINVAL, nm + ": a block table row needs an entry");
  if (seqs > 0x3FFFFFFF || total > 0x7FFFFFFF) return fail(NVFP4_EUNSUPPORTED, nm + ": too many sequences or tokens");
  if (!aligned16(k) || !aligned16(v) || reinterpret_cast<uintptr_t>(table) % 4 != 0 ||
      reinterpret_cast<uintptr_t>(starts) % 4 != 0)
    return fail(NVFP4_EALIGN, nm + ": k and v must be 16-byte aligned, table and starts aligned to their elements");
  const CacheDims c{cache->pages, sh, cache->kv_heads, cache->dim};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == MXFP4_BF16) return read_launch<__nv_bfloat16>(cache, c, table, table_ld, seqs, starts, total, k, v, s);
  if (dtype == MXFP4_FP16) return read_launch<__half>(cache, c, table, table_ld, seqs, starts, total, k, v, s);
  return read_launch<float>(cache, c, table, table_ld, seqs, starts, total, k, v, s);
}
