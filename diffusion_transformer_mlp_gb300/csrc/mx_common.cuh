// Device helpers of the MXFP4 operators: the element types outside the 4-bit
// format, the block encoder and the E2M1 / E8M0 decoders.
//
// A block is 32 consecutive elements with one E8M0 scale 2^(E-127), E - 127 =
// floor(log2 max|x|) - 2, so the block's largest element lands in [4, 8) and
// E2M1 (largest value 6) saturates it.  Scaling by a power of two is exact,
// which leaves the E2M1 rounding as the only one.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "common.cuh"
#include "mxfp4.h"

namespace nvfp4 {

// Lets `kernel` use `bytes` of dynamic shared memory on the current device,
// once a device (bit of `ready`): the attribute call costs as much as a small
// kernel's launch.
inline nvfp4_status allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& ready) {
  int dev = 0;
  nvfp4_status st = cuda_check(cudaGetDevice(&dev), "cudaGetDevice");
  if (st != NVFP4_OK) return st;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (dev < 64 && (ready.load(std::memory_order_acquire) & bit)) return NVFP4_OK;
  st = cuda_check(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes),
                  "cudaFuncSetAttribute");
  if (st == NVFP4_OK && dev < 64) ready.fetch_or(bit, std::memory_order_release);
  return st;
}

// Launches `kernel` so that it may be set up while the kernel before it in the
// stream drains (programmatic dependent launch).  Every kernel launched this
// way calls grid_wait() before it touches global memory: it waits until the
// kernel before it has ended and its writes are visible, so that the order of
// the stream holds.  Back to back launches of small kernels come 1-2 us closer.
// No kernel lets the next one start before its own blocks end: waiting blocks
// then held places on the SMs (decoding a batch took 128 us instead of 92).
template <class... Params, class... Args>
nvfp4_status launch(const char* what, void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, int cluster,
                    cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...), what);
}

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

inline int mx_elem_bytes(int32_t dtype) { return dtype == MXFP4_FP32 ? 4 : 2; }
inline bool mx_dtype_ok(int32_t dtype) { return dtype == MXFP4_BF16 || dtype == MXFP4_FP16 || dtype == MXFP4_FP32; }

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Two 16-bit elements of a 32-bit word as binary32.
template <typename T>
__device__ __forceinline__ float2 word_to_f32(uint32_t w);
template <>
__device__ __forceinline__ float2 word_to_f32<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <>
__device__ __forceinline__ float2 word_to_f32<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// Two binary32 values rounded to nearest even into one word (lo in bits 0..15).
template <typename T>
__device__ __forceinline__ uint32_t f32_to_word(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t f32_to_word<__half>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <>
__device__ __forceinline__ uint32_t f32_to_word<__nv_bfloat16>(float lo, float hi) {
  return bf16x2_rn(lo, hi);
}

// 32 bytes.  Written at once where the address allows it: two stores of 16
// bytes by neighbouring lanes each touch half of every 32-byte sector (4,096 x
// 14,336 to bf16: 38 us, at once 28).  Read they are two loads, of which the
// second finds its sectors in L1 (quantising the same: 27 us, at once 33).
__device__ __forceinline__ void load32b(const void* p, uint32_t (&w)[8]) {
  const uint4 x = static_cast<const uint4*>(p)[0], y = static_cast<const uint4*>(p)[1];
  w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
}
__device__ __forceinline__ void store32b(void* p, const uint32_t (&w)[8]) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// 16 consecutive elements at a 16-byte aligned address.
template <typename T>
__device__ __forceinline__ void load16(const T* __restrict__ p, float (&f)[16]) {
#pragma unroll
  for (int h = 0; h < int(sizeof(T)) / 2; ++h) {
    uint32_t w[8];
    load32b(reinterpret_cast<const uint8_t*>(p) + 32 * h, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 4) {
        f[8 * h + i] = __uint_as_float(w[i]);
      } else {
        const float2 t = word_to_f32<T>(w[i]);
        f[2 * i] = t.x, f[2 * i + 1] = t.y;
      }
    }
  }
}
template <typename T>
__device__ __forceinline__ void store16(T* __restrict__ p, const float (&f)[16]) {
#pragma unroll
  for (int h = 0; h < int(sizeof(T)) / 2; ++h) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(f[8 * h + i]);
      else w[i] = f32_to_word<T>(f[2 * i], f[2 * i + 1]);
    }
    store32b(reinterpret_cast<uint8_t*>(p) + 32 * h, w);
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Eight E2M1 codes of a word, element i in bits 4i .. 4i+3.
__device__ __forceinline__ uint32_t e2m1x8(const float* q) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return w;
}

// Half of a block: the lane and its neighbour (lane ^ 1) hold 16 elements
// each.  Returns the lane's 16 codes and the block's scale code.  A block
// with an infinity or a NaN gets E = 255 and zero codes.
__device__ __forceinline__ uint2 mx_encode_half(float (&f)[16], uint32_t& scale) {
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) am = max_nan(am, fabsf(f[i]));
  am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
  const uint32_t eb = (__float_as_uint(am) >> 23) & 0xFFu;  // biased exponent: floor(log2 am) + 127 for normal am
  if (eb == 255u) {
    scale = 255u;
    return make_uint2(0u, 0u);
  }
  const uint32_t e = eb > 2u ? eb - 2u : 0u;
  scale = e;
  const float inv = __uint_as_float((254u - e) << 23);  // 2^(127 - E), E <= 252
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] *= inv;
  return make_uint2(e2m1x8(f), e2m1x8(f + 8));
}

// A whole block in one lane: its 32 codes and its scale code.
__device__ __forceinline__ uint4 mx_encode_block(float (&f)[32], uint32_t& scale) {
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) am = max_nan(am, fabsf(f[i]));
  const uint32_t eb = (__float_as_uint(am) >> 23) & 0xFFu;
  if (eb == 255u) {
    scale = 255u;
    return make_uint4(0u, 0u, 0u, 0u);
  }
  const uint32_t e = eb > 2u ? eb - 2u : 0u;
  scale = e;
  const float inv = __uint_as_float((254u - e) << 23);
#pragma unroll
  for (int i = 0; i < 32; ++i) f[i] *= inv;
  return make_uint4(e2m1x8(f), e2m1x8(f + 8), e2m1x8(f + 16), e2m1x8(f + 24));
}

// The eight E2M1 values of a word as four pairs of FP16 (exact).
__device__ __forceinline__ void e2m1x8_to_half(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Value of an E8M0 code: 2^(E-127), NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t e) {
  return __uint_as_float(e == 0u ? 0x00400000u : (e == 255u ? 0x7FFFFFFFu : e << 23));
}

// 16 values of one lane's codes under one scale.
__device__ __forceinline__ void mx_decode16(uint2 q, uint32_t scale, float (&f)[16]) {
  const float s = e8m0_value(scale);
  uint32_t h[4];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    e2m1x8_to_half(half ? q.y : q.x, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = word_to_f32<__half>(h[i]);
      f[8 * half + 2 * i] = t.x * s, f[8 * half + 2 * i + 1] = t.y * s;
    }
  }
}

}  // namespace nvfp4
