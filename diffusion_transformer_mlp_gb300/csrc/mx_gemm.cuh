// What the two MXFP4 product kernels share: descriptors, tensor maps, limits.
#pragma once

#include "mx_common.cuh"

namespace nvfp4 {

// Instruction descriptor bit of E8M0 scales (scale format 1) for the
// block-scaled kinds.
constexpr uint32_t kIdescE8m0 = 1u << 23;

// About two seconds at the highest clock, as the NVFP4 GEMM's limit: far above
// any legitimate wait.
constexpr uint64_t kMxWaitLimitCycles = 4000000000ull;

// Shared-memory descriptor of a K-major tile with 128-byte rows and the
// 128-byte swizzle (8-row atoms 1,024 bytes apart).
__device__ __forceinline__ uint64_t desc_k128(uint32_t saddr) {
  return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}

// Tensor map of an MXFP4 operand's QDATA [rows, cols_pad / 2] with boxes of
// box_rows x 128 bytes (256 elements), 128-byte swizzle.
nvfp4_status mx_operand_map(CUtensorMap* map, const void* q, int64_t rows, int64_t cols, int box_rows,
                            const char* what);

// Tensor map through the driver (gemm.cu).
nvfp4_status make_map(CUtensorMap* map, CUtensorMapDataType dt, const void* base, int rank, const cuuint64_t* dims,
                      const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle, const char* what);

// The kernel for few rows (mx_rows.cu).
nvfp4_status mx_rows(const void* a_q, const void* a_s, const void* w_q, const void* w_s, int64_t m, int64_t n,
                     int64_t k, void* out, int32_t dtype, int64_t ldo, uint32_t* dev_status, cudaStream_t stream);

// The same for up to kMxRowsX rows of x before quantisation.
constexpr int64_t kMxRowsX = 32;
nvfp4_status mx_rows_x(const void* x, int32_t x_dtype, int64_t ldx, const void* w_q, const void* w_s, int64_t m,
                       int64_t n, int64_t k, void* out, int32_t dtype, int64_t ldo, uint32_t* dev_status,
                       cudaStream_t stream);

// The CTA-pair kernel (gemm.cu).
nvfp4_status mx_pairs(const void* a_q, const void* a_s, const void* w_q, const void* w_s, int64_t m, int64_t n,
                      int64_t k, void* out, int32_t dtype, int64_t ldo, uint32_t* dev_status, cudaStream_t stream);

}  // namespace nvfp4
