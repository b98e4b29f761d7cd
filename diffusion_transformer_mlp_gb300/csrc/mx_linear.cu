// Entry points of the MXFP4 product.
#include <string>

#include "mx_gemm.cuh"

namespace nvfp4 {

nvfp4_status mx_operand_map(CUtensorMap* map, const void* q, int64_t rows, int64_t cols, int box_rows,
                            const char* what) {
  const int64_t row_bytes = mxfp4_padded_cols(cols) / 2;
  const cuuint64_t dims[2] = {cuuint64_t(row_bytes), cuuint64_t(rows)};
  const cuuint64_t strides[1] = {cuuint64_t(row_bytes)};
  const cuuint32_t box[2] = {128, cuuint32_t(box_rows)};
  return make_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B, what);
}

namespace {

nvfp4_status check_product(const void* w_q, const void* w_s, int64_t m, int64_t n, int64_t k, const void* out,
                           int32_t dtype, int64_t ldo, const std::string& nm) {
  if (!w_q || !w_s || !out) return fail(NVFP4_EINVAL, nm + ": null pointer");
  if (!mx_dtype_ok(dtype)) return fail(NVFP4_EINVAL, nm + ": unknown element type");
  if (m < 1 || n < 1 || k < 1) return fail(NVFP4_EINVAL, nm + ": m, n and k must be positive");
  if (ldo < n) return fail(NVFP4_EINVAL, nm + ": output leading dimension too small");
  if (k > (int64_t(1) << 24) || m > (int64_t(1) << 30) || n > (int64_t(1) << 30))
    return fail(NVFP4_EUNSUPPORTED, nm + ": problem too large");
  if (!aligned16(w_q) || !aligned16(w_s) || reinterpret_cast<uintptr_t>(out) % mx_elem_bytes(dtype) != 0)
    return fail(NVFP4_EALIGN, nm + ": operands must be 16-byte aligned, the output aligned to its element");
  return NVFP4_OK;
}

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

nvfp4_status product(const void* a_q, const void* a_s, const void* w_q, const void* w_s, int64_t m, int64_t n,
                     int64_t k, void* out, int32_t dtype, int64_t ldo, uint32_t* dev_status, nvfp4_stream_t stream) {
  // mx_rows reads the weight once for every 128 rows and splits k, mx_pairs
  // keeps 256 x 256 tiles on two SMs each and walks k whole.  Up to 128 rows
  // the first wins at every shape tried (128 x 5376 x 14336: 16.8 against
  // 27.7 us); beyond, as long as its 128 x 128 tiles leave SMs to split k over
  // (512 x 2048 x 14336, 64 tiles: 20.3 against 26.9; 192 x 5376 x 14336, 84
  // tiles: 32.5 against 27.7).
  const bool few = m <= 128 || ((m + 127) / 128) * ((n + 127) / 128) <= sm_count() / 2;
  auto kernel = few ? mx_rows : mx_pairs;
  return kernel(a_q, a_s, w_q, w_s, m, n, k, out, dtype, ldo, dev_status, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status mxfp4_gemm(const void* a_q, const void* a_s, const void* w_q, const void* w_s, int64_t m,
                                   int64_t n, int64_t k, void* out, int32_t dtype, int64_t ldo, uint32_t* dev_status,
                                   nvfp4_stream_t stream) {
  const std::string nm("mxfp4_gemm");
  if (!a_q || !a_s) return fail(NVFP4_EINVAL, nm + ": null pointer");
  const nvfp4_status st = check_product(w_q, w_s, m, n, k, out, dtype, ldo, nm);
  if (st != NVFP4_OK) return st;
  if (!aligned16(a_q) || !aligned16(a_s)) return fail(NVFP4_EALIGN, nm + ": operands must be 16-byte aligned");
  return product(a_q, a_s, w_q, w_s, m, n, k, out, dtype, ldo, dev_status, stream);
}

extern "C" int64_t mxfp4_linear_workspace_bytes(int64_t m, int64_t k) {
  return m <= kMxRowsX ? 0 : align256(mxfp4_qdata_bytes(m, k)) + mxfp4_scale_bytes(m, k);
}

extern "C" nvfp4_status mxfp4_linear(const void* x, int32_t x_dtype, int64_t m, int64_t ldx, const void* w_q,
                                     const void* w_s, int64_t n, int64_t k, void* out, int32_t dtype, int64_t ldo,
                                     void* workspace, int64_t workspace_bytes, uint32_t* dev_status,
                                     nvfp4_stream_t stream) {
  const std::string nm("mxfp4_linear");
  if (!x || (!workspace && m > kMxRowsX)) return fail(NVFP4_EINVAL, nm + ": null pointer");
  nvfp4_status st = check_product(w_q, w_s, m, n, k, out, dtype, ldo, nm);
  if (st != NVFP4_OK) return st;
  if (!mx_dtype_ok(x_dtype)) return fail(NVFP4_EINVAL, nm + ": unknown element type");
  if (ldx < k) return fail(NVFP4_EINVAL, nm + ": row stride of x smaller than a row");
  if (!aligned16(workspace) || reinterpret_cast<uintptr_t>(x) % mx_elem_bytes(x_dtype) != 0)
    return fail(NVFP4_EALIGN, nm + ": workspace must be 16-byte aligned, x aligned to its element");
  if (workspace_bytes < mxfp4_linear_workspace_bytes(m, k))
    return fail(NVFP4_EINVAL, nm + ": workspace too small, " + std::to_string(mxfp4_linear_workspace_bytes(m, k)) +
                                  " bytes are needed");
  if (m <= kMxRowsX)
    return mx_rows_x(x, x_dtype, ldx, w_q, w_s, m, n, k, out, dtype, ldo, dev_status,
                     reinterpret_cast<cudaStream_t>(stream));
  uint8_t* a_q = static_cast<uint8_t*>(workspace);
  uint8_t* a_s = a_q + align256(mxfp4_qdata_bytes(m, k));
  if ((st = mxfp4_quantize(x, x_dtype, m, k, ldx, a_q, a_s, stream)) != NVFP4_OK) return st;
  return product(a_q, a_s, w_q, w_s, m, n, k, out, dtype, ldo, dev_status, stream);
}
