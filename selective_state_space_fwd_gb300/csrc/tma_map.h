// tma_map.h -- host-side encoding of the tensor maps of TMA copies.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace ssm {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once; null when the driver has none.
inline EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

// A [rows, inner] tensor with rows `pitch` elements apart, copied in boxes of
// 128 bytes (64 bf16 or 32 fp32 elements) x box_rows rows, 128-byte swizzled.
// Loads read zeros past either extent; stores write nothing there.  The base is
// 16-byte aligned and the pitch a multiple of 16 bytes (the caller's checks).
inline bool map_sw128(CUtensorMap* m, bool f32, const void* base, int64_t inner, int64_t rows,
                      int64_t pitch, int box_rows) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const unsigned size = f32 ? 4 : 2;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch) * size};
  const cuuint32_t box[2] = {128 / size, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
inline bool map_bf16_sw128(CUtensorMap* m, const void* base, int64_t inner, int64_t rows,
                           int64_t pitch, int box_rows) {
  return map_sw128(m, false, base, inner, rows, pitch, box_rows);
}
inline bool map_f32_sw128(CUtensorMap* m, const void* base, int64_t inner, int64_t rows,
                          int64_t pitch, int box_rows) {
  return map_sw128(m, true, base, inner, rows, pitch, box_rows);
}

}  // namespace ssm
