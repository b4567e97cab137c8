// tma.cu -- host side of the TMA tensor maps.
#include <mutex>

#include "common.cuh"
#include "e4m3.cuh"
#include "tma.h"

namespace q2 {

namespace {
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}
}  // namespace

static q2_status make_tmap_2d(CUtensorMap* out, CUtensorMapDataType type, uint32_t elem, const void* base,
                              uint64_t rows, uint64_t cols, uint64_t pitch_bytes, uint32_t box_rows,
                              uint32_t box_cols, int swizzle_bytes) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) {
    set_error("cuTensorMapEncodeTiled is not available");
    return Q2_ERR_CUDA;
  }
  if ((reinterpret_cast<uintptr_t>(base) & 15) || (pitch_bytes & 15) || ((box_cols * elem) & 15)) {
    set_error("tensor map: base, pitch and box width must be 16-byte multiples");
    return Q2_ERR_INVALID_ARG;
  }
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {pitch_bytes};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUtensorMapSwizzle sw = swizzle_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                          : swizzle_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                          : swizzle_bytes == 32 ? CU_TENSOR_MAP_SWIZZLE_32B
                                                : CU_TENSOR_MAP_SWIZZLE_NONE;
  CUresult r = fn(out, type, 2, const_cast<void*>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (CUresult " + std::to_string((int)r) + ")");
    return Q2_ERR_CUDA;
  }
  return Q2_OK;
}

q2_status make_tmap_2d_bf16(CUtensorMap* out, const void* base, uint64_t rows, uint64_t cols,
                            uint64_t pitch_bytes, uint32_t box_rows, uint32_t box_cols,
                            int swizzle_bytes) {
  return make_tmap_2d(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, rows, cols, pitch_bytes, box_rows, box_cols,
                      swizzle_bytes);
}

q2_status make_tmap_2d_u8(CUtensorMap* out, const void* base, uint64_t rows, uint64_t cols,
                          uint64_t pitch_bytes, uint32_t box_rows, uint32_t box_cols, int swizzle_bytes) {
  return make_tmap_2d(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, base, rows, cols, pitch_bytes, box_rows, box_cols,
                      swizzle_bytes);
}

q2_status make_tmap_2d_f32(CUtensorMap* out, const void* base, uint64_t rows, uint64_t cols,
                           uint64_t pitch_bytes, uint32_t box_rows, uint32_t box_cols, int swizzle_bytes) {
  return make_tmap_2d(out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, base, rows, cols, pitch_bytes, box_rows, box_cols,
                      swizzle_bytes);
}

}  // namespace q2
