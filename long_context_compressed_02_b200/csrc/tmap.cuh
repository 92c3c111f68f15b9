// Host-side construction of TMA tensor maps (cuTensorMapEncodeTiled through
// the runtime's driver entry point, so the library does not link libcuda).
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

namespace csa {

inline PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// 2-D row-major tensor [rows, inner] of `dtype` (row pitch = inner elements),
// boxes of [box_rows, box_inner] with the given swizzle.
inline bool encode_2d(CUtensorMap* map, CUtensorMapDataType dtype, uint32_t elem_bytes, const void* base,
                      uint64_t inner, uint64_t rows, uint32_t box_inner, uint32_t box_rows,
                      CUtensorMapSwizzle swz) {
  auto enc = tmap_encoder();
  if (!enc) return false;
  cuuint64_t gdim[2] = {inner, rows};
  cuuint64_t gstride[1] = {inner * elem_bytes};
  cuuint32_t box[2] = {box_inner, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, dtype, 2, const_cast<void*>(base), gdim, gstride, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same rows as [inner / 64 slabs][rows][64], boxes of `box_slabs` slabs of
// box_rows x 64: one copy fills consecutive 128-byte-swizzled slabs (bf16).
inline bool encode_slabs(CUtensorMap* map, const void* base, uint64_t inner, uint64_t rows, uint32_t box_rows,
                         uint32_t box_slabs) {
  auto enc = tmap_encoder();
  if (!enc) return false;
  cuuint64_t gdim[3] = {64, rows, inner / 64};
  cuuint64_t gstride[2] = {inner * 2, 128};
  cuuint32_t box[3] = {64, box_rows, box_slabs};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), gdim, gstride, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace csa
