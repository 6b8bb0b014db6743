// Host-side TMA tensor maps for the kernels that read or write strided bf16
// tensors.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"

namespace mla {

// The driver's cuTensorMapEncodeTiled, looked up once (null if the driver
// has none).  The static's initialisation is thread-safe.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult qr;
    void *f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &qr) ==
            cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
  }();
  return fn;
}

// A bf16 tensor [d2][d1][d0] with element strides s2, s1 (innermost 1), read
// in 128-byte swizzled boxes of b2 x b1 x 64 values (or b0, not swizzled).  The strides are
// multiples of 8 elements (16 bytes); the stride of an axis of one entry is
// never used, so it is replaced by a valid one.
inline bool make_map_3d(CUtensorMap *m, const void *ptr, uint64_t d0, uint64_t d1, uint64_t d2, int64_t s1, int64_t s2,
                        uint32_t b1, uint32_t b2, uint32_t b0 = 64, bool swizzle = true) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  if (d1 == 1) s1 = (int64_t)d0;
  if (d2 == 1) s2 = (int64_t)(d0 * d1);
  cuuint64_t dims[3] = {d0, d1, d2};
  cuuint64_t strides[2] = {(cuuint64_t)s1 * 2, (cuuint64_t)s2 * 2};
  cuuint32_t box[3] = {b0, b1, b2};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace mla
