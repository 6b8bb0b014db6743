// FP8 cache rows as bf16 values: codes exactly, and products of codes and scales as sums of two.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace mla {

// 16 e4m3 codes -> 16 bf16 values, exactly.
__device__ __forceinline__ void codes16(const uint4 &codes, uint4 &lo, uint4 &hi) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint16_t pair = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    uint32_t half2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(half2) : "h"(pair));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&half2));
    const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
    o[i] = *reinterpret_cast<const uint32_t *>(&v);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// 16 e4m3 codes times a scale, as sums first + rest of two bf16 values.
__device__ __forceinline__ void widen16_twice(const uint4 &codes, float scale, uint4 (&first)[2], uint4 (&rest)[2]) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  uint32_t hi[8], lo[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint16_t pair = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    uint32_t half2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(half2) : "h"(pair));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&half2));
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x * scale, f.y * scale);
    hi[i] = *reinterpret_cast<const uint32_t *>(&h);
    const __nv_bfloat162 l = __floats2bfloat162_rn(fmaf(f.x, scale, -__uint_as_float(hi[i] << 16)),
                                                   fmaf(f.y, scale, -__uint_as_float(hi[i] & 0xffff0000u)));
    lo[i] = *reinterpret_cast<const uint32_t *>(&l);
  }
#pragma unroll
  for (int i = 0; i < 2; i++) {
    first[i] = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
    rest[i] = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
  }
}

}  // namespace mla
