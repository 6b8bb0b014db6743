// Decoding of FP8 cache rows to 16-bit values.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace mla {

// 16 e4m3 codes times a scale -> 16 bf16 values, each rounded once (every code is
// exact in f16, and the product is made in fp32).
__device__ __forceinline__ void widen16(const uint4 &codes, float scale, uint4 &lo, uint4 &hi) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint16_t pair = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    uint32_t half2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(half2) : "h"(pair));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&half2));
    float x, y;  // both products in one instruction
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(x), "=f"(y)
        : "f"(f.x), "f"(f.y), "f"(scale));
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    o[i] = *reinterpret_cast<const uint32_t *>(&v);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

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

// fp16 with a power of two that brings values of at most `most` (bits of a positive
// float) below 2^15, and back.  What is 2^29 smaller than `most` and less then loses bits,
// none of which is 2^-40 of `most`.
__device__ __forceinline__ float to_f16_range(uint32_t most) {
  return __uint_as_float((268u - max(most >> 23, 15u)) << 23);  // 2^(141 - E), a value's exponent being E - 127
}
__device__ __forceinline__ float from_f16_range(uint32_t most) { return __uint_as_float((max(most >> 23, 15u) - 14u) << 23); }

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// Two bf16 values, times a power of two, as fp16.
__device__ __forceinline__ uint32_t f16_of_bf16(uint32_t v, float factor) {
  return pack_f16(__uint_as_float(v << 16) * factor, __uint_as_float(v & 0xffff0000u) * factor);
}

// The larger finite one of two bf16 values' sizes (bits).
__device__ __forceinline__ uint32_t largest_bf16(uint32_t v) {
  const uint32_t a = v & 0x7fffu, b = (v >> 16) & 0x7fffu;
  return max(a < 0x7f80u ? a : 0u, b < 0x7f80u ? b : 0u);
}

// 16 e4m3 codes times a scale: 16 keys, of the scale times `factor`, as sums k + rest of two
// fp16 values, and 16 bf16 values.
__device__ __forceinline__ void widen16_twice(const uint4 &codes, float scale, float factor, uint4 (&k)[2], uint4 (&rest)[2],
                                              uint4 (&v)[2]) {
  widen16(codes, scale, v[0], v[1]);
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  const float s = scale * factor;
  uint32_t hi[8], lo[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint16_t pair = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    uint32_t half2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(half2) : "h"(pair));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&half2));
    hi[i] = pack_f16(f.x * s, f.y * s);
    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi[i]));
    lo[i] = pack_f16(fmaf(f.x, s, -h.x), fmaf(f.y, s, -h.y));
  }
#pragma unroll
  for (int i = 0; i < 2; i++) {
    k[i] = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
    rest[i] = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
  }
}

}  // namespace mla
