// E4M3 codes and power-of-two row scales, shared by the 8-bit cache's kernels.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace llama {

// Two floats to two E4M3 codes (round to nearest even, saturating): a in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(b), "f"(a));
  return c;
}
// Two E4M3 codes (low byte first) back to floats.
__device__ __forceinline__ float2 e4m3x2_to_f2(uint32_t c) {
  uint32_t h;
  asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(c));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The row scale's exponent: the smallest e in -100 .. 100 with u <= 448 * 2^e (u >= 0).  448 = 1.75 * 2^8,
// so e is u's exponent less 8, and one more where its significand is above 1.75: a carry out of
// the mantissa when 2^-2 less one ulp is added to it.
__device__ __forceinline__ int row_scale_exp(float u) {
  const int e = (int)((__float_as_uint(u) + 0x1FFFFFu) >> 23) - 127 - 8;
  return min(max(e, -100), 100);
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

}  // namespace llama
