// Conversions between fp32 and e4m3 (1 sign, 4 exponent, 3 mantissa bits; no
// infinity, largest value 448), 16 values at a time.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace spr {

// Two values rounded to nearest even: a in the low byte. NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3_2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// e4m3 of x * f (f a power of two, |x * f| <= 448; infinities become NaN)
__device__ __forceinline__ uint4 to_e4m3_16(const float (&x)[16], float f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = x[4 * i + j];
      y[j] = fabsf(v) == INFINITY ? __int_as_float(0x7fffffff) : v * f;
    }
    w[i] = to_e4m3_2(y[0], y[1]) | (to_e4m3_2(y[2], y[3]) << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Two e4m3 values (low 16 bits) as fp16, exactly: every e4m3 value is one.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t r;
  const uint16_t u = static_cast<uint16_t>(v);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(u));
  return r;
}

__device__ __forceinline__ void from_e4m3_16(const uint4 u, float (&x)[16]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t h = e4m3x2_to_f16x2(w[i] >> (16 * j));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      x[4 * i + 2 * j] = f.x;
      x[4 * i + 2 * j + 1] = f.y;
    }
}

__device__ __forceinline__ float from_e4m3(uint8_t v) {
  const uint32_t h = e4m3x2_to_f16x2(v);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xffff)));
}

}  // namespace spr
