// 8-bit rows: their layout and the conversions the kernels share (the format
// is described in attnres.h).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace attnres {

// Two e4m3 codes as fp16 (exact: fp16 holds every e4m3 number).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}

__device__ __forceinline__ float2 f16x2_f32(uint32_t h) { return __half22float2(*reinterpret_cast<__half2*>(&h)); }

// Four codes of a word as fp32 pairs.
__device__ __forceinline__ void decode4(uint32_t c, float2& a, float2& b) {
  a = f16x2_f32(e4m3x2_f16x2(static_cast<uint16_t>(c)));
  b = f16x2_f32(e4m3x2_f16x2(static_cast<uint16_t>(c >> 16)));
}

__device__ __forceinline__ void decode16(const uint4& c, float2 (&v)[8]) {
  decode4(c.x, v[0], v[1]);
  decode4(c.y, v[2], v[3]);
  decode4(c.z, v[4], v[5]);
  decode4(c.w, v[6], v[7]);
}

// Four fp32 values as codes, rounded to nearest even, NaN kept.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// The biased exponent e + 127 of the scale of a group whose largest magnitude
// has the bits `amax`: with amax = f 2^k, 1 <= f < 2, it is 2^(k - 8) when
// f <= 1.75 (448 = 1.75 2^8), else 2^(k - 7). From 1 to 247.
__device__ __forceinline__ uint32_t q8_exponent(uint32_t amax) {
  const int e = static_cast<int>(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < 1 ? 1u : static_cast<uint32_t>(e);
}
__device__ __forceinline__ float q8_scale(uint32_t e) { return __uint_as_float(e << 23); }
__device__ __forceinline__ float q8_inverse(uint32_t e) { return __uint_as_float((254u - e) << 23); }
// The largest code magnitude: above 240, 2^120 times a code is no fp32 number.
__device__ __forceinline__ float q8_top(uint32_t e) { return e == 247u ? 240.f : 448.f; }

constexpr uint32_t kInfBits = 0x7f800000u;

}  // namespace attnres
