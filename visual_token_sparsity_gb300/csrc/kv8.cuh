// Device helpers of the 8-bit paged cache: e4m3 values, and for each page and
// KV head one fp32 factor of its keys and one of its values.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace sv {
namespace kv8 {

constexpr float kLeastScale = 1.1754943508222875e-38f;   // 2^-126

// Two e4m3 values as halves (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t v) {
  const uint32_t h = e4m3x2_to_half2(v);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Four floats to four e4m3 values, the first in the lowest byte: to nearest
// even, infinities and what lies beyond 448 to 448, NaN to NaN.
__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// The smallest power of two, at least 2^-126, that times 448 reaches the
// largest finite magnitude `top` (bf16 bits): 448 is 1.75 * 2^8, so the exponent
// goes up by one where the mantissa is above 1.75.
__device__ __forceinline__ float scale_of(uint32_t top) {
  const int e = (int)(((top << 16) + 0x1fffffu) >> 23) - 8;
  return __uint_as_float((uint32_t)max(e, 1) << 23);
}

// The larger magnitudes of two pairs of bf16 values, those that are not finite
// left out.
__device__ __forceinline__ uint32_t max_finite2(uint32_t top, uint32_t v) {
  v &= 0x7fff7fffu;
  if ((v & 0x7fffu) >= 0x7f80u) v &= 0xffff0000u;
  if (v >= 0x7f800000u) v &= 0xffffu;
  return __vmaxu2(top, v);
}

// A line of `total` things cut into C pieces of one size, give or take one: the first
// thing of piece c, floor(total * c / C), in 32 bits, and the piece that thing s lies in.
__host__ __device__ __forceinline__ uint32_t piece_begin(uint32_t total, uint32_t c, uint32_t C) {
  const uint32_t q = total / C;
  return q * c + (total - q * C) * c / C;
}
__device__ __forceinline__ int piece_of(uint32_t total, uint32_t s, uint32_t C) {
  return (int)(((unsigned long long)(s + 1) * C - 1) / total);
}

}  // namespace kv8
}  // namespace sv
