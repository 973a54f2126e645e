// fp8.cuh -- rows and weights in 8 bits: e4m3 codes, one fp32 scale for each
// block of 128 columns (rows) or each tile of 128 x 128 (weights).
//
//   scale = 2^ceil(log2(amax / 448)), at least 2^-126   (448: the largest e4m3)
//   code  = e4m3(v / scale), to nearest, ties to even
// The scale is a power of two, so v / scale is exact and the code is v rounded
// once (to 4 significant bits, half a step = 2^-4 of the value at most; below
// 2^-6 of a scale in steps of 2^-9): nothing depends on how a division rounds.
// It costs no precision, e4m3's steps being relative, and at most one of the 18
// powers of two that a block spans.  amax is taken over bit patterns, so that a
// block that holds an infinity or a NaN has an amax at or above infinity's: its
// scale and its codes are NaN.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace moe {
namespace fp8 {

constexpr int kBlock = 128;

__host__ __device__ constexpr int blocks_of(int n) { return (n + kBlock - 1) / kBlock; }

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

struct Scale {
  float scale, inv;
};

// From the largest magnitude's bits.  448 = 1.75 * 2^8, so amax / 448 is a
// power of two or less when amax's fraction is at most 0x600000: adding
// 0x1fffff carries into the exponent exactly when it is more.
__device__ __forceinline__ Scale scale_of(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return {quiet_nan(), quiet_nan()};
  const int e = max((int)((amax_bits + 0x1fffffu) >> 23) - 8, 1);
  return {__int_as_float(e << 23), __int_as_float((254 - e) << 23)};
}

// Two codes, lo in the low byte.
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return codes2(a, b) | (codes2(c, d) << 16);
}

// The values of two codes (without the scale); every e4m3 value is an fp16 value.
__device__ __forceinline__ float2 values2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  float2 f;
  asm("{\n\t.reg .f16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.f32.f16 %0, lo;\n\t"
      "cvt.f32.f16 %1, hi;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

}  // namespace fp8
}  // namespace moe
