// e4m3fn codes with a shared fp32 scale: value = code * scale.
#pragma once

#include "common.hpp"

namespace misa {

constexpr float kE4M3Max = 448.f;

// Scale and code multiplier of values whose largest magnitude is `amax`.
// Below 2^-100, where 448 / amax nears overflow, the values count as zeros.
__device__ __forceinline__ void e4m3_scale(float amax, float& scale, float& mult) {
  const bool some = amax >= 0x1p-100f;
  scale = some ? amax / kE4M3Max : 1.f;
  mult = some ? kE4M3Max / amax : 1.f;
}

// What 448 / amax has beyond its fp32 rounding `mult`.  x * mult alone is off by up
// to a step of fp32, and bf16 values whose exact quotient lies midway between two
// codes (about one of 1000 does) would not always go to the even one.
__device__ __forceinline__ float e4m3_rest(float amax, float mult) {
  const bool some = amax >= 0x1p-100f && amax < INFINITY;
  return some ? __builtin_fmaf(-mult, amax, kE4M3Max) * mult * (1.f / kE4M3Max) : 0.f;
}

// Four codes of x * mult in one dword (hardware conversion, round to nearest
// even).  |x| is at most the amax that gave mult, so that a product exceeds 448 by
// a few roundings at most, and everything below 464 becomes 448: no clamp.
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d, float mult) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a * mult, b * mult, 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c * mult, d * mult, r, true);
  return static_cast<uint32_t>(r);
}

// The larger magnitude, a NaN left out.
__device__ __forceinline__ float amax_step(float m, float x) { return fmaxf(m, fabsf(x)); }

}  // namespace misa
