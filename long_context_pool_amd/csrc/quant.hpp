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

// Quotients by one scale, rounded as a division rounds them: x times the scale's
// reciprocal is off by two steps of fp32 at most, and what the product with the scale then
// lacks of x, times the reciprocal, corrects it (Markstein).  A code is then the nearest
// to x of those that the scale gives; x * (448 / amax), rounded twice, takes the
// neighbour for about one of 1000 bf16 values.
struct Quotient {
  float inv, back;
  __device__ __forceinline__ explicit Quotient(float scale)
      : inv(1.f / scale), back(scale < INFINITY ? -scale : 0.f) {}  // by infinity: zero, as it is
  __device__ __forceinline__ float of(float x) const {
    const float q = x * inv;
    return __builtin_fmaf(__builtin_fmaf(q, back, x), inv, q);
  }
};

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
