// Device helpers shared by the MISA kernels (gfx950, wave64).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace misa {

constexpr int kWave = 64;
constexpr int kD = 128;  // head dimension supported by this build

enum DType : int32_t { kF32 = 0, kBF16 = 1, kFP8 = 2 };

// ---------------------------------------------------------------- element loads

__device__ __forceinline__ float bf16_bits_to_f32(uint32_t bits16) {
  return __uint_as_float(bits16 << 16);
}

// OCP e4m3fn byte -> fp32 through the gfx950 hardware converter (this target's
// fp8 conversions use the OCP encoding).
__device__ __forceinline__ float fp8_to_f32(uint32_t byte) {
  return __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(byte), 0);
}

// Load element i of a row in dtype DT as fp32.
template <int DT>
__device__ __forceinline__ float load_elem(const void* base, int64_t i) {
  if constexpr (DT == kF32) {
    return static_cast<const float*>(base)[i];
  } else if constexpr (DT == kBF16) {
    return bf16_bits_to_f32(static_cast<const uint16_t*>(base)[i]);
  } else {
    return fp8_to_f32(static_cast<const uint8_t*>(base)[i]);
  }
}

template <int DT>
constexpr int elem_bytes() {
  return DT == kF32 ? 4 : (DT == kBF16 ? 2 : 1);
}

// ReLU as one v_med3_f32: clamp(x, 0, 3e38) equals max(x, 0) for every finite
// score (fmaxf adds a NaN-quieting v_max per element).
__device__ __forceinline__ float relu(float x) { return __builtin_amdgcn_fmed3f(x, 0.f, 3.0e38f); }

// ---------------------------------------------------------------- ordering keys

// Order-preserving map fp32 -> u32 (larger float <=> larger key); -0 maps like +0.
// Host-callable too (the top-k key intervals are checked exhaustively on the CPU).
__host__ __device__ __forceinline__ uint32_t float_key(float f) {
  uint32_t u = __builtin_bit_cast(uint32_t, f);
  if (u == 0x80000000u) u = 0;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// ---------------------------------------------------------------- wave / block scans

__device__ __forceinline__ int lane_id() { return threadIdx.x & (kWave - 1); }

// Number of set bits of a 64-bit lane mask strictly below this lane.
__device__ __forceinline__ int lanes_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32),
                                   __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0));
}

__device__ __forceinline__ int wave_inclusive_sum(int v) {
  const int lane = lane_id();
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int y = __shfl_up(v, o, kWave);
    if (lane >= o) v += y;
  }
  return v;
}

// Lane l's partner at step `o` of an all-reduction over neighbouring lanes (o =
// 1, 2, 4, ... in order: the values of both halves of 2o lanes are alike by
// then, so that a mirrored partner is as good as lane l ^ o): register moves
// instead of LDS permutes.
template <int O>
__device__ __forceinline__ float lanes_partner(float x) {
  const int u = __float_as_int(x);
  if constexpr (O == 1) {
    return __int_as_float(__builtin_amdgcn_update_dpp(u, u, 0xB1, 0xF, 0xF, false));  // quad_perm 1 0 3 2
  } else if constexpr (O == 2) {
    return __int_as_float(__builtin_amdgcn_update_dpp(u, u, 0x4E, 0xF, 0xF, false));  // quad_perm 2 3 0 1
  } else if constexpr (O == 4) {
    return __int_as_float(__builtin_amdgcn_update_dpp(u, u, 0x141, 0xF, 0xF, false));  // row_half_mirror
  } else if constexpr (O == 8) {
    return __int_as_float(__builtin_amdgcn_update_dpp(u, u, 0x140, 0xF, 0xF, false));  // row_mirror
  } else if constexpr (O == 16) {
    // Swaps the odd rows of one copy with the even rows of the other: one of
    // the results is x itself, the other its partner.
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return __int_as_float((threadIdx.x & 16) ? r[0] : r[1]);
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __int_as_float((threadIdx.x & 32) ? r[0] : r[1]);
  }
}

// Sum (MAX: maximum, NaN left out) over N neighbouring lanes, known to all.
template <int N, bool MAX>
__device__ __forceinline__ float lanes_reduce(float x) {
  if constexpr (N > 1) x = MAX ? fmaxf(x, lanes_partner<1>(x)) : x + lanes_partner<1>(x);
  if constexpr (N > 2) x = MAX ? fmaxf(x, lanes_partner<2>(x)) : x + lanes_partner<2>(x);
  if constexpr (N > 4) x = MAX ? fmaxf(x, lanes_partner<4>(x)) : x + lanes_partner<4>(x);
  if constexpr (N > 8) x = MAX ? fmaxf(x, lanes_partner<8>(x)) : x + lanes_partner<8>(x);
  if constexpr (N > 16) x = MAX ? fmaxf(x, lanes_partner<16>(x)) : x + lanes_partner<16>(x);
  if constexpr (N > 32) x = MAX ? fmaxf(x, lanes_partner<32>(x)) : x + lanes_partner<32>(x);
  return x;
}

// Block-wide exclusive prefix sum of `v` in thread order; `total` receives the
// block sum.  `tmp` is LDS scratch of NT/64 ints.  Contains __syncthreads().
template <int NT>
__device__ __forceinline__ int block_exclusive_sum(int v, int* tmp, int& total) {
  constexpr int NW = NT / kWave;
  const int lane = lane_id();
  const int wid = threadIdx.x / kWave;
  const int inc = wave_inclusive_sum(v);
  if (lane == kWave - 1) tmp[wid] = inc;
  __syncthreads();
  int base = 0, tot = 0;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    const int c = tmp[i];
    base += (i < wid) ? c : 0;
    tot += c;
  }
  __syncthreads();
  total = tot;
  return base + inc - v;
}

}  // namespace misa
