// Root-mean-square norm of rows with the residual's addition before it and an
// 8-bit output with one scale per row after it (misa_rms_norm in misa.h).
#include "common.hpp"
#include "launch.hpp"
#include "mfma.hpp"
#include "quant.hpp"

namespace misa {

namespace {

__device__ __forceinline__ void store_elem(int dt, void* base, int64_t i, float x) {
  if (dt == kF32)
    static_cast<float*>(base)[i] = x;
  else
    static_cast<__bf16*>(base)[i] = static_cast<__bf16>(x);
}

// Any n and any groups: one workgroup per row, the row's sums in LDS; wave w
// takes the parts w, w + 4, ... one after the other.
template <int XT>
__global__ __launch_bounds__(256) void norm_any_kernel(int32_t n, int32_t size, int32_t out_dtype,
                                                       float eps, const void* x,
                                                       const void* residual,
                                                       const float* __restrict__ weight,
                                                       void* sum_out, void* __restrict__ out,
                                                       float* __restrict__ out_scale) {
  extern __shared__ float z[];
  __shared__ float top[4];
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * n;
  float amax = 0.f;
  for (int32_t p0 = wave * size; p0 < n; p0 += 4 * size) {
    float ss = 0.f;
    for (int32_t e = lane; e < size; e += kWave) {
      const int64_t i = base + p0 + e;
      float y = load_elem<XT>(x, i);
      if (residual) y += load_elem<XT>(residual, i);
      if (sum_out) store_elem(XT, sum_out, i, y);
      z[p0 + e] = y;
      ss += y * y;
    }
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) ss += __shfl_xor(ss, o, kWave);
    const float r = 1.f / sqrtf(ss / static_cast<float>(size) + eps);
    for (int32_t e = lane; e < size; e += kWave) {
      const float v = z[p0 + e] * r * weight[e];
      z[p0 + e] = v;
      amax = amax_step(amax, v);
    }
  }
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o, kWave));
  if (lane == 0) top[wave] = amax;
  __syncthreads();
  if (out_dtype != kFP8) {
    for (int32_t e = threadIdx.x; e < n; e += 256) store_elem(out_dtype, out, base + e, z[e]);
    return;
  }
  float scale, mult;
  e4m3_scale(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), scale, mult);
  for (int32_t e = threadIdx.x; e < n; e += 256)
    static_cast<uint8_t*>(out)[base + e] = static_cast<uint8_t>(e4m3_pack4(z[e], 0.f, 0.f, 0.f, mult));
  if (threadIdx.x == 0) out_scale[blockIdx.x] = scale;
}

}  // namespace

hipError_t launch_rms_norm(int32_t rows, int32_t n, int32_t groups, int32_t x_dtype,
                           int32_t out_dtype, float eps, const void* x, const void* residual,
                           const float* weight, void* sum_out, void* out, float* out_scale,
                           hipStream_t st) {
  const size_t lds = static_cast<size_t>(n) * sizeof(float);
  const void* f = x_dtype == kF32 ? reinterpret_cast<const void*>(norm_any_kernel<kF32>)
                                  : reinterpret_cast<const void*>(norm_any_kernel<kBF16>);
  if (lds > 48 * 1024) {
    const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize,
                                             kMaxNorm * sizeof(float));
    if (e != hipSuccess) return e;
  }
  if (x_dtype == kF32)
    norm_any_kernel<kF32><<<rows, 256, lds, st>>>(n, n / groups, out_dtype, eps, x, residual,
                                                  weight, sum_out, out, out_scale);
  else
    norm_any_kernel<kBF16><<<rows, 256, lds, st>>>(n, n / groups, out_dtype, eps, x, residual,
                                                   weight, sum_out, out, out_scale);
  return hipGetLastError();
}

}  // namespace misa
