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

// Eight elements at e (a multiple of 8; 16-byte aligned) as fp32.
template <int XT>
__device__ __forceinline__ void load8(const void* base, int64_t e, float (&x)[8]) {
  if constexpr (XT == kF32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + e);
    const float4 a = p[0], b = p[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + e);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ void store8(int dt, void* base, int64_t e, const float (&x)[8]) {
  if (dt == kF32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + e);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    bf16x8 y;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = static_cast<__bf16>(x[i]);
    *reinterpret_cast<bf16x8*>(static_cast<uint16_t*>(base) + e) = y;
  }
}

// Sum (MAX: maximum) over the T threads of a row, in a fixed order, known to
// all of them.  T = 256: a workgroup; tmp is LDS for its four waves.
template <int T, bool MAX>
__device__ __forceinline__ float row_reduce(float x, float* tmp) {
  x = lanes_reduce<(T < kWave ? T : kWave), MAX>(x);
  if constexpr (T > kWave) {
    if (lane_id() == 0) tmp[threadIdx.x / kWave] = x;
    __syncthreads();
    x = MAX ? fmaxf(fmaxf(tmp[0], tmp[1]), fmaxf(tmp[2], tmp[3])) : (tmp[0] + tmp[1]) + (tmp[2] + tmp[3]);
  }
  return x;
}

// ss over the `lanes` (a power of two) neighbouring lanes of a part.
template <int O, int V>
__device__ __forceinline__ void part_sums(float (&ss)[V], int lanes) {
  if (lanes <= O) return;  // wave-uniform
#pragma unroll
  for (int v = 0; v < V; ++v) ss[v] += lanes_partner<O>(ss[v]);
  if constexpr (O < kWave / 2) part_sums<2 * O>(ss, lanes);
}

// Parts that are multiples of 8 elements.  T threads per row, V vectors of 8
// elements in registers per thread: one read of x and residual, one write.
// Parts of a row (GROUPED) are 2^k <= 64 vectors, neighbouring lanes of a wave,
// so that their sums are shuffles.  Bound by memory traffic: 8192 rows of 64
// parts of 128, bf16 -> fp8 (201 MB), @NORM_BIG@; 32 rows of 4096
// with residual, @NORM_SMALL@.
template <int XT, int T, int V, bool GROUPED>
__global__ __launch_bounds__(256) void norm_kernel(int32_t rows, int32_t n, int32_t part_vecs,
                                                   int32_t out_dtype, float inv_size, float eps,
                                                   const void* x, const void* residual,
                                                   const float* __restrict__ weight, void* sum_out,
                                                   void* __restrict__ out,
                                                   float* __restrict__ out_scale) {
  __shared__ float tmp[2][4];
  const int t = threadIdx.x % T;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / T) + threadIdx.x / T;
  if (row >= rows) return;  // T < 256: whole rows of lanes leave; T = 256: never
  const int64_t base = row * n;
  const int nv = n / 8;
  float y[V][8];
  float ss[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = v * T + t;
    ss[v] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[v][e] = 0.f;
    if (i < nv) load8<XT>(x, base + i * 8, y[v]);
  }
  if (residual) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = v * T + t;
      if (i < nv) {
        float z[8];
        load8<XT>(residual, base + i * 8, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[v][e] += z[e];
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (sum_out && v * T + t < nv) store8(XT, sum_out, base + (v * T + t) * 8, y[v]);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss[v] += y[v][e] * y[v][e];
  }
  // Few vectors: the weights are on their way during the reduction.
  constexpr int WV = V <= 4 ? V : 1;
  float w[WV][8];
  auto load_w = [&](int v, float (&to)[8]) {
    const int i = v * T + t;
    load8<kF32>(weight, (GROUPED ? i & (part_vecs - 1) : min(i, nv - 1)) * 8, to);
  };
  if constexpr (V <= 4) {
#pragma unroll
    for (int v = 0; v < V; ++v) load_w(v, w[v]);
  }
  float r[V];
  if constexpr (GROUPED) {
    part_sums<1>(ss, part_vecs);
#pragma unroll
    for (int v = 0; v < V; ++v) r[v] = __builtin_amdgcn_rsqf(ss[v] * inv_size + eps);
  } else {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) s += ss[v];
    const float f = __builtin_amdgcn_rsqf(row_reduce<T, false>(s, tmp[0]) * inv_size + eps);
#pragma unroll
    for (int v = 0; v < V; ++v) r[v] = f;
  }
  float amax = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = v * T + t;
    if (i < nv) {
      if constexpr (V > 4) load_w(v, w[0]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[v][e] = y[v][e] * r[v] * w[V <= 4 ? v : 0][e];
        amax = amax_step(amax, y[v][e]);
      }
    }
  }
  if (out_dtype != kFP8) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * T + t < nv) store8(out_dtype, out, base + (v * T + t) * 8, y[v]);
    return;
  }
  float scale, mult;
  e4m3_scale(row_reduce<T, true>(amax, tmp[1]), scale, mult);
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (v * T + t < nv)
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(out) + base + (v * T + t) * 8) =
          make_uint2(e4m3_pack4(y[v][0], y[v][1], y[v][2], y[v][3], mult),
                     e4m3_pack4(y[v][4], y[v][5], y[v][6], y[v][7], mult));
  if (t == 0) out_scale[row] = scale;
}

struct NormArgs {
  int32_t rows, n, groups, x_dtype, out_dtype;
  float eps;
  const void *x, *residual;
  const float* weight;
  void *sum_out, *out;
  float* out_scale;
};

template <int XT, int T, int V, bool GROUPED>
void launch_norm(const NormArgs& a, hipStream_t st) {
  const int32_t size = a.n / a.groups;
  const int32_t per = 256 / T;
  norm_kernel<XT, T, V, GROUPED><<<(a.rows - 1) / per + 1, 256, 0, st>>>(
      a.rows, a.n, size / 8, a.out_dtype, 1.f / static_cast<float>(size), a.eps, a.x, a.residual,
      a.weight, a.sum_out, a.out, a.out_scale);
}

// Threads per row and vectors per thread, by the row's length: rows up to 128
// (512) elements share a wave (workgroup), longer ones have a workgroup, whose
// registers hold up to 32768.
template <int XT, bool GROUPED>
void launch_norm_size(const NormArgs& a, hipStream_t st) {
  const int32_t nv = a.n / 8;
  if (nv <= 16) launch_norm<XT, 16, 1, GROUPED>(a, st);
  else if (nv <= 64) launch_norm<XT, 64, 1, GROUPED>(a, st);
  else if (nv <= 256) launch_norm<XT, 256, 1, GROUPED>(a, st);
  else if (nv <= 512) launch_norm<XT, 256, 2, GROUPED>(a, st);
  else if (nv <= 1024) launch_norm<XT, 256, 4, GROUPED>(a, st);
  else if (nv <= 2048) launch_norm<XT, 256, 8, GROUPED>(a, st);
  else launch_norm<XT, 256, 16, GROUPED>(a, st);
}

// Every other n and groups: one workgroup per row, the row's sums in LDS; wave w
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
  const int32_t size = n / groups;
  const bool pow2 = (size & (size - 1)) == 0;
  if (size % 8 == 0 && (groups == 1 || (pow2 && size <= 512))) {
    const NormArgs a{rows, n, groups, x_dtype, out_dtype, eps, x, residual, weight, sum_out, out, out_scale};
    if (x_dtype == kF32)
      groups == 1 ? launch_norm_size<kF32, false>(a, st) : launch_norm_size<kF32, true>(a, st);
    else
      groups == 1 ? launch_norm_size<kBF16, false>(a, st) : launch_norm_size<kBF16, true>(a, st);
    return hipGetLastError();
  }
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
