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

// Eight elements at e as fp32: one or two 16-byte loads, which need not be
// aligned to more than an element (rows of odd length start anywhere).
struct __attribute__((packed, aligned(2))) Bf16x8 {
  uint32_t w[4];
};
struct __attribute__((packed, aligned(4))) F32x8 {
  float w[8];
};

// bf16 and 8-bit outputs from this size on leave the L2s (32 MB) before anyone
// reads them; they are marked as not to be kept there, which leaves more of the
// inputs: 8192 x 64 x 128 to fp8 35.5 us, 40.3 without; 12000 rows of 4096 in bf16
// 31.4 and 39.4; 2000 rows of 8192 to fp8 11.5 and 11.3.  fp32 sums so marked
// would cost (12000 rows of 4096 144 us against 123).
constexpr int64_t kOnceStores = int64_t{16} << 20;

// N dwords to an address that is a multiple of A; `once`: marked as not to be kept.
template <int N, int A>
__device__ __forceinline__ void store_words(void* to, const uint32_t (&w)[N], bool once) {
  typedef __attribute__((ext_vector_type(N))) uint32_t V;
  typedef V __attribute__((aligned(A))) U;
  V x;
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = w[i];
  if (once) {
    asm volatile("");  // on both sides, or the branches are merged into a plain store
    __builtin_nontemporal_store(x, static_cast<U*>(to));
    asm volatile("");
  } else {
    *static_cast<U*>(to) = x;
  }
}

template <int XT>
__device__ __forceinline__ void load8(const void* base, int64_t e, float (&x)[8]) {
  if constexpr (XT == kF32) {
    const F32x8 v = *reinterpret_cast<const F32x8*>(static_cast<const float*>(base) + e);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v.w[i];
  } else {
    const Bf16x8 v = *reinterpret_cast<const Bf16x8*>(static_cast<const uint16_t*>(base) + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(v.w[i] << 16);
      x[2 * i + 1] = __uint_as_float(v.w[i] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ void store8(int dt, void* base, int64_t e, const float (&x)[8], bool once) {
  if (dt == kF32) {  // always kept: each of its two stores leaves out every other 16 bytes of a line
    F32x8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v.w[i] = x[i];
    *reinterpret_cast<F32x8*>(static_cast<float*>(base) + e) = v;
  } else {
    bf16x8 y;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = static_cast<__bf16>(x[i]);
    const uint4 v = __builtin_bit_cast(uint4, y);
    store_words<4, 2>(static_cast<uint16_t*>(base) + e, {v.x, v.y, v.z, v.w}, once);
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

// Vectors of a thread up to which the weights are loaded before the row's sum is
// known: with more they cost the registers of a second workgroup on the CU.
constexpr int kEarlyWeights = 4;
// 1 / rms beyond which it is multiplied in first.
constexpr float kFarRoot = 0x1p16f;
// A sum of squares may leave fp32's range where their mean (of at most 2^15) does
// not: an infinite one is formed again from elements divided by this.
constexpr float kFarSquares = 0x1p16f;

__device__ __forceinline__ float far_squares(const float (&y)[8]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = y[i] * (1.f / kFarSquares);
    s += x * x;
  }
  return s;
}

// T threads per row, V vectors of eight elements in registers per thread: one
// read of x and residual, one write.  The parts of a row (GROUPED) have 2^k <=
// 64 places of a vector each, neighbouring lanes of a wave, of which the last
// may be empty, so that their sums are register moves.  ODD: a row's length is
// no multiple of eight; its last vector ends with the row, and the elements that
// the one before already has are left out of sums and stores.  Bound by memory
// traffic: 8192 rows of 64 parts of 128, bf16 -> fp8 (201 MB), 35.5 us, 5.7 TB/s;
// 32 rows of 4096 with residual, 3.6 us, a launch and two loads' latency.
template <int XT, int T, int V, bool GROUPED, bool ODD>
__global__ __launch_bounds__(256) void norm_kernel(int32_t rows, int32_t n, int32_t size,
                                                   int32_t part_shift, int32_t out_dtype,
                                                   float inv_size, float eps, bool once,
                                                   const void* x, const void* residual,
                                                   const float* __restrict__ weight, void* sum_out,
                                                   void* __restrict__ out,
                                                   float* __restrict__ out_scale) {
  __shared__ float tmp[3][4];
  const int t = threadIdx.x % T;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / T) + threadIdx.x / T;
  if (row >= rows) return;  // T < 256: whole rows of lanes leave; T = 256: never
  const int64_t base = row * n;
  // Place v * T + t: its element in the row and in its part, and how many of its
  // elements are left out; false: an empty place.
  auto place = [&](int v, int& e, int& w, int& skip) {
    const int i = v * T + t;
    skip = 0;
    if constexpr (GROUPED) {
      const int part = i >> part_shift, at = (i & ((1 << part_shift) - 1)) * 8;
      e = part * size + at;
      w = min(at, size - 8);
      return e < n && at < size;
    } else {
      e = i * 8;
      const bool inside = e < n;
      if (ODD && inside) skip = max(e + 8 - n, 0);
      e -= skip;
      w = min(e, n - 8);
      return inside;
    }
  };
  auto store = [&](int dt, void* to, int e, int skip, const float(&z)[8]) {
    if (!ODD || skip == 0) {
      store8(dt, to, base + e, z, once);
    } else {
#pragma unroll
      for (int i = 1; i < 8; ++i)
        if (i >= skip) store_elem(dt, to, base + e + i, z[i]);
    }
  };
  float y[V][8], ss[V];
  int e, at, skip;
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[v][i] = 0.f;
    if (place(v, e, at, skip)) load8<XT>(x, base + e, y[v]);
  }
  if (residual) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (place(v, e, at, skip)) {
        float z[8];
        load8<XT>(residual, base + e, z);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[v][i] += z[i];
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const bool inside = place(v, e, at, skip);
    if (sum_out && inside) store(XT, sum_out, e, skip, y[v]);
    ss[v] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (ODD && i < skip) y[v][i] = 0.f;
      ss[v] += y[v][i] * y[v][i];
    }
  }
  // Weights on their way during the reduction: of parts, one vector for all of a
  // thread's places (T is a multiple of a part's); else where they are few.
  constexpr bool kEarly = GROUPED || V <= kEarlyWeights;
  constexpr int WV = GROUPED || !kEarly ? 1 : V;
  float w[WV][8];
  if constexpr (kEarly) {
#pragma unroll
    for (int v = 0; v < WV; ++v) {
      place(v, e, at, skip);
      load8<kF32>(weight, at, w[v]);
    }
  }
  float r[V];
  if constexpr (GROUPED) {
    part_sums<1>(ss, 1 << part_shift);
    bool over = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      r[v] = ss[v] * inv_size;
      over |= ss[v] == INFINITY;
    }
    if (__any(over)) {  // wave-uniform, like the parts
      float far[V];
#pragma unroll
      for (int v = 0; v < V; ++v) far[v] = far_squares(y[v]);
      part_sums<1>(far, 1 << part_shift);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (ss[v] == INFINITY) r[v] = far[v] * inv_size * (kFarSquares * kFarSquares);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) r[v] = __builtin_amdgcn_rsqf(r[v] + eps);
  } else {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) s += ss[v];
    s = row_reduce<T, false>(s, tmp[0]);
    float mean = s * inv_size;
    if (__any(s == INFINITY)) {  // uniform over a workgroup with one row
      float far = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) far += far_squares(y[v]);
      far = row_reduce<T, false>(far, tmp[2]);
      if (s == INFINITY) mean = far * inv_size * (kFarSquares * kFarSquares);
    }
    const float f = __builtin_amdgcn_rsqf(mean + eps);
#pragma unroll
    for (int v = 0; v < V; ++v) r[v] = f;
  }
  // z = y w now; r, the same for a part, comes in with the last product.  A large
  // (small) r comes first: y w of the smallest (largest) values could leave fp32's
  // range while y r w does not, and so could r times the codes' multiplier.
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const bool first = r[v] > kFarRoot || r[v] < 1.f / kFarRoot;
    if (__any(first)) {
      const float f = first ? r[v] : 1.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[v][i] *= f;
      r[v] = first ? 1.f : r[v];
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (!kEarly) {
      place(v, e, at, skip);
      load8<kF32>(weight, at, w[0]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) y[v][i] *= w[v < WV ? v : 0][i];
  }
  if (out_dtype != kFP8) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!place(v, e, at, skip)) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[v][i] *= r[v];
      store(out_dtype, out, e, skip, y[v]);
    }
    return;
  }
  float amax = 0.f;  // empty places and left-out elements hold zeros, or NaN if their part does
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = amax_step(top, y[v][i]);
    amax = fmaxf(amax, top * r[v]);
  }
  float scale, mult;
  e4m3_scale(row_reduce<T, true>(amax, tmp[1]), scale, mult);
  auto* codes = static_cast<uint8_t*>(out) + base;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (!place(v, e, at, skip)) continue;
    const float f = r[v] * mult;
    const uint32_t c[2] = {e4m3_pack4(y[v][0], y[v][1], y[v][2], y[v][3], f),
                           e4m3_pack4(y[v][4], y[v][5], y[v][6], y[v][7], f)};
    if (!ODD || skip == 0) {
      store_words<2, 1>(codes + e, c, once);
    } else {
#pragma unroll
      for (int i = 1; i < 8; ++i)
        if (i >= skip) codes[e + i] = static_cast<uint8_t>(c[i / 4] >> (i % 4 * 8));
    }
  }
  if (t == 0) out_scale[row] = scale;
}

struct NormArgs {
  int32_t rows, n, groups, part_shift, x_dtype, out_dtype;
  float eps;
  const void *x, *residual;
  const float* weight;
  void *sum_out, *out;
  float* out_scale;
};

template <int XT, int T, int V, bool GROUPED, bool ODD>
void launch_norm(const NormArgs& a, hipStream_t st) {
  const int32_t per = 256 / T;
  const bool once = static_cast<int64_t>(a.rows) * a.n * (a.out_dtype == kF32 ? 4 : a.out_dtype == kBF16 ? 2 : 1) >= kOnceStores;
  norm_kernel<XT, T, V, GROUPED, ODD><<<(a.rows - 1) / per + 1, 256, 0, st>>>(
      a.rows, a.n, a.n / a.groups, a.part_shift, a.out_dtype, 1.f / static_cast<float>(a.n / a.groups),
      a.eps, once, a.x, a.residual, a.weight, a.sum_out, a.out, a.out_scale);
}

// Threads per row and vectors per thread, by the vectors' places in a row: the
// fewest of both that hold it.  Up to 256 places a row stays in a wave, or a part
// of one, and needs no barrier; longer ones have a workgroup, whose registers hold
// up to 4096.  60 million bf16 elements to fp8, rows of 256: 40 us in 32 lanes, 71
// in 64; of 1024: 35 us in a wave, 63 in a workgroup; of 2048: 38.8 and 41.9; of
// 4096: 48.7 and 36.9; of 5120: 38.9 us with three vectors a thread, 43.9 with four.
template <int XT, bool GROUPED, bool ODD>
void launch_norm_size(const NormArgs& a, hipStream_t st) {
  const int32_t places = GROUPED ? a.groups << a.part_shift : (a.n + 7) / 8;
  if (places <= 16) launch_norm<XT, 16, 1, GROUPED, ODD>(a, st);
  else if (places <= 32) launch_norm<XT, 32, 1, GROUPED, ODD>(a, st);
  else if (places <= 64) launch_norm<XT, 64, 1, GROUPED, ODD>(a, st);
  else if (places <= 128) launch_norm<XT, 64, 2, GROUPED, ODD>(a, st);
  else if (places <= 256) launch_norm<XT, 64, 4, GROUPED, ODD>(a, st);
  else if (places <= 512) launch_norm<XT, 256, 2, GROUPED, ODD>(a, st);
  else if (places <= 768) launch_norm<XT, 256, 3, GROUPED, ODD>(a, st);
  else if (places <= 1024) launch_norm<XT, 256, 4, GROUPED, ODD>(a, st);
  else if (places <= 2048) launch_norm<XT, 256, 8, GROUPED, ODD>(a, st);
  else launch_norm<XT, 256, 16, GROUPED, ODD>(a, st);
}

template <int XT>
void launch_norm_type(const NormArgs& a, hipStream_t st) {
  if (a.groups > 1) launch_norm_size<XT, true, false>(a, st);
  else if (a.n % 8 == 0) launch_norm_size<XT, false, false>(a, st);
  else launch_norm_size<XT, false, true>(a, st);
}

// Rows below eight elements and every other division into parts: one workgroup
// per row, the row's sums in LDS; wave w takes the parts w, w + 4, ... one after
// the other.  Bound by its passes over LDS and the reductions between them.
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
    float mean = ss / static_cast<float>(size);
    if (ss == INFINITY) {  // every lane alike
      ss = 0.f;
      for (int32_t e = lane; e < size; e += kWave) {
        const float y = z[p0 + e] * (1.f / kFarSquares);
        ss += y * y;
      }
#pragma unroll
      for (int o = 1; o < kWave; o <<= 1) ss += __shfl_xor(ss, o, kWave);
      mean = ss / static_cast<float>(size) * (kFarSquares * kFarSquares);
    }
    const float r = 1.f / sqrtf(mean + eps);
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
  int32_t shift = 0;  // 2^shift places of eight elements hold a part
  while (groups > 1 && (8 << shift) < size) ++shift;
  const bool in_registers =
      groups == 1 ? n >= 8 : (size % 8 == 0 && shift <= 6 && (static_cast<int64_t>(groups) << shift) * 8 <= kMaxNorm);
  if (in_registers) {
    const NormArgs a{rows, n, groups, shift, x_dtype, out_dtype, eps, x, residual, weight, sum_out, out, out_scale};
    if (x_dtype == kF32)
      launch_norm_type<kF32>(a, st);
    else
      launch_norm_type<kBF16>(a, st);
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
