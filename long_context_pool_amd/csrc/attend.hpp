// Shared by the attention kernels (attend.hip, attend_latent.hip): arguments,
// token lookup, the division of rows into splits and their join.
#pragma once

#include "common.hpp"
#include "launch.hpp"
#include "mfma.hpp"

namespace misa {

typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(2))) int i32x2;

constexpr float kLn2 = 0.6931471805599453f;
// The sums are rescaled to a new maximum only when a score exceeds the old one
// by this much (log2): until then weights go up to 2^8, which loses nothing in
// fp32 and in the weights' bf16 parts, and O's registers are left alone.
constexpr float kSlack = 8.f;
constexpr uint32_t kHidden = 0xFFFFFFFFu;  // the slot of a token that is not visible

// n / P for 0 <= n < 2^31 by a multiplication: with l = ceil(log2 P), m =
// floor(2^(31+l) / P) + 1 is at most 1 above 2^(31+l) / P, so n * m / 2^(31+l)
// exceeds n / P by less than n / 2^(31+l) < 2^-l <= 1 / P: the same quotient.
struct Div {
  uint32_t m, shift, P;
};

inline Div make_div(uint32_t P) {
  uint32_t l = 0;
  while ((1u << l) < P) ++l;
  return {static_cast<uint32_t>((uint64_t{1} << (31 + l)) / P + 1), 31 + l, P};
}

__device__ __forceinline__ uint32_t div_page(uint32_t n, Div d) {
  return static_cast<uint32_t>((static_cast<uint64_t>(n) * d.m) >> d.shift);
}

struct Args {
  const uint16_t* q;
  const uint8_t* k_pages;
  const float* k_scale;
  const uint8_t* v_pages;
  const float* v_scale;
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* idx;
  uint16_t* out;
  float* lse;
  float* part_o;   // [rows, heads, splits, dv] unnormalised sums of a split
  float2* part_ml;  // [rows, heads, splits] maximum (log2) and sum
  int32_t rows, heads, share, k, splits, row_pages, pages, kv_heads;
  int32_t tiles;  // that a workgroup works on at a time, a power of two
  float scale2;  // scale * log2(e): softmax by powers of two
  Div div;
};

// Tokens of row `row` to look at, and the pool slot of the t-th of them.
__device__ __forceinline__ int32_t tokens_of(const Args& a, int row, int32_t& len) {
  const int32_t cap = a.row_pages * static_cast<int32_t>(a.div.P);
  len = min(max(a.lengths[row], 0), cap);
  return a.idx ? (len > 0 ? a.k : 0) : len;
}

__device__ __forceinline__ uint32_t slot_of(const Args& a, int row, int kvh, int32_t len, int32_t t) {
  const int32_t s = a.idx ? a.idx[static_cast<int64_t>(row) * a.k + t] : t;
  if (s < 0 || s >= len) return kHidden;
  const uint32_t e = div_page(s, a.div);
  const int32_t page = a.table[static_cast<int64_t>(row) * a.row_pages + e];
  if (page < 0 || page >= a.pages) return kHidden;
  return (static_cast<uint32_t>(page) * a.kv_heads + kvh) * a.div.P + (s - e * a.div.P);
}

// Workgroups go round the 8 XCDs, each with its own L2: the chunks of query
// heads that read the same cached rows are 8 workgroups apart, on one XCD.
__device__ __forceinline__ void unit_chunk(int chunks, int& unit, int& chunk) {
  const int b = blockIdx.x;
  chunk = b / 8 % chunks;
  unit = b / (8 * chunks) * 8 + b % 8;
}

// How the tiles of a row are divided: every split takes the same number, a
// multiple of those that its workgroup works on at a time (four waves, or a
// latent kernel's two token groups).
constexpr int kTileTokens = 32;
__device__ __forceinline__ int32_t tiles_per_split(const Args& a, int32_t todo) {
  const int32_t tiles = (todo + kTileTokens - 1) / kTileTokens;
  return (((tiles + a.splits - 1) / a.splits) + a.tiles - 1) & ~(a.tiles - 1);
}

constexpr int kStage = 2048;  // tokens whose slots (and scales) are in LDS at a time

// Eight e4m3 codes -> bf16, exact.
__device__ __forceinline__ bf16x8 fp8x8_to_bf16(uint32_t lo, uint32_t hi) {
  uint4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true));
  return as_bf16x8(r);
}

// What the sums of a part with maximum m and sum l count under the common
// maximum.  A part without tokens counts nothing; a NaN sum without a maximum
// (every score NaN) stays one.
__device__ __forceinline__ float part_factor(float m, float l, float mall) {
  if (m == -INFINITY) return l == 0.f ? 0.f : 1.f;
  return __builtin_amdgcn_exp2f(m - mall);
}

// Reductions over the four lane groups of a query head (lanes l % 16 alike).
__device__ __forceinline__ float groups_max(float x) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float groups_sum(float x) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// log of the sum of exponentials from its log2 maximum and scaled sum.
__device__ __forceinline__ float final_lse(float m, float l) {
  return (m == -INFINITY ? 0.f : m * kLn2) + __logf(l);
}


// The splits of one (row, head) joined by one workgroup: D / 4 threads hold
// four dimensions each, and 1024 / D groups of them take every such split; the
// groups' sums are added in order.  A launch of its own: a workgroup that waits
// for its peers' sums would need an arrival count that is known to start at zero.
// 32 heads of one row, 16 splits: 3.5 us, a launch and two dependent loads; 32
// rows of 128 heads of 512 in 4 splits (34 MB) 8.6 us, 3.9 TB/s.
template <int D>
__global__ __launch_bounds__(256) void attend_join_kernel(Args a) {
  constexpr int T = D / 4, GS = 256 / T;
  __shared__ float4 sums[GS][T];
  __shared__ float total[GS];
  const int head = blockIdx.x, row = blockIdx.y;
  const int d = threadIdx.x % T, grp = threadIdx.x / T;
  int32_t len;
  const int32_t todo = tokens_of(a, row, len);
  const int32_t per = tiles_per_split(a, todo) * kTileTokens;
  const int32_t n = todo > 0 ? (todo + per - 1) / per : 1;  // split 0 always writes
  const int64_t at = static_cast<int64_t>(row) * a.heads + head;
  const float2* ml = a.part_ml + at * a.splits;
  float m = -INFINITY;
  for (int s = lane_id(); s < n; s += kWave) m = fmaxf(m, ml[s].x);
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
  const float4* src = reinterpret_cast<const float4*>(a.part_o + at * a.splits * D) + d;
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = grp; s < n; s += GS) {
    const float2 x = ml[s];
    const float4 y = src[static_cast<int64_t>(s) * T];
    const float f = part_factor(x.x, x.y, m);
    l += x.y * f;
    o.x += y.x * f;
    o.y += y.y * f;
    o.z += y.z * f;
    o.w += y.w * f;
  }
  if (n > 1) {  // with one split, group 0 has it all
    sums[grp][d] = o;
    if (d == 0) total[grp] = l;
    __syncthreads();
    if (grp != 0) return;
    for (int i = 1; i < min(GS, n); ++i) {
      const float4 y = sums[i][d];
      l += total[i];
      o.x += y.x;
      o.y += y.y;
      o.z += y.z;
      o.w += y.w;
    }
  }
  if (grp != 0) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (d == 0 && a.lse) a.lse[at] = l == 0.f ? -INFINITY : final_lse(m, l);
  bf16x2 y0, y1;
  y0[0] = static_cast<__bf16>(o.x * inv);
  y0[1] = static_cast<__bf16>(o.y * inv);
  y1[0] = static_cast<__bf16>(o.z * inv);
  y1[1] = static_cast<__bf16>(o.w * inv);
  *reinterpret_cast<uint2*>(a.out + at * D + 4 * d) =
      make_uint2(__builtin_bit_cast(uint32_t, y0), __builtin_bit_cast(uint32_t, y1));
}

// Latent caches; the grid is that of launch_attend's plan.
constexpr int kLatentK = 576, kLatentV = 512;
constexpr int kLatentHeads = 64;  // query heads of a workgroup
hipError_t launch_attend_latent(int32_t dtype, const Args& a, uint32_t grid, hipStream_t st);

}  // namespace misa
