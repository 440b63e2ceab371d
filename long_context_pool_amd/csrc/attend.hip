// Attention of one new token per row over a paged cache (misa_attend in
// misa.h): every cached token of the row, or those of an index list.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "mfma.hpp"

namespace misa {

namespace {

typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(2))) int i32x2;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The sums are rescaled to a new maximum only when a score exceeds the old one
// by this much (log2): until then weights go up to 2^8, which loses nothing in
// fp32 and in the weights' bf16 parts, and O's registers are left alone.
constexpr float kSlack = 8.f;
constexpr uint32_t kHidden = 0xFFFFFFFFu;  // the slot of a token that is not visible

// n / P for 0 <= n < 2^31 by a multiplication: with l = ceil(log2 P), m =
// floor(2^(31+l) / P) + 1 exceeds 2^(31+l) / P by less than 2^l / P * P, so
// n * m >> (31+l) is the quotient.
struct Div {
  uint32_t m, shift, P;
};

Div make_div(uint32_t P) {
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

// How the tiles of a row are divided: every split takes `per` tiles, a
// multiple of the workgroup's four waves.
constexpr int kTileTokens = 32;
__device__ __forceinline__ int32_t tiles_per_split(int32_t todo, int32_t splits) {
  const int32_t tiles = (todo + kTileTokens - 1) / kTileTokens;
  return (((tiles + splits - 1) / splits) + 3) & ~3;
}

constexpr int kStage = 2048;  // tokens whose slots (and scales) are in LDS at a time

// ---------------------------------------------------------------- dk = dv

// Eight e4m3 codes -> bf16, exact.
__device__ __forceinline__ bf16x8 fp8x8_to_bf16(uint32_t lo, uint32_t hi) {
  uint4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true));
  return as_bf16x8(r);
}

// Two columns of V^T from the dwords (two bf16 dimensions each) of eight value
// rows, and their products with both parts of the weights.
template <int RT, int NJ>
__device__ __forceinline__ void columns(const uint32_t (&w)[8], const bf16x8 (&ph)[RT],
                                        const bf16x8 (&pl)[RT], f32x4 (&acc)[RT][NJ], int j) {
  uint4 even, odd;
  even.x = __builtin_amdgcn_perm(w[1], w[0], 0x05040100);
  even.y = __builtin_amdgcn_perm(w[3], w[2], 0x05040100);
  even.z = __builtin_amdgcn_perm(w[5], w[4], 0x05040100);
  even.w = __builtin_amdgcn_perm(w[7], w[6], 0x05040100);
  odd.x = __builtin_amdgcn_perm(w[1], w[0], 0x07060302);
  odd.y = __builtin_amdgcn_perm(w[3], w[2], 0x07060302);
  odd.z = __builtin_amdgcn_perm(w[5], w[4], 0x07060302);
  odd.w = __builtin_amdgcn_perm(w[7], w[6], 0x07060302);
  const bf16x8 v0 = as_bf16x8(even), v1 = as_bf16x8(odd);
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    acc[r][j] = mfma16_bf16(v0, ph[r], acc[r][j]);
    acc[r][j + 1] = mfma16_bf16(v1, ph[r], acc[r][j + 1]);
    acc[r][j] = mfma16_bf16(v0, pl[r], acc[r][j]);
    acc[r][j + 1] = mfma16_bf16(v1, pl[r], acc[r][j + 1]);
  }
}

// The dimension that product j gives for row c of V^T (the lane that loaded it).
template <int D, int DT>
__device__ __forceinline__ int value_dim(int c, int j) {
  constexpr int per = DT == kFP8 ? D / 16 : (D / 16 < 8 ? D / 16 : 8);  // contiguous per lane
  return (j / per) * 16 * per + c * per + j % per;
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


// One workgroup of four waves per (split, kv head and chunk of 16 * RT query
// heads, row); a wave takes every fourth tile of 32 tokens.  All products are
// transposed, so that a lane keeps one query head (l % 16):
//   S^T = K Q^T   16x16x32 bf16, rows = tokens, columns = heads,
//   O^T = V^T P^T with P^T read from S^T's registers as they are: lane group g
//         holds the tokens 4g .. 4g+3 of both 16-token halves, and V's rows
//         are loaded in that order.  Eight rows of V make eight columns of V^T
//         by byte permutes in registers.
// A weight goes into the product as two bf16 parts (its rounding and the rest,
// 2^-17 together), or the result would be off by a second bf16 rounding; the
// cached values are exact in bf16.  Maximum, sums and O stay in fp32 registers.
template <int D, int DT, int RT>
__global__ __launch_bounds__(256) void attend_kernel(Args a) {
  constexpr int EB = DT == kFP8 ? 1 : 2;
  constexpr int ROW = D * EB;       // bytes of a cached row
  constexpr int KL = ROW / 64;      // 16-byte loads per lane and key row
  constexpr int KS = D / 32;        // matrix steps of a dot product
  constexpr int VB = D / 16 * EB;   // bytes of a value row per lane
  constexpr int VW = VB / 4;
  constexpr int NJ = D / 16;        // products of 16 dimensions
  constexpr int NR = RT * (NJ * 4 + 1);  // registers of a wave's result
  constexpr bool kFp8 = DT == kFP8;
  struct Stage {
    uint32_t slot[kStage];
    float ks[kFp8 ? kStage : 4];
    float vs[kFp8 ? kStage : 4];
  };
  union Shared {
    Stage st;
    float red[2][NR][kWave];
  };
  __shared__ __attribute__((aligned(16))) Shared sh;
  __shared__ float top[4][RT][16];

  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int split = blockIdx.x, row = blockIdx.z;
  const int chunks = (a.share + 16 * RT - 1) / (16 * RT);
  const int kvh = blockIdx.y / chunks, chunk = blockIdx.y % chunks;
  const int head0 = kvh * a.share + chunk * 16 * RT;       // first query head
  const int nheads = min(16 * RT, a.share - chunk * 16 * RT);
  int32_t len;
  const int32_t todo = tokens_of(a, row, len);
  const int32_t per = tiles_per_split(todo, a.splits) * kTileTokens;
  const int32_t t0 = split * per, t1 = min(t0 + per, todo);
  if (t0 >= t1 && split > 0) return;  // nothing here; the join does not look at it

  // Q^T fragments: head c of each row tile, the dimensions that K's loads give.
  bf16x8 qf[RT][KS];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int h = r * 16 + c;
    const uint16_t* src = a.q + (static_cast<int64_t>(row) * a.heads + head0 + (h < nheads ? h : 0)) * D;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d0 = kFp8 ? 64 * (s / 2) + 16 * g + 8 * (s % 2) : 32 * s + 8 * g;
      qf[r][s] = as_bf16x8(*reinterpret_cast<const uint4*>(src + d0));
    }
  }

  f32x4 acc[RT][NJ];
  float m[RT], l[RT];  // reference maximum of the head (all lanes alike), this lane's part of the sum
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[r][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  uint4 kreg[2][KL];
  uint32_t vreg[8][VW];
  auto load_k = [&](int tile) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t s = sh.st.slot[tile * 32 + 16 * h + c];
      const uint8_t* p = a.k_pages + static_cast<uint64_t>(s == kHidden ? 0 : s) * ROW + g * 16;
#pragma unroll
      for (int u = 0; u < KL; ++u) kreg[h][u] = *reinterpret_cast<const uint4*>(p + u * 64);
    }
  };
  auto load_v = [&](int tile) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t s = sh.st.slot[tile * 32 + (i / 4) * 16 + 4 * g + i % 4];
      const uint8_t* p = a.v_pages + static_cast<uint64_t>(s == kHidden ? 0 : s) * ROW;
      if constexpr (VB == 4) {
        vreg[i][0] = *reinterpret_cast<const uint32_t*>(p + c * 4);
      } else if constexpr (VB == 8) {
        const uint2 x = *reinterpret_cast<const uint2*>(p + c * 8);
        vreg[i][0] = x.x;
        vreg[i][1] = x.y;
      } else {
#pragma unroll
        for (int u = 0; u < VB / 16; ++u) {
          const uint4 x = *reinterpret_cast<const uint4*>(p + u * 256 + c * 16);
          vreg[i][4 * u] = x.x;
          vreg[i][4 * u + 1] = x.y;
          vreg[i][4 * u + 2] = x.z;
          vreg[i][4 * u + 3] = x.w;
        }
      }
    }
  };

  for (int32_t base = t0; base < t1; base += kStage) {
    const int32_t count = min(kStage, t1 - base);
    const int32_t tiles = (count + kTileTokens - 1) / kTileTokens;
    if (base != t0) __syncthreads();
    for (int32_t i = threadIdx.x; i < tiles * kTileTokens; i += 256) {
      const uint32_t s = i < count ? slot_of(a, row, kvh, len, base + i) : kHidden;
      sh.st.slot[i] = s;
      if constexpr (kFp8) {
        sh.st.ks[i] = s == kHidden ? 0.f : a.k_scale[s];
        sh.st.vs[i] = s == kHidden ? 0.f : a.v_scale[s];
      }
    }
    __syncthreads();
    if (wave < tiles) {
      load_k(wave);
      load_v(wave);
    }
    for (int32_t tile = wave; tile < tiles; tile += 4) {
      const bool more = tile + 4 < tiles;
      // scores of this lane's eight tokens (i < 4: token 4g + i, else 16 + 4g + i - 4)
      f32x4 st[RT][2];
#pragma unroll
      for (int r = 0; r < RT; ++r) st[r][0] = st[r][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          bf16x8 kf;
          if constexpr (kFp8) {
            const uint4 x = kreg[h][s / 2];
            kf = fp8x8_to_bf16(s % 2 ? x.z : x.x, s % 2 ? x.w : x.y);
          } else {
            kf = as_bf16x8(kreg[h][s]);
          }
#pragma unroll
          for (int r = 0; r < RT; ++r) st[r][h] = mfma16_bf16(kf, qf[r][s], st[r][h]);
        }
      if (more) load_k(tile + 4);
      uint32_t sl[8];
      float ks[8], vs[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = tile * 32 + 16 * h + 4 * g;
        const uint4 x = *reinterpret_cast<const uint4*>(&sh.st.slot[at]);
        sl[4 * h] = x.x; sl[4 * h + 1] = x.y; sl[4 * h + 2] = x.z; sl[4 * h + 3] = x.w;
        if constexpr (kFp8) {
          const float4 y = *reinterpret_cast<const float4*>(&sh.st.ks[at]);
          ks[4 * h] = y.x; ks[4 * h + 1] = y.y; ks[4 * h + 2] = y.z; ks[4 * h + 3] = y.w;
          const float4 z = *reinterpret_cast<const float4*>(&sh.st.vs[at]);
          vs[4 * h] = z.x; vs[4 * h + 1] = z.y; vs[4 * h + 2] = z.z; vs[4 * h + 3] = z.w;
        }
      }
      bool hidden = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) hidden |= sl[i] == kHidden;
      bf16x8 ph[RT], pl[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float x[8], high = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float y = st[r][i / 4][i % 4] * a.scale2;
          if constexpr (kFp8) y *= ks[i];
          x[i] = sl[i] == kHidden ? -INFINITY : y;
          high = fmaxf(high, x[i]);
        }
        if (__any(high > m[r] + kSlack)) {  // wave-uniform
          const float next = fmaxf(m[r], groups_max(high));
          const float f = next == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[r] - next);
          m[r] = next;
          l[r] *= f;
#pragma unroll
          for (int j = 0; j < NJ; ++j) acc[r][j] *= f;
        }
        const float mb = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = __builtin_amdgcn_exp2f(x[i] - mb);
          l[r] += p;
          const float w = kFp8 ? p * vs[i] : p;
          const __bf16 hi = static_cast<__bf16>(w);
          ph[r][i] = hi;
          pl[r][i] = static_cast<__bf16>(w - static_cast<float>(hi));
        }
      }
      if (__any(hidden)) {  // hidden slots may hold anything: 0 * NaN must not reach O
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int u = 0; u < VW; ++u) vreg[i][u] = sl[i] == kHidden ? 0u : vreg[i][u];
      }
#pragma unroll
      for (int u = 0; u < VW; ++u) {
        // dword u of the eight rows: 2 (bf16) or 4 (fp8) columns of V^T
        if constexpr (kFp8) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              w[i] = __builtin_bit_cast(
                  uint32_t, half ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(vreg[i][u], 1.f, true)
                                 : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(vreg[i][u], 1.f, false));
            columns(w, ph, pl, acc, 4 * u + 2 * half);
          }
        } else {
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = vreg[i][u];
          columns(w, ph, pl, acc, 2 * u);
        }
      }
      if (more) load_v(tile + 4);
    }
  }

  // Join the four waves: common maximum, then a tree through LDS into wave 0.
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    l[r] = groups_sum(l[r]);
    if (g == 0) top[wave][r][c] = m[r];
  }
  __syncthreads();
  float mall[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    mall[r] = fmaxf(fmaxf(top[0][r][c], top[1][r][c]), fmaxf(top[2][r][c], top[3][r][c]));
    const float f = part_factor(m[r], l[r], mall[r]);
    l[r] *= f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[r][j] *= f;
  }
#pragma unroll
  for (int step = 2; step >= 1; step >>= 1) {
    if (wave >= step && wave < 2 * step) {
      int n = 0;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        sh.red[wave - step][n++][lane] = l[r];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) sh.red[wave - step][n++][lane] = acc[r][j][e];
      }
    }
    __syncthreads();
    if (wave < step) {
      int n = 0;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        l[r] += sh.red[wave][n++][lane];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[r][j][e] += sh.red[wave][n++][lane];
      }
    }
    __syncthreads();
  }
  if (wave != 0) return;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int h = r * 16 + c;
    if (h >= nheads) continue;
    const int64_t at = static_cast<int64_t>(row) * a.heads + head0 + h;
    if (a.splits == 1) {
      const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
      if (g == 0 && a.lse) a.lse[at] = l[r] == 0.f ? -INFINITY : final_lse(mall[r], l[r]);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < NJ; j += 2) {
          bf16x2 x;
          x[0] = static_cast<__bf16>(acc[r][j][e] * inv);
          x[1] = static_cast<__bf16>(acc[r][j + 1][e] * inv);
          *reinterpret_cast<bf16x2*>(a.out + at * D + value_dim<D, DT>(4 * g + e, j)) = x;
        }
    } else {
      const int64_t part = at * a.splits + split;
      if (g == 0) a.part_ml[part] = make_float2(mall[r], l[r]);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < NJ; j += 4)
          *reinterpret_cast<float4*>(a.part_o + part * D + value_dim<D, DT>(4 * g + e, j)) =
              make_float4(acc[r][j][e], acc[r][j + 1][e], acc[r][j + 2][e], acc[r][j + 3][e]);
    }
  }
}

// The splits of one (row, head) joined by one workgroup: D / 4 threads hold
// four dimensions each, and 1024 / D groups of them take every such split; the
// groups' sums are added in order.
template <int D>
__global__ __launch_bounds__(256) void attend_join_kernel(Args a) {
  constexpr int T = D / 4, GS = 256 / T;
  __shared__ float4 sums[GS][T];
  __shared__ float total[GS];
  const int head = blockIdx.x, row = blockIdx.y;
  const int d = threadIdx.x % T, grp = threadIdx.x / T;
  int32_t len;
  const int32_t todo = tokens_of(a, row, len);
  const int32_t per = tiles_per_split(todo, a.splits) * kTileTokens;
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

// ---------------------------------------------------------------- latent rows

// Every wave of the workgroup arrives, from whichever of its barriers; nothing
// moves over it.  LDS writes of this wave are done.
__device__ __forceinline__ void barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// This wave's direct loads to LDS have landed.
__device__ __forceinline__ void landed() { __builtin_amdgcn_s_waitcnt(0x0F70); }

constexpr int kLatentK = 576, kLatentV = 512;
constexpr int kLatentHeads = 64;  // query heads of a workgroup
constexpr int kLatentStage = 512;  // tokens whose slots are in LDS at a time

// One workgroup of eight waves per (split, 64 query heads, row): waves 0-3 and
// 4-7 are two token groups, and wave w of a group has the query heads 16 (w %
// 4) .. +15.  A group's tile of 32 cached rows goes to LDS once, by direct
// loads into one of two buffers while the other is worked on, and its four
// waves read it twice: as K for the scores, and its first 512 elements, by
// transposing reads, as V^T.  The products are those of attend_kernel.
//
// The groups work half a step apart: while one has its scores and softmax, the
// other has its values, so that LDS, matrix and vector work overlap.
//
// A tile is nine column blocks of 8 (fp8: 4) chunks of 16 bytes, each [32 rows]
// [chunks]: a direct load fills 64 consecutive chunks, here of 8 (16) rows, from
// whole 128- (64-) byte pieces of them.  Chunk x of row r sits at x ^ swz(r) of
// its block, so that neither the 16 rows of a key fragment nor the rows of a
// transposing read share banks.
template <int DT>
__global__ __launch_bounds__(512) void attend_latent_kernel(Args a) {
  constexpr bool kFp8 = DT == kFP8;
  constexpr int EB = kFp8 ? 1 : 2;
  constexpr int CH = kLatentK * EB / 16;     // chunks of a cached row
  constexpr int CB = CH / 9;                 // chunks of a column block
  constexpr int KU = kLatentK * EB / 64;     // key chunks per lane
  constexpr int KS = kLatentK / 32;          // matrix steps of a score
  constexpr int NJ = kLatentV / 16;
  constexpr int QL = 3;      // query fragments in LDS: in registers they spill
  constexpr int kKeyAhead = 6, kAhead = 4;  // LDS reads under way
  // The two buffers are arrays of their own: the compiler orders a read after
  // every direct load that might be to the same array.
  __shared__ __attribute__((aligned(128))) uint4 even[2][32 * CH];  // [token group]
  __shared__ __attribute__((aligned(128))) uint4 odd[2][32 * CH];
  __shared__ uint4 q_lds[4][QL][kWave];
  __shared__ __attribute__((aligned(16))) uint32_t slots[kLatentStage];
  __shared__ __attribute__((aligned(16))) float scales[kFp8 ? kLatentStage : 4];
  __shared__ float top[4][16], sum[4][16];

  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int hw = wave & 3, grp = wave >> 2;
  // Workgroups go round the 8 XCDs: the head chunks of one (row, split) are 8
  // apart, on one XCD, so that the second reads the cache rows from its L2.
  const int chunks = (a.heads + kLatentHeads - 1) / kLatentHeads;
  const int chunk = blockIdx.x / 8 % chunks;
  const int unit = blockIdx.x / (8 * chunks) * 8 + blockIdx.x % 8;
  const int row = unit / a.splits, split = unit - row * a.splits;
  if (row >= a.rows) return;
  const int head0 = chunk * kLatentHeads + hw * 16;
  int32_t len;
  const int32_t todo = tokens_of(a, row, len);
  const int32_t per = tiles_per_split(todo, a.splits) * kTileTokens;
  const int32_t t0 = split * per, t1 = min(t0 + per, todo);
  if (t0 >= t1 && split > 0) return;

  bf16x8 qf[KS - QL];
  {
    const int h = head0 + c < a.heads ? head0 + c : 0;
    const uint16_t* src = a.q + (static_cast<int64_t>(row) * a.heads + h) * kLatentK;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d0 = kFp8 ? 64 * (s / 2) + 16 * g + 8 * (s % 2) : 32 * s + 8 * g;
      const uint4 x = *reinterpret_cast<const uint4*>(src + d0);
      if (s < KS - QL)
        qf[s] = as_bf16x8(x);
      else if (grp == 0)
        q_lds[hw][s - (KS - QL)][lane] = x;
    }
  }
  auto query = [&](int s) {
    return s < KS - QL ? qf[s < KS - QL ? s : 0] : as_bf16x8(q_lds[hw][s < KS - QL ? 0 : s - (KS - QL)][lane]);
  };
  f32x4 acc[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;

  auto swz = [](int r) { return kFp8 ? (r >> 2 & 3) ^ (r >> 4 << 1) : (r >> 1 & 1) << 2 | (r >> 2 & 3); };
  // The group's four waves load its tile of pair `it`.  A direct load takes one
  // column block of 8 (fp8: 16) rows; this lane always has the same row, r, and
  // the same chunk of it, so a tile costs it one slot.  Whether any of the
  // wave's slots is hidden is returned.
  constexpr int RL = kWave / CB;                  // rows of a load
  const int r = (kFp8 ? hw % 2 : hw) * RL + lane / CB;
  const int block0 = kFp8 ? hw / 2 : 0;           // this wave's column blocks: every other one for fp8
  constexpr int BS = kFp8 ? 2 : 1;
  const int lds0 = (kFp8 ? hw % 2 : hw) * kWave;  // first chunk of a load in its block
  auto issue = [&](int it, uint4 (&tile)[2][32 * CH]) {
    const uint32_t s = slots[(2 * it + grp) * 32 + r];
    const uint8_t* src = a.k_pages + static_cast<uint64_t>(s == kHidden ? 0 : s) * (kLatentK * EB) +
                         block0 * (CB * 16) + (lane % CB ^ swz(r)) * 16;
    uint4* buf = tile[grp] + block0 * (32 * CB) + lds0;
#pragma unroll
    for (int n = 0; n < 9; n += BS)
      if (n + block0 < 9)
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(src + n * (CB * 16)),
                                         (__attribute__((address_space(3))) void*)(buf + n * (32 * CB)), 16, 0, 0);
    return static_cast<bool>(__any(s == kHidden));
  };
  // Hidden slots may hold anything, and 0 * NaN must not reach O: zeros in
  // their place, by the lanes that loaded them.
  auto clear_hidden = [&](int it, uint4 (&tile)[2][32 * CH]) {
    if (slots[(2 * it + grp) * 32 + r] != kHidden) return;
    for (int n = block0; n < 9; n += BS) tile[grp][n * (32 * CB) + lds0 + lane] = make_uint4(0, 0, 0, 0);
  };

  // LDS bytes of this lane's first key and value chunks.  A step within a
  // column block is an exclusive or of the address bits that the swizzle
  // changes; every other step is an immediate offset.
  constexpr int kVStep = 16 * EB;  // bytes of 16 dimensions
  constexpr int kBlock = 32 * CB * 16, kRow = CB * 16;
  const int koff = c * kRow + (g ^ swz(c)) * 16;
  int voff;  // the row that this lane reads for its 16 lanes' transposed 4 x 16 (fp8: 8 x 16)
  if constexpr (kFp8) {
    const int i = c / 2, vr = (i / 4) * 16 + 4 * g + i % 4;
    voff = vr * kRow + swz(vr) * 16 + c % 2 * 8;
  } else {
    const int vr = 4 * g + c / 4;
    voff = vr * kRow + ((c / 2 % 2) ^ swz(vr)) * 16 + c % 2 * 8;
  }

  bool hidden = false;
  auto step = [&](int it, int pairs, uint4 (&tile)[2][32 * CH], uint4 (&next)[2][32 * CH]) __attribute__((always_inline)) {
    landed();  // this wave's loads ...
    if (hidden) clear_hidden(it, tile);
    barrier();  // ... and the group's, and its other buffer is free
    const uint8_t* buf = reinterpret_cast<const uint8_t*>(tile[grp]);
    const int first = (2 * it + grp) * 32;
    // Scores.  Fragment f = 2u + h: 16 bytes of token half h; kAhead reads are
    // under way (the barriers keep the compiler from undoing that).
    auto key = [&](int f) {
      const int u = f / 2, h = f % 2;
      const int x = kFp8 ? 32 * h : u % 2 * 64;  // fp8: the swizzle of rows 16 and up
      return *reinterpret_cast<const uint4*>(buf + (koff ^ x) + 16 * h * kRow + (kFp8 ? u : u / 2) * kBlock);
    };
    f32x4 st[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
    uint4 kb[kKeyAhead];
#pragma unroll
    for (int f = 0; f < kKeyAhead; ++f) kb[f] = key(f);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int f = 0; f < 2 * KU; ++f) {
      const uint4 x = kb[f % kKeyAhead];
      if constexpr (kFp8) {
        st[f % 2] = mfma16_bf16(fp8x8_to_bf16(x.x, x.y), query(f / 2 * 2), st[f % 2]);
        st[f % 2] = mfma16_bf16(fp8x8_to_bf16(x.z, x.w), query(f / 2 * 2 + 1), st[f % 2]);
      } else {
        st[f % 2] = mfma16_bf16(as_bf16x8(x), query(f / 2), st[f % 2]);
      }
      if (f + kKeyAhead < 2 * KU) kb[f % kKeyAhead] = key(f + kKeyAhead);
      __builtin_amdgcn_sched_barrier(0);
    }
    // V^T fragment j: 16 dimensions of this lane group's eight tokens.
    auto value = [&](int j, uint4& v) {
      const uint8_t* p = buf + (voff ^ (j % 4 * kVStep)) + j / 4 * kBlock;
      if constexpr (kFp8) {
        const i32x2 y = __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2*)p);
        v.x = y[0];
        v.y = y[1];
      } else {
        const s16x4 y0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
        const s16x4 y1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4*)(p + 16 * kRow));
        v = __builtin_bit_cast(uint4, __builtin_shufflevector(y0, y1, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    };
    uint32_t sl[8];
    float ks[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = first + 16 * h + 4 * g;
      const uint4 x = *reinterpret_cast<const uint4*>(&slots[at]);
      sl[4 * h] = x.x; sl[4 * h + 1] = x.y; sl[4 * h + 2] = x.z; sl[4 * h + 3] = x.w;
      if constexpr (kFp8) {
        const float4 y = *reinterpret_cast<const float4*>(&scales[at]);
        ks[4 * h] = y.x; ks[4 * h + 1] = y.y; ks[4 * h + 2] = y.z; ks[4 * h + 3] = y.w;
      }
    }
    float x[8], high = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float y = st[i / 4][i % 4] * a.scale2;
      if constexpr (kFp8) y *= ks[i];
      x[i] = sl[i] == kHidden ? -INFINITY : y;
      high = fmaxf(high, x[i]);
    }
    if (__any(high > m + kSlack)) {
      const float next = fmaxf(m, groups_max(high));
      const float f = next == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - next);
      m = next;
      l *= f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[j] *= f;
    }
    const float mb = m == -INFINITY ? 0.f : m;
    bf16x8 ph, pl;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = __builtin_amdgcn_exp2f(x[i] - mb);
      l += p;
      const float w = kFp8 ? p * ks[i] : p;
      const __bf16 hi = static_cast<__bf16>(w);
      ph[i] = hi;
      pl[i] = static_cast<__bf16>(w - static_cast<float>(hi));
    }
    barrier();
    if (it + 1 < pairs) hidden = issue(it + 1, next);
    __builtin_amdgcn_sched_barrier(0);
    uint4 vb[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) value(j, vb[j]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < NJ; j += 2) {
      const uint4 y0 = vb[j % kAhead], y1 = vb[(j + 1) % kAhead];
      const bf16x8 v0 = kFp8 ? fp8x8_to_bf16(y0.x, y0.y) : as_bf16x8(y0);
      const bf16x8 v1 = kFp8 ? fp8x8_to_bf16(y1.x, y1.y) : as_bf16x8(y1);
      acc[j] = mfma16_bf16(v0, ph, acc[j]);
      acc[j + 1] = mfma16_bf16(v1, ph, acc[j + 1]);
      acc[j] = mfma16_bf16(v0, pl, acc[j]);
      acc[j + 1] = mfma16_bf16(v1, pl, acc[j + 1]);
      if (j + kAhead < NJ) {
        value(j + kAhead, vb[j % kAhead]);
        value(j + 1 + kAhead, vb[(j + 1) % kAhead]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  for (int32_t base = t0; base < t1; base += kLatentStage) {
    const int32_t count = min(kLatentStage, t1 - base);
    const int32_t pairs = (count + 63) / 64;
    if (base != t0) __syncthreads();
    for (int32_t i = threadIdx.x; i < pairs * 64; i += 512) {
      const uint32_t s = i < count ? slot_of(a, row, 0, len, base + i) : kHidden;
      slots[i] = s;
      if constexpr (kFp8) scales[i] = s == kHidden ? 0.f : a.k_scale[s];
    }
    __syncthreads();
    hidden = issue(0, even);
    if (grp == 1) barrier();  // half a step behind
    for (int32_t it = 0; it < pairs; it += 2) {
      step(it, pairs, even, odd);
      if (it + 1 < pairs) step(it + 1, pairs, odd, even);
    }
    if (grp == 0) barrier();  // as many as group 1
  }

  // Join the two token groups: group 1 hands its sums to group 0 through LDS, a
  // quarter of the dimensions at a time.
  constexpr int kPart = NJ / 4;  // products of a quarter
  l = groups_sum(l);
  __syncthreads();
  if (grp == 1 && g == 0) {
    top[hw][c] = m;
    sum[hw][c] = l;
  }
  const int64_t at = static_cast<int64_t>(row) * a.heads + min(head0 + c, a.heads - 1);
  const int64_t part = at * a.splits + split;
  const bool mine = grp == 0 && head0 + c < a.heads;
  float f0 = 0.f, f1 = 0.f;
#pragma unroll
  for (int qt = 0; qt < 4; ++qt) {
    float4* red = reinterpret_cast<float4*>(qt % 2 ? odd : even);  // [product][wave][lane]
    if (grp == 1) {
#pragma unroll
      for (int j = 0; j < kPart; ++j) {
        const f32x4 y = acc[qt * kPart + j];
        red[(j * 4 + hw) * kWave + lane] = make_float4(y[0], y[1], y[2], y[3]);
      }
    }
    __syncthreads();
    if (qt == 0 && grp == 0) {
      const float m1 = top[hw][c], l1 = sum[hw][c];
      const float mall = fmaxf(m, m1);
      f0 = part_factor(m, l, mall);
      f1 = part_factor(m1, l1, mall);
      const float lall = l * f0 + l1 * f1;
      if (g == 0 && mine) {
        if (a.splits > 1)
          a.part_ml[part] = make_float2(mall, lall);
        else if (a.lse)
          a.lse[at] = lall == 0.f ? -INFINITY : final_lse(mall, lall);
      }
      if (a.splits == 1) {
        const float inv = lall == 0.f ? 0.f : 1.f / lall;
        f0 *= inv;
        f1 *= inv;
      }
    }
    if (mine) {
#pragma unroll
      for (int j = 0; j < kPart; ++j) {
        const int d = 16 * (qt * kPart + j) + 4 * g;
        const f32x4 y = acc[qt * kPart + j];
        const float4 z = red[(j * 4 + hw) * kWave + lane];
        const float4 o = make_float4(y[0] * f0 + z.x * f1, y[1] * f0 + z.y * f1, y[2] * f0 + z.z * f1,
                                     y[3] * f0 + z.w * f1);
        if (a.splits > 1) {
          *reinterpret_cast<float4*>(a.part_o + part * kLatentV + d) = o;
        } else {
          bf16x2 u, v;
          u[0] = static_cast<__bf16>(o.x);
          u[1] = static_cast<__bf16>(o.y);
          v[0] = static_cast<__bf16>(o.z);
          v[1] = static_cast<__bf16>(o.w);
          *reinterpret_cast<uint2*>(a.out + at * kLatentV + d) =
              make_uint2(__builtin_bit_cast(uint32_t, u), __builtin_bit_cast(uint32_t, v));
        }
      }
    }
  }
}

constexpr int kMinSplitTokens = 128;  // a split gives each wave a tile

// Query heads of a workgroup: a matrix tile of 16, or two where a kv head has
// more and the registers hold them.
int group_heads(const Cache& c, int32_t share) {
  if (c.latent()) return kLatentHeads;
  return share > 16 && c.dk <= 128 ? 32 : 16;
}

struct Plan {
  int32_t chunks, splits;
};

Plan plan(const Cache& c, int32_t heads, int32_t k) {
  const int32_t share = heads / c.kv_heads;
  const int32_t per = group_heads(c, share);
  Plan p;
  p.chunks = (share + per - 1) / per;
  const int64_t groups = static_cast<int64_t>(c.rows) * c.kv_heads * p.chunks;
  const int64_t most = k > 0 ? k : static_cast<int64_t>(c.row_pages) * c.P;
  int64_t s = c.latent() ? (k > 0 ? 256 : 512) / groups : (1024 + groups - 1) / groups;
  s = std::min<int64_t>(s, (most + kMinSplitTokens - 1) / kMinSplitTokens);
  p.splits = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(s, 128)));
  return p;
}

template <int D, int DT>
hipError_t launch_dim(const Cache& c, const Args& a, const Plan& p, hipStream_t st) {
  const dim3 grid(p.splits, c.kv_heads * p.chunks, c.rows);
  if constexpr (D <= 128) {
    if (group_heads(c, a.share) == 32)
      attend_kernel<D, DT, 2><<<grid, 256, 0, st>>>(a);
    else
      attend_kernel<D, DT, 1><<<grid, 256, 0, st>>>(a);
  } else {
    attend_kernel<D, DT, 1><<<grid, 256, 0, st>>>(a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  attend_join_kernel<D><<<dim3(a.heads, c.rows), 256, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_latent(const Cache& c, const Args& a, const Plan& p, hipStream_t st) {
  const int64_t units = (static_cast<int64_t>(c.rows) * p.splits + 7) / 8 * 8;
  const uint32_t grid = static_cast<uint32_t>(units * p.chunks);
  if (c.dtype == kFP8)
    attend_latent_kernel<kFP8><<<grid, 512, 0, st>>>(a);
  else
    attend_latent_kernel<kBF16><<<grid, 512, 0, st>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  attend_join_kernel<kLatentV><<<dim3(a.heads, c.rows), 256, 0, st>>>(a);
  return hipGetLastError();
}

template <int D>
hipError_t launch_type(const Cache& c, const Args& a, const Plan& p, hipStream_t st) {
  return c.dtype == kFP8 ? launch_dim<D, kFP8>(c, a, p, st) : launch_dim<D, kBF16>(c, a, p, st);
}

}  // namespace

size_t attend_ws_bytes(const Cache& c, int32_t heads, int32_t k) {
  const Plan p = plan(c, heads, k);
  if (p.splits == 1) return 0;
  const size_t parts = static_cast<size_t>(c.rows) * heads * p.splits;
  return align_up(parts * sizeof(float2)) + parts * c.dv * sizeof(float);
}

hipError_t launch_attend(const Cache& c, int32_t heads, int32_t k, float scale, const void* q,
                         const void* k_pages, const float* k_scale, const void* v_pages,
                         const float* v_scale, const int32_t* table, const int32_t* lengths,
                         const int32_t* idx, void* out, float* lse, void* ws, hipStream_t st) {
  const Plan p = plan(c, heads, k);
  Args a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k_pages = static_cast<const uint8_t*>(k_pages);
  a.k_scale = k_scale;
  a.v_pages = static_cast<const uint8_t*>(v_pages);
  a.v_scale = v_scale;
  a.table = table;
  a.lengths = lengths;
  a.idx = idx;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  const size_t parts = static_cast<size_t>(c.rows) * heads * p.splits;
  a.part_ml = static_cast<float2*>(ws);
  a.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + align_up(parts * sizeof(float2)));
  a.rows = c.rows;
  a.heads = heads;
  a.share = heads / c.kv_heads;
  a.k = k;
  a.splits = p.splits;
  a.row_pages = c.row_pages;
  a.pages = c.pages;
  a.kv_heads = c.kv_heads;
  a.scale2 = scale * kLog2e;
  a.div = make_div(c.P);
  if (c.latent()) return launch_latent(c, a, p, st);
  switch (c.dk) {
    case 64: return launch_type<64>(c, a, p, st);
    case 128: return launch_type<128>(c, a, p, st);
    default: return launch_type<256>(c, a, p, st);
  }
}

}  // namespace misa
