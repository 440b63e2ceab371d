// Attention of one new token per row over a paged cache (misa_attend in
// misa.h): every cached token of the row, or those of an index list.
#include <algorithm>

#include "attend.hpp"

namespace misa {

namespace {

// A vector of N dwords, aligned to its size.
template <bool ONCE, int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* to) {
  typedef __attribute__((ext_vector_type(N))) uint32_t V;
  const V* q = reinterpret_cast<const V*>(p);
  const V x = ONCE ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
  for (int i = 0; i < N; ++i) to[i] = x[i];
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

// One workgroup of four waves per (split, kv head and chunk of 16 * RT query
// heads, row); a wave takes every fourth tile of 32 tokens.  All products are
// transposed, so that a lane keeps one query head (l % 16):
//   S^T = K Q^T   16x16x32 bf16, rows = tokens, columns = heads,
//   O^T = V^T P^T with P^T read from S^T's registers as they are: lane group g
//         holds the tokens 4g .. 4g+3 of both 16-token halves, and V's rows
//         are loaded in that order.  Eight rows of V make eight columns of V^T
//         by byte permutes in registers.
// A weight goes into the product as two bf16 parts (2^-16 together), or the result
// would be off by a second bf16 rounding; the cached values are exact in bf16.
// Neither part of a positive weight is zero or negative, so that an infinite value
// stays an infinity of its sign: the first is the weight's predecessor cut off,
// the second the rest.  Maximum, sums and O stay in fp32 registers.
// No tile goes through LDS: a cached row has few query heads, each of its bytes
// one reader, and the next tile's loads are under way while one is worked on.
//
// Bound by memory: 8 rows of up to 131072 fp8 tokens of 8 heads of 128 (1.73 GB)
// 292 to 309 us on several boxes, 5.6 to 5.9 TB/s; 32 rows x 2048 listed bf16 tokens
// (261 MB, pieces of 256 bytes) 51 us, 5.1 TB/s.  One row of 2000 tokens (8 MB) 6.2
// us: a launch, three dependent loads to a slot, one tile's loads and the join of
// the waves' sums.
//
// ONCE: the cache is read once (one chunk of query heads) and is large, so its
// loads are marked as not to be kept (the 8 rows above: 298 us, 322 with plain loads;
// with two chunks that share a row through L2 it is the other way round, 564 us
// against 505 us).
template <int D, int DT, int RT, bool ONCE>
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
  const int chunks = (a.share + 16 * RT - 1) / (16 * RT);
  int unit, chunk;
  unit_chunk(chunks, unit, chunk);
  const int split = unit % a.splits;
  const int kvh = unit / a.splits % a.kv_heads, row = unit / a.splits / a.kv_heads;
  if (row >= a.rows) return;
  const int head0 = kvh * a.share + chunk * 16 * RT;       // first query head
  const int nheads = min(16 * RT, a.share - chunk * 16 * RT);
  int32_t len;
  const int32_t todo = tokens_of(a, row, len);
  const int32_t per = tiles_per_split(a, todo) * kTileTokens;
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
      for (int u = 0; u < KL; ++u) {
        uint32_t w[4];
        load_words<ONCE, 4>(p + u * 64, w);
        kreg[h][u] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  };
  auto load_v = [&](int tile) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t s = sh.st.slot[tile * 32 + (i / 4) * 16 + 4 * g + i % 4];
      const uint8_t* p = a.v_pages + static_cast<uint64_t>(s == kHidden ? 0 : s) * ROW;
      if constexpr (VB < 16) {
        load_words<ONCE, VW>(p + c * VB, vreg[i]);
      } else {
#pragma unroll
        for (int u = 0; u < VB / 16; ++u) load_words<ONCE, 4>(p + u * 256 + c * 16, vreg[i] + 4 * u);
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
          const uint32_t hi = __builtin_elementwise_sub_sat(__float_as_uint(w), 1u) & 0xFFFF0000u;
          ph[r][i] = __builtin_bit_cast(__bf16, static_cast<uint16_t>(hi >> 16));
          pl[r][i] = static_cast<__bf16>(w - __uint_as_float(hi));
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

// Tiles that a workgroup works on at a time: a wave's each, or a token group's; a
// split has at least those.
int32_t tiles_at_once(const Cache& c) { return c.latent() ? 2 : 4; }

// Query heads of a workgroup: a matrix tile of 16, or two where a kv head has
// more and the registers hold them (8 rows of 8000 bf16 tokens of 8 heads of 128,
// 256 query heads: 49.7 us with 32, 58.2 with 16; heads of 64 31.3 and 30.3, fp8
// 24.8 and 25.8).
int group_heads(const Cache& c, int32_t share) {
  if (c.latent()) return kLatentHeads;
  return share > 16 && c.dk <= 128 ? 32 : 16;
}

// Workgroups that a CU holds at a time, by the kernels' registers.
int resident(const Cache& c, int32_t share) {
  const int one = c.dk == 64 ? 4 : c.dk == 128 ? 3 : 2;
  return group_heads(c, share) == 32 ? one - 1 : one;
}

constexpr int kCus = 256;
constexpr int kMaxSplits = 128;

// Splits of a latent row.  A workgroup (one per CU) takes 2.8 us for a pair of
// tiles; a join costs about 6 us and, for each split, the way of its sums to
// memory and back, 4 KB a head at 5.1 TB/s.  24 rows of 128 heads: 384 listed
// tokens 23.7 us whole, 25.0 us in two splits; 4096 171, 102, 75, 63, 78 and 89 us
// in 1, 2, 3, 4, 8 and 16.  With sixteen rounds of workgroups and more, a split
// could save at most a part of the last one.  An fp8 pair takes a tenth more; in
// seven cases of it, 1 to 200 rows, the choice is at most 7% from the best count.
int32_t latent_splits(int64_t groups, int64_t tokens, int64_t heads, int64_t limit) {
  if (groups >= 16 * kCus) return 1;
  int32_t best = 1;
  double least = 0;
  for (int32_t s = 1; s <= limit; ++s) {
    const int64_t pairs = (tokens + s * 64 - 1) / (s * 64), rounds = (groups * s + kCus - 1) / kCus;
    const double us = 2.8 * pairs * rounds + (s > 1 ? 6.0 + s * heads * (4096 / 5.1e6) : 0.0);
    if (s == 1 || us < least) {
      best = s;
      least = us;
    }
  }
  return best;
}

// Splits of a dense row: at most those that fill the card in one round, since more
// only add to the join and to the last round's tail (8 rows of up to 131072 fp8
// tokens: 768 workgroups 322 us, 1024 340 us, 512 342 us; all with plain loads), and
// fewer where their join costs more than the steps that it saves.  A wave's step,
// one tile of K and of V, takes 0.55 us and for each workgroup on its CU the four
// waves' share of memory and instructions; a join 5.8 us and the sums' way through
// memory.  Fitted to 730 cases with caches from memory, of which the choice is 4%
// from the best one, as many splits as fill the card 9%: 32 rows of 600 tokens, 64
// heads on 8, 16.0 us whole, 21.4 us in three; 16 rows of 1000 with 256 heads 21.4
// and 24.1 us; one row of 2000, 64 heads on 8, 9.7 us in sixteen, 24.8 us whole.
// Groups beyond half of one round stay whole: 8 fp8 heads, rows of 32768 tokens, 48
// rows in two splits 539 us, 49 rows whole 632 us.
int32_t dense_splits(const Cache& c, int32_t heads, int32_t share, int64_t groups, int64_t tokens,
                     int64_t limit) {
  const int32_t held = resident(c, share);
  const int64_t most = std::min<int64_t>(kCus * held / groups, limit);
  const int32_t all = static_cast<int32_t>((tokens + kTileTokens - 1) / kTileTokens);
  const int32_t tile_bytes = kTileTokens * (c.dk + c.dv) * (c.dtype == kFP8 ? 1 : 2);
  const double each = tile_bytes * 8.5e-5 + group_heads(c, share) * c.dk * 1e-4;
  const double sums = 3.3e-6 * c.rows * heads * c.dk;
  int32_t best = 1;
  double least = 0;
  for (int32_t s = static_cast<int32_t>(most); s >= 1; s = s > 1 ? std::max(1, s * 3 / 4) : 0) {
    const int32_t per = ((all + s - 1) / s + 3) & ~3, parts = (all + per - 1) / per;
    const int32_t on_cu = static_cast<int32_t>((groups * parts + kCus - 1) / kCus);
    const double us = per / 4 * (0.55 + on_cu * each) + (parts > 1 ? 5.8 + parts * sums : 0.0);
    if (least == 0 || us < least) {
      best = parts;
      least = us;
    }
  }
  return best;
}

struct Plan {
  int32_t chunks, splits;
  bool once;
};

// Below this much to read, a cache may still be on the chip from the call
// before: one row of 2000 bf16 tokens (8 MB) 9.0 us, and 9.7 us with loads that
// are not kept.
constexpr int64_t kOnceBytes = int64_t{64} << 20;

Plan plan(const Cache& c, int32_t heads, int32_t k) {
  const int32_t share = heads / c.kv_heads;
  const int32_t per = group_heads(c, share);
  Plan p;
  p.chunks = (share + per - 1) / per;
  const int64_t groups = static_cast<int64_t>(c.rows) * c.kv_heads * p.chunks;
  const int64_t most = k > 0 ? k : static_cast<int64_t>(c.row_pages) * c.P;
  const int64_t least = tiles_at_once(c) * kTileTokens;
  const int64_t limit = std::min<int64_t>((most + least - 1) / least, kMaxSplits);
  if (c.latent()) {
    p.splits = latent_splits(groups, most, static_cast<int64_t>(c.rows) * heads, limit);
  } else {
    p.splits = dense_splits(c, heads, share, groups, most, limit);
  }
  const int64_t row_bytes = static_cast<int64_t>(c.dk + c.dv) * (c.dtype == kFP8 ? 1 : 2);
  p.once = p.chunks == 1 && c.rows * most * c.kv_heads * row_bytes >= kOnceBytes;
  return p;
}

uint32_t grid_size(const Cache& c, const Plan& p) {
  const int64_t units = static_cast<int64_t>(c.rows) * c.kv_heads * p.splits;
  return static_cast<uint32_t>((units + 7) / 8 * 8 * p.chunks);
}

template <int D, int DT, int RT>
void launch_rows(const Cache& c, const Args& a, const Plan& p, hipStream_t st) {
  if (p.once)
    attend_kernel<D, DT, RT, true><<<grid_size(c, p), 256, 0, st>>>(a);
  else
    attend_kernel<D, DT, RT, false><<<grid_size(c, p), 256, 0, st>>>(a);
}

template <int D, int DT>
hipError_t launch_dim(const Cache& c, const Args& a, const Plan& p, hipStream_t st) {
  if constexpr (D <= 128) {
    if (group_heads(c, a.share) == 32)
      launch_rows<D, DT, 2>(c, a, p, st);
    else
      launch_rows<D, DT, 1>(c, a, p, st);
  } else {
    launch_rows<D, DT, 1>(c, a, p, st);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  attend_join_kernel<D><<<dim3(a.heads, c.rows), 256, 0, st>>>(a);
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
  a.tiles = tiles_at_once(c);
  a.row_pages = c.row_pages;
  a.pages = c.pages;
  a.kv_heads = c.kv_heads;
  a.scale2 = scale * kLog2e;
  a.div = make_div(c.P);
  if (c.latent()) return launch_attend_latent(c.dtype, a, grid_size(c, p), st);
  switch (c.dk) {
    case 64: return launch_type<64>(c, a, p, st);
    case 128: return launch_type<128>(c, a, p, st);
    default: return launch_type<256>(c, a, p, st);
  }
}

}  // namespace misa
