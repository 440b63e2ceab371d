// Attention of several new tokens of a row at a time over the block-scaled cache
// (misa_block_attend in misa.h): drafts and chunks of prompts.
#include <algorithm>
#include <cmath>

#include "attend.hpp"
#include "quant.hpp"

namespace misa {

namespace {

typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;

constexpr int kThreads = 256;
// Rows (queries times the query heads of a kv head) of a workgroup whose waves have RW
// times 32 of them.
constexpr int row_shift(int RW) { return RW == 4 ? 7 : 6; }
constexpr float kLift = 7.f;  // weights go up to 2^(kSlack + kLift) < 65504, f16's largest
constexpr float kNoGroup = -1e9f;  // the exponent of a group without a page
constexpr float kFar = 60.f, kNear = 8.f;
constexpr int kGroups = 64;  // groups of 16 tokens that are looked up at a time

struct TileArgs {
  const uint16_t* q;
  const uint8_t *k_pages, *v_pages;
  const float *k_scale, *v_scale;
  const int32_t* table;
  const int32_t* lengths;
  Packed rows;
  uint16_t* out;
  float* lse;
  float* part_o;    // [kv_heads, slots, part_rows, d] sums of a part of a unit's tokens
  float2* part_ml;  // [kv_heads, slots, part_rows] maximum (log2) and sum; 0: nothing seen
  int2* where;      // [units] a unit's first slot and its number of them
  int32_t slots, full;  // workgroups of a kv head (0: one a unit, by its number), of them for parts (kSlots)
  int32_t part_rows;    // rows that a unit can have
  int32_t heads, share, kv_heads, row_pages, pages, shift;
  uint32_t q_and, q_xor;  // a negative scale turns the queries' signs, a zero one clears them
  float scale2;           // |scale| * log2(e), above zero
  Div page, by_share;
};

// 16 codes -> 16 bf16 (F16: f16) times a power of two, in two chunks, exact.
template <bool F16>
__device__ __forceinline__ void widen(uint4 c, float scale, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t r[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (F16) {
      r[2 * j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[j], scale, false));
      r[2 * j + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[j], scale, true));
    } else {
      r[2 * j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[j], scale, false));
      r[2 * j + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[j], scale, true));
    }
  }
  lo = make_uint4(r[0], r[1], r[2], r[3]);
  hi = make_uint4(r[4], r[5], r[6], r[7]);
}

__device__ __forceinline__ float halves_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// 0xFF for each of four codes that is NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xFFu;
}

__device__ __forceinline__ float halves_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Up to 2^SHIFT of a batch row's (query, query head of a kv head) pairs: a tile's rows.
struct Unit {
  int32_t r, begin, count;  // the batch row, its first packed query, its queries
  int64_t flat0, flats;  // first pair of the unit, pairs of the row (below 2^27)
  int64_t before;        // tokens before the new ones
  int32_t least, most;   // tokens that its first and its last pair see
  __device__ __forceinline__ bool there() const { return flat0 >= 0 && flat0 < flats; }
};

__device__ __forceinline__ int32_t seen_by(const TileArgs& a, int64_t before, int32_t token) {
  const int64_t n = before + token + 1, cap = static_cast<int64_t>(a.row_pages) * a.page.P;  // at most 2^30
  return static_cast<int32_t>(n < 0 ? 0 : n < cap ? n : cap);
}

template <int SHIFT>
__device__ __forceinline__ Unit unit_of(const TileArgs& a, int64_t unit, int32_t r, int32_t begin, int32_t end) {
  Unit u;
  u.r = r;
  u.begin = begin;
  u.count = end - begin;
  u.flat0 = (unit - unit_base(begin, a.share, SHIFT, r, 1)) << SHIFT;
  u.flats = static_cast<int64_t>(max(u.count, 0)) * a.share;
  u.before = static_cast<int64_t>(a.lengths[r]) - u.count;
  if (u.there()) {
    const int32_t last = static_cast<int32_t>(min(u.flat0 + (1 << SHIFT), u.flats)) - 1;
    u.least = seen_by(a, u.before, static_cast<int32_t>(div_page(static_cast<int32_t>(u.flat0), a.by_share)));
    u.most = seen_by(a, u.before, static_cast<int32_t>(div_page(last, a.by_share)));
  }
  return u;
}

constexpr int kMaxUnits = 1024;  // that are shared out
constexpr int kMaxParts = 32;    // of a unit
constexpr int kLeastTokens = 256;  // of a part

// Slot `slot` of a kv head's: units' tiles in parts of at most q, the smallest q that gives
// no more parts than there are slots for them.  Each workgroup finds it out for
// itself: with as many parts for each unit instead, five drafts on 16 rows of 16384 to
// 32768 tokens took 199 us for 189, four 179 for 163 (heads of 256 732 for 660), 32 tokens
// 575 for 530; one prompt of 512 tokens 27.5 for 30.0.
template <int TK, int SHIFT>
__device__ __forceinline__ bool part_of(const TileArgs& a, int32_t units, int32_t slot, int32_t* lds, int64_t& unit,
                                        int32_t& first, int32_t& parts) {
  int32_t *offsets = lds, *tiles = lds + kMaxUnits + 4;  // -1: no such unit
  const int32_t rows = a.rows.rows;                      // <= units
  for (int32_t i = threadIdx.x; i <= rows; i += kThreads) offsets[i] = a.rows.at(i);
  __syncthreads();
  for (int32_t u = threadIdx.x; u < units; u += kThreads) {
    int32_t lo = 0, hi = rows - 1;  // the last row whose units begin at or before u
    while (lo < hi) {
      const int32_t mid = lo + (hi - lo + 1) / 2;
      if (unit_base(offsets[mid], a.share, SHIFT, mid, 1) <= u)
        lo = mid;
      else
        hi = mid - 1;
    }
    const Unit x = unit_of<SHIFT>(a, u, lo, offsets[lo], offsets[lo + 1]);
    tiles[u] = x.there() ? (x.most + TK - 1) / TK : -1;
  }
  __syncthreads();
  const int lane = lane_id();
  float active = 0.f, sum = 0.f, top = 0.f;
  for (int32_t u = lane; u < units; u += kWave) {
    // Up to 2^25; beyond 2^24 fp32 holds even numbers alone, and none may be counted short.
    const int32_t whole = tiles[u];
    const float n = static_cast<float>(whole > 1 << 24 ? whole + (whole & 1) : whole);
    active += n >= 0.f;
    sum += fmaxf(n, 0.f);
    top = fmaxf(top, n);
  }
  active = lanes_reduce<kWave, false>(active);
  sum = lanes_reduce<kWave, false>(sum);
  top = lanes_reduce<kWave, true>(top);
  const float budget = fminf(a.slots, fmaxf(a.full, active));
  const auto parts_with = [&](int32_t n, int32_t q) {
    return n < 0 ? 0u : max(1u, static_cast<uint32_t>(n + q - 1) / static_cast<uint32_t>(q));
  };
  const int32_t least = max(kLeastTokens / TK, (static_cast<int32_t>(top) + kMaxParts - 1) / kMaxParts);
  int32_t lo = max(least, static_cast<int32_t>(sum * 0.999f / budget));
  // ceil(n / q) < n / q + 1: parts of this size fit; and so do whole units.
  int32_t hi = static_cast<int32_t>(top);
  if (budget > active) hi = static_cast<int32_t>(fminf(top, sum * 1.001f / (budget - active) + 1.f));
  hi = max(hi, lo);
  while (lo < hi) {
    const int32_t q = lo + (hi - lo) / 2;
    float n = 0.f;  // exact where it fits
    for (int32_t u = lane; u < units; u += kWave) n += static_cast<float>(parts_with(tiles[u], q));
    if (lanes_reduce<kWave, false>(n) <= budget)
      hi = q;
    else
      lo = q + 1;
  }
  int32_t before = 0;
  for (int32_t u0 = 0; u0 < units; u0 += kWave) {
    const int32_t mine = u0 + lane < units ? static_cast<int32_t>(parts_with(tiles[u0 + lane], lo)) : 0;
    int32_t end = mine;  // and of the lanes before
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
      const int32_t other = __shfl_up(end, d);
      if (lane >= d) end += other;
    }
    const uint64_t has = __ballot(before + end - mine <= slot && slot < before + end);
    if (has) {
      const int at = __builtin_ctzll(has);
      unit = __builtin_amdgcn_readfirstlane(u0 + at);
      first = __builtin_amdgcn_readlane(before + end - mine, at);
      parts = __builtin_amdgcn_readlane(mine, at);
      return true;
    }
    before += __builtin_amdgcn_readlane(end, kWave - 1);
  }
  return false;
}

// One workgroup of four waves per (tile of 128 rows, part of their tokens, kv head): a wave has 32
// rows, and all share the tiles of TK tokens in LDS, K widened to bf16 and V to f16
// as they are staged, one of two buffers while the other is worked on.
//   S^T = K Q^T, O^T = V^T P^T  (32x32x16), a lane keeps one row (l % 32),
// so that the softmax is within a lane but for its other half, and P^T's operand is
// S^T's registers: of 16 tokens, lane half g holds 4g .. 4g+3 and 8+4g .. 8+4g+3,
// and V's transposing reads give them in that order.  e4m3 codes are exact in both
// types, K's with its scale.
// Weights are f16, in one part of 11 bits, lifted by 2^7 so that what f16 loses is
// 2^-32 of the largest; maximum, sums and O are fp32.  V's scale goes into the weights
// relative to a reference exponent of the row, `eref`, which O's registers are in units of
// and which follows the loudest scale that the row sees in a tile when that leaves its
// neighbourhood.
// NaN values of tokens that some rows do not see yet are left out as zeros, since a
// weight of zero would not hide them, and put in at the end for the rows that see them.
//
// Bound by the matrix unit, LDS and the vector unit taking turns, at clocks that power
// holds back (1.85 to 2.1 of 2.4 GHz): 8192 queries of three rows of up to 32768 tokens,
// 64 heads on 8 of 128 (6.96 TFLOP), 7.5 to 8.2 ms on several cards, 850 to 925 TFLOP/s,
// 70 to 76% of what a large library product reaches; matrix unit busy 44%.  Of it the
// values' products take 2.9 ms, the scores' 2.2, widening the tiles 1.6, the
// exponentials 0.2.  Heads of 64 780 to 810 TFLOP/s, of 256 (one workgroup a CU) 635.
// Tried and not kept: scores on the 8-bit matrix instructions with queries in two
// e4m3 parts (10% less time, but sums of products off by 2^-18, more than fp32's);
// 256 rows a workgroup, in step (9.4 ms) or in two groups that take turns (equal);
// the next tile's scores beside this one's weights (9.2); three waves a SIMD (9.5).
//
// RW = 4: the waves have 32 rows each.  RW = 2: two have 32 rows and half the tokens of
// a tile each, two the same rows and the other half; their sums are joined at the end.
// By memory, then, with two tiles' loads under way: 16 rows of up to 32768 tokens, 64
// heads on 8, five drafts each (789 MB) 189 us, 4.2 TB/s, four 163 us, 4.85 TB/s (five 213
// with one tile's and look-ups between the tiles, whose branches' ends waited for all
// loads, and 198 without; the prompt above 7.87 and 7.73 ms).
template <int D, int TK, int RW>
__global__ __launch_bounds__(kThreads, D <= 128 ? 2 : 1) void attend_tiles_kernel(TileArgs a) {
  constexpr int kRowShift = row_shift(RW), kRows = 1 << kRowShift;
  constexpr int CH = D / 8;              // 16-byte chunks of a widened row
  constexpr int CC = D / 16;             // of a row of codes
  constexpr int NC = TK * CC / kThreads;  // loads of K, and of V, a thread and tile
  constexpr int KS = D / 16, NJ = D / 32;
  constexpr int NG = TK / 16;            // groups of 16 tokens
  constexpr int NH = TK / 32 * RW / 4;   // a wave's halves of 32 tokens
  static_assert(NH > 0, "a wave has 32 tokens of a tile");
  constexpr int GT = kGroups / NG;       // tiles of a stage of groups
  __shared__ __attribute__((aligned(128))) uint4 kt[2][TK * CH];
  __shared__ __attribute__((aligned(128))) uint4 vt[2][TK * CH];
  // Groups of 16 tokens: their slots (kHidden: no page there), K's scales, the exponents of V's.
  __shared__ __attribute__((aligned(16))) uint32_t slots[2 * kGroups];
  __shared__ __attribute__((aligned(16))) float k_unit[2 * kGroups];
  __shared__ __attribute__((aligned(16))) float v_exp[2 * kGroups];
  __shared__ float4 join[RW < 4 ? kRows : 1];
  __shared__ int any_nan;  // in V's codes of tiles with tokens that some rows do not see

  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 31, g = lane >> 5;
  const int wave_rows = 32 * (wave % RW), h0 = wave / RW * NH;  // first row, first half of the tokens
  const int kvh = blockIdx.x % a.kv_heads;
  const int64_t units = unit_base(a.rows.n, a.share, kRowShift, a.rows.rows, 1);
  const int32_t slot = blockIdx.x / a.kv_heads;
  int64_t unit = units - 1 - slot;  // the longest rows of a prompt first
  int32_t first = slot, parts = 1;
  if (a.slots) {
    static_assert(sizeof(kt) >= (2 * kMaxUnits + 4) * sizeof(int32_t), "rows' offsets and units' tiles");
    if (!part_of<TK, kRowShift>(a, static_cast<int32_t>(units), slot, reinterpret_cast<int32_t*>(kt), unit, first, parts))
      return;
    if (kvh == 0 && slot == first && threadIdx.x == 0) a.where[unit] = make_int2(first, parts);
  }
  const int32_t r = last_row(a.rows.rows, unit,
                             [&](int32_t x) { return unit_base(a.rows.at(x), a.share, kRowShift, x, 1); });
  const Unit u = unit_of<kRowShift>(a, unit, r, a.rows.at(r), a.rows.at(r + 1));
  if (!u.there()) return;
  const int32_t least = u.least, most = u.most;
  const auto token_of = [&](int32_t flat) { return static_cast<int32_t>(div_page(flat, a.by_share)); };
  const int32_t last = static_cast<int32_t>(min(u.flat0 + kRows, u.flats)) - 1;
  const int32_t flat = static_cast<int32_t>(u.flat0) + wave_rows + c;
  const bool mine = flat <= last;
  const int32_t token = token_of(min(flat, last));
  const int32_t seen = seen_by(a, u.before, token);
  const int64_t at = static_cast<int64_t>(u.begin + token) * a.heads + kvh * a.share + (min(flat, last) - token * a.share);
  const auto part_at = [&] { return (static_cast<int64_t>(kvh) * a.slots + slot) * a.part_rows + wave_rows + c; };
  const bool busy = static_cast<int32_t>(u.flat0) + wave_rows <= last;  // the wave has rows

  const int32_t tiles = (most + TK - 1) / TK, per = (tiles + parts - 1) / parts;
  // Scalars, which the compiler does not see through the search above.
  const int32_t t0 = __builtin_amdgcn_readfirstlane((slot - first) * per);
  const int32_t t1 = __builtin_amdgcn_readfirstlane(min(t0 + per, tiles));
  if (t0 >= t1) {
    if (h0 > 0) return;
    if (mine && g == 0) {
      if (parts > 1)
        a.part_ml[part_at()] = make_float2(-INFINITY, 0.f);
      else if (a.lse)
        a.lse[at] = -INFINITY;
    }
    if (mine && parts == 1)
      for (int i = 0; i < D / 16; ++i)
        *reinterpret_cast<uint4*>(a.out + at * D + (2 * i + g) * 8) = make_uint4(0, 0, 0, 0);
    return;
  }

  bf16x8 qf[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    uint4 x = *reinterpret_cast<const uint4*>(a.q + at * D + 16 * s + 8 * g);
    x.x = (x.x & a.q_and) ^ a.q_xor;
    x.y = (x.y & a.q_and) ^ a.q_xor;
    x.z = (x.z & a.q_and) ^ a.q_xor;
    x.w = (x.w & a.q_and) ^ a.q_xor;
    qf[s] = as_bf16x8(x);
  }

  // Groups of 16 tokens, which are in one page and block, are looked up a stage of 64 at
  // a time, a lane each, and by the waves in turn: where stage s begins, the wave of stage
  // s + 1 puts what it found into LDS and looks its next one's pages up, whose scales it
  // loads two stages later.  No tile's loads wait for these.
  const int32_t* table = a.table + static_cast<int64_t>(r) * a.row_pages;
  int32_t own = wave;  // the wave's stage
  int32_t group_page = -1;
  uint32_t group_slot = kHidden;
  float group_k = 0.f, group_v = 0.f;
  const auto slot_at = [&](int32_t t, int32_t page) {
    const uint32_t in = static_cast<uint32_t>(t) - div_page(t, a.page) * a.page.P;
    return (static_cast<uint32_t>(page) * a.kv_heads + kvh) * a.page.P + in;
  };
  const auto group_token = [&] { return (static_cast<int64_t>(t0) + own * GT) * TK + lane * 16; };
  const auto find_pages = [&] {
    const int64_t t = group_token();
    group_page = -1;
    if (t < min(most, t1 * TK)) group_page = table[div_page(static_cast<int32_t>(t), a.page)];
  };
  const auto find_scales = [&] {
    group_slot = kHidden;
    if (group_page >= 0 && group_page < a.pages) {
      group_slot = slot_at(static_cast<int32_t>(group_token()), group_page);
      group_k = a.k_scale[group_slot >> a.shift];
      group_v = a.v_scale[group_slot >> a.shift];
    }
  };
  const auto keep_groups = [&] {
    const int at = (own & 1) * kGroups + lane;
    slots[at] = group_slot;
    k_unit[at] = group_k;
    v_exp[at] = group_slot == kHidden ? kNoGroup : static_cast<float>(static_cast<int>(__float_as_uint(group_v) >> 23) - 127);
    own += kThreads / kWave;
    find_pages();
  };
  static_assert(kGroups == kWave && kThreads == 4 * kWave, "a lane each, of four waves");

  // Thread i has chunk i % CC of tokens i / CC, + kThreads / CC, ...
  // Swizzles of the chunks, so that 16 rows' reads of a chunk (K) and four rows' of
  // 64 bytes (V) are in different banks, and so are eight threads' writes of every
  // other chunk of a row (a quarter of all LDS cycles were conflicts of those).
  const auto spread = [](int row, int chunk) { return D == 64 ? row & 1 : chunk >> 3 & 1; };
  const auto k_at = [&](int row, int chunk) {
    return row * CH + (chunk ^ (D == 64 ? row >> 1 & 7 : row & 15) ^ spread(row, chunk));
  };
  const auto v_at = [&](int row, int chunk) {
    return row * CH + (chunk ^ (D == 64 ? (row >> 1 & 1) << 2 : (row & 3) << 2) ^ spread(row, chunk));
  };
  const int my_token = threadIdx.x / CC, my_chunk = threadIdx.x % CC;
  // Rows i of a thread are a multiple of 16 apart (or it has one): one address
  // within a group.
  const uint8_t* k_from = a.k_pages + (my_token % 16) * D + my_chunk * 16;
  const uint8_t* v_from = a.v_pages + (my_token % 16) * D + my_chunk * 16;
  struct Codes {  // a thread's part of a tile
    uint4 k[NC], v[NC];
    float unit[NC];
    bool there[NC];  // V's tokens
  };
  const auto load_k = [&](int32_t tile, Codes& x) __attribute__((always_inline)) {
    const int32_t first = ((tile - t0) & (2 * GT - 1)) * NG + my_token / 16;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const uint32_t s = slots[first + i * (kThreads / CC) / 16];
      x.unit[i] = k_unit[first + i * (kThreads / CC) / 16];
      const uint64_t off = static_cast<uint64_t>(s != kHidden ? s : 0) * D;  // some page: what it holds is not used
      x.k[i] = *reinterpret_cast<const uint4*>(k_from + off);
    }
  };
  const auto load_v = [&](int32_t tile, Codes& x) __attribute__((always_inline)) {
    const int32_t first = ((tile - t0) & (2 * GT - 1)) * NG + my_token / 16;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const uint32_t s = slots[first + i * (kThreads / CC) / 16];
      x.there[i] = s != kHidden;
      const uint64_t off = static_cast<uint64_t>(x.there[i] ? s : 0) * D;
      x.v[i] = *reinterpret_cast<const uint4*>(v_from + off);
    }
  };
  const auto widen_k = [&](int b, const Codes& x) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int row = my_token + i * (kThreads / CC);
      uint4 lo, hi;
      widen<false>(x.k[i], x.unit[i], lo, hi);
      kt[b][k_at(row, 2 * my_chunk)] = lo;
      kt[b][k_at(row, 2 * my_chunk + 1)] = hi;
    }
  };
  const auto widen_v = [&](int32_t tile, int b, Codes& x) __attribute__((always_inline)) {
    // A NaN must not meet a weight of zero: tokens that no row sees are zeros, and where
    // some rows do not see some token, NaN codes are.
    const bool edge = (tile + 1) * TK > least;
    bool whole = !edge;
#pragma unroll
    for (int i = 0; i < NC; ++i) whole = whole && !__any(!x.there[i]);
    if (!whole) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const bool seen = x.there[i] && tile * TK + my_token + i * (kThreads / CC) < most;
        uint32_t* w = reinterpret_cast<uint32_t*>(&x.v[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t bad = seen && edge ? nan_bytes(w[j]) : 0u;
          if (bad) any_nan = 1;
          w[j] = seen ? w[j] & ~bad : 0u;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int row = my_token + i * (kThreads / CC);
      uint4 lo, hi;
      widen<true>(x.v[i], 1.f, lo, hi);
      vt[b][v_at(row, 2 * my_chunk)] = lo;
      vt[b][v_at(row, 2 * my_chunk + 1)] = hi;
    }
  };

  f32x16 acc[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[j][e] = 0.f;
  float m = -INFINITY, l = 0.f;  // of this lane's row, and of its half of the tokens
  float eref = kNoGroup, loudest = kNoGroup;  // whole numbers, of what this lane's row sees
  const int vrow = 4 * g + (lane & 15) / 4, vcol = 2 * (lane >> 4 & 1) + (lane & 3) / 2;  // transposing reads

  const auto score = [&](int b, f32x16 (&st)[NH]) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int e = 0; e < 16; ++e) st[h][e] = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int h = 0; h < NH; ++h)
        st[h] = mfma32_bf16(as_bf16x8(kt[b][k_at(32 * (h0 + h) + c, 2 * s + g)]), qf[s], st[h]);
  };
  // The exponents of a tile's groups, alike in all lanes but in vector registers: as scalars they
  // would cost the way there and its waits (a third of the weights' time).
  const auto exponents = [&](int32_t tile, float (&ve)[2 * NH]) __attribute__((always_inline)) {
    const int32_t first = ((tile - t0) & (2 * GT - 1)) * NG + 2 * h0;
#pragma unroll
    for (int i = 0; i < 2 * NH; ++i) ve[i] = v_exp[first + i];
  };
  // Weights of a tile from its scores.
  const auto weigh = [&](int32_t tile, float (&ve)[2 * NH], f32x16 (&st)[NH], f16x8 (&w)[2 * NH]) __attribute__((always_inline)) {
    float still = ve[0];
#pragma unroll
    for (int i = 1; i < 2 * NH; ++i) still = fminf(still, ve[i]);
    if ((tile + 1) * TK > least || __any(still == kNoGroup)) {  // some row does not see some token
      __builtin_amdgcn_sched_barrier(0);  // a branch, not 32 selects in every tile
      // A block behind what a row sees has no part in that row's reference, however loud.
#pragma unroll
      for (int i = 0; i < 2 * NH; ++i) ve[i] = tile * TK + 32 * h0 + 16 * i < seen ? ve[i] : kNoGroup;
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          st[h][e] = tile * TK + 32 * (h0 + h) + 8 * (e / 4) + 4 * g + e % 4 < seen && ve[2 * h + e / 8] != kNoGroup
                         ? st[h][e] : -INFINITY;
    }
    float loud = ve[0];
#pragma unroll
    for (int i = 1; i < 2 * NH; ++i) loud = fmaxf(loud, ve[i]);
    float high = -INFINITY;
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int e = 0; e < 16; ++e) high = fmaxf(high, st[h][e]);
    high *= a.scale2;
    // A new reference maximum or exponent: O's registers follow.
    if (__any(high > m + kSlack || loud > eref || (loud < eref - kNear && loud != kNoGroup))) {
      const float next = fmaxf(m, halves_max(high));
      float f = next == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - next);
      m = next;
      l *= f;
      if (loud != kNoGroup) {
        loudest = fmaxf(loudest, loud);
        const float unit = loud <= eref && loud >= eref - kNear ? eref : fmaxf(loud, loudest - kFar);
        f = __builtin_amdgcn_ldexpf(f, static_cast<int>(fmaxf(eref - unit, -200.f)));
        eref = unit;
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[j] *= f;
    }
    const float mb = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < 2 * NH; ++i) {
      // Far below the reference a block's values no longer count, but its weights do.
      const float lift = kLift + fmaxf(ve[i] - eref, -100.f), base = lift - mb;
      float sum = 0.f;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(st[i / 2][i % 2 * 8 + x], a.scale2, base));
        sum += p;
        w[i][x] = static_cast<_Float16>(p);
      }
      l += __builtin_amdgcn_ldexpf(sum, static_cast<int>(-lift));
    }
  };
  const auto add_values = [&](int b, const f16x8 (&w)[2 * NH]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2 * NH; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const auto part = [&](int row) {
          const uint8_t* p = reinterpret_cast<const uint8_t*>(&vt[b][v_at(row, 4 * j + vcol)]) + (lane & 1) * 8;
          return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
        };
        const s16x4 y0 = part(16 * (2 * h0 + i) + vrow), y1 = part(16 * (2 * h0 + i) + 8 + vrow);
        const f16x8 v = __builtin_bit_cast(f16x8, __builtin_shufflevector(y0, y1, 0, 1, 2, 3, 4, 5, 6, 7));
        acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, w[i], acc[j], 0, 0, 0);
      }
  };
  if (threadIdx.x == 0) any_nan = 0;
  find_pages();
  find_scales();
  if (own < 2) keep_groups();
  __syncthreads();
  constexpr int AHEAD = RW < 4 ? 2 : 1;  // tiles whose loads are under way
  Codes codes[AHEAD];
  load_k(t0, codes[0]);
  load_v(t0, codes[0]);
  if constexpr (AHEAD > 1) {
    load_k(min(t0 + 1, t1 - 1), codes[1]);
    load_v(min(t0 + 1, t1 - 1), codes[1]);
  }
  widen_k(0, codes[0]);
  widen_v(t0, 0, codes[0]);
  __syncthreads();
  // Tile `tile`, number n of the split's; loads of tile + AHEAD to `to`, the next tile's are in `next`.
  const auto step = [&](int32_t tile, int n, Codes& to, Codes& next) __attribute__((always_inline)) {
    load_k(min(tile + AHEAD, t1 - 1), to);  // no branch: the compiler would wait where it ends
    load_v(min(tile + AHEAD, t1 - 1), to);
    if (busy) {
      f32x16 st[NH];
      f16x8 w[2 * NH];
      float ve[2 * NH];
      exponents(tile, ve);
      score(n & 1, st);
      weigh(tile, ve, st, w);
      add_values(n & 1, w);
    }
    if (tile + 1 < t1) {
      widen_k(n + 1 & 1, next);
      widen_v(tile + 1, n + 1 & 1, next);
    }
    __syncthreads();
  };
  int32_t tile = t0;
  for (int32_t stage = 0; tile < t1; ++stage) {
    if (own == stage + 1) keep_groups();
    if (own == stage + 3) find_scales();
    const int32_t end = min(tile + GT, t1);
    if constexpr (AHEAD == 1) {
      for (; tile < end; ++tile) step(tile, tile - t0, codes[0], codes[0]);
    } else {
      for (; tile + 1 < end; tile += 2) {
        step(tile, 0, codes[0], codes[1]);
        step(tile + 1, 1, codes[1], codes[0]);
      }
      if (tile < end) {  // the split's last
        step(tile, 0, codes[0], codes[1]);
        ++tile;
      }
    }
  }

  l = halves_sum(l);
  __syncthreads();
  if constexpr (RW < 4) {  // the second half's sums to the first, through K's buffers
    static_assert(sizeof(kt) >= sizeof(float) * D / 2 * kRows * 2, "two waves' O");
    float* to = reinterpret_cast<float*>(kt) + wave_rows * 2 + lane;
    if (h0 > 0) {
      if (g == 0) join[wave_rows + c] = make_float4(m, l, eref, 0.f);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) to[(16 * j + e) * (2 * kRows)] = acc[j][e];
    }
    __syncthreads();
    if (h0 > 0) return;
    const float4 x = join[wave_rows + c];
    const float both = fmaxf(m, x.x), unit = fmaxf(eref, x.z);
    const float f0 = part_factor(m, l, both), f1 = part_factor(x.x, x.y, both);
    const float s0 = __builtin_amdgcn_ldexpf(f0, static_cast<int>(fmaxf(eref - unit, -200.f)));
    const float s1 = __builtin_amdgcn_ldexpf(f1, static_cast<int>(fmaxf(x.z - unit, -200.f)));
    m = both;
    l = l * f0 + x.y * f1;
    eref = unit;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[j][e] = acc[j][e] * s0 + to[(16 * j + e) * (2 * kRows)] * s1;
  }
  if (!mine) return;
  if (any_nan) {  // the NaN values left out above, for the rows that see them
    for (int32_t s = max(t0 * TK, least / TK * TK); s < min(t1 * TK, seen); ++s) {
      const int32_t page = table[div_page(s, a.page)];
      if (page < 0 || page >= a.pages) continue;
      const uint8_t* v = a.v_pages + static_cast<uint64_t>(slot_at(s, page)) * D + 4 * g;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t bad = nan_bytes(*reinterpret_cast<const uint32_t*>(v + 32 * j + 8 * e));
#pragma unroll
          for (int x = 0; x < 4; ++x) acc[j][4 * e + x] = bad >> 8 * x & 1 ? NAN : acc[j][4 * e + x];
        }
    }
  }
  const float unit_o = __builtin_amdgcn_ldexpf(1.f, static_cast<int>(fmaxf(eref, -200.f) - kLift));
  const int64_t part = parts > 1 ? part_at() : 0;
  if (g == 0) {
    if (parts > 1)
      a.part_ml[part] = make_float2(m, l);
    else if (a.lse)
      a.lse[at] = l == 0.f ? -INFINITY : final_lse(m, l);
  }
  const float f = parts > 1 ? unit_o : l == 0.f ? 0.f : unit_o / l;
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = 32 * j + 8 * e + 4 * g;
      const float4 o = make_float4(acc[j][4 * e] * f, acc[j][4 * e + 1] * f, acc[j][4 * e + 2] * f, acc[j][4 * e + 3] * f);
      if (parts > 1) {
        *reinterpret_cast<float4*>(a.part_o + part * D + d) = o;
      } else {
        bf16x2 x, y;
        x[0] = static_cast<__bf16>(o.x);
        x[1] = static_cast<__bf16>(o.y);
        y[0] = static_cast<__bf16>(o.z);
        y[1] = static_cast<__bf16>(o.w);
        *reinterpret_cast<uint2*>(a.out + at * D + d) =
            make_uint2(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y));
      }
    }
}

// The parts of a query's heads joined: D / 4 threads a head, 1024 / D heads a
// workgroup, eight parts' loads at a time.  75 queries of 64 heads of 128 in three to five
// parts 5.9 us, four dependent loads; part after part 9.0.
template <int D, int RW>
__global__ __launch_bounds__(256) void join_tiles_kernel(TileArgs a) {
  constexpr int T = D / 4;
  const int32_t i = blockIdx.x;
  int32_t r, begin, end;
  if (!row_of_entry(a.rows, i, r, begin, end)) return;
  const int head = blockIdx.y * (256 / T) + threadIdx.x / T, d = threadIdx.x % T * 4;
  if (head >= a.heads) return;
  const int64_t at = static_cast<int64_t>(i) * a.heads + head;
  const int32_t kvh = head / a.share;
  const int64_t flat = static_cast<int64_t>(i - begin) * a.share + (head - kvh * a.share);
  int2 w = a.where[unit_base(begin, a.share, row_shift(RW), r, 1) + (flat >> row_shift(RW))];
  if (w.y == 1) return;  // written already
  w.y = min(max(w.y, 1), kMaxParts);  // whatever offsets that do not ascend left there
  w.x = min(max(w.x, 0), a.slots - w.y);
  if (w.x < 0) return;
  const int64_t part = (static_cast<int64_t>(kvh) * a.slots + w.x) * a.part_rows + (flat & ((1 << row_shift(RW)) - 1));
  constexpr int R = 8;  // parts whose loads are under way together
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < w.y; s0 += R) {
    float2 x[R];
    float4 y[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t from = part + static_cast<int64_t>(min(s0 + j, w.y - 1)) * a.part_rows;
      x[j] = a.part_ml[from];
      y[j] = *reinterpret_cast<const float4*>(a.part_o + from * D + d);  // used if the part saw something
    }
    float next = m;
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (s0 + j < w.y) next = fmaxf(next, x[j].x);
    const float before = part_factor(m, l, next);
    m = next;
    l *= before;
    o.x *= before;
    o.y *= before;
    o.z *= before;
    o.w *= before;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (s0 + j >= w.y || x[j].y == 0.f) continue;  // nothing seen, nothing written
      const float f = part_factor(x[j].x, x[j].y, m);
      l += x[j].y * f;
      o.x += y[j].x * f;
      o.y += y[j].y * f;
      o.z += y[j].z * f;
      o.w += y[j].w * f;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (d == 0 && a.lse) a.lse[at] = l == 0.f ? -INFINITY : final_lse(m, l);
  bf16x2 x, y;
  x[0] = static_cast<__bf16>(o.x * inv);
  x[1] = static_cast<__bf16>(o.y * inv);
  y[0] = static_cast<__bf16>(o.z * inv);
  y[1] = static_cast<__bf16>(o.w * inv);
  *reinterpret_cast<uint2*>(a.out + at * D + d) =
      make_uint2(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y));
}

// Workgroups that units are shared out to: those that the card holds at a time, two a CU.
// It holds one of heads of 256, whose parts run in two rounds: with 256 of them four new
// tokens on 20 rows of up to 8192, 64 heads on 8, took 405 us for 234 and on 16 of 32768 767 for
// 655, but on 8 of 2000 37 for 47, and a prompt of 512 40 for 61.
constexpr int kSlots = 512;

// Two waves' rows where no row of the batch has more: 16 rows of 32768 tokens, 64 heads
// on 8 of 128, eight new tokens each (64 pairs of query and head) 198 us, 223 with
// four waves' rows; nine 334 and 252 us.
int row_waves(const Cache& c, const BlockAttend& b) {
  return c.dk <= 128 && static_cast<int64_t>(b.most) * (b.heads / c.kv_heads) <= 64 ? 2 : 4;
}

int64_t tile_units(const Cache& c, const BlockAttend& b) {
  return unit_base(b.n, b.heads / c.kv_heads, row_shift(row_waves(c, b)), c.rows, 1);
}

// Slots of a kv head where units are shared out in parts: if those that rows with up to
// `most` new tokens can have are half of kSlots at most; as many as the card
// holds (kSlots), or one a unit that can have work.  A row's c pairs are floor(c / size) + 1 units
// at most, so that those are a unit more for each query or row, whichever are fewer.
// (With a unit more for each row of the table, as units are numbered, five drafts on 16
// rows had half the parts, 333 us for 215; and four queries of 1024 heads on 64, in a table of
// 1000 rows, a workspace of 2.0 GiB for 16 MiB.)
int32_t tile_slots(const Cache& c, const BlockAttend& b) {
  const int64_t rows = 32 * row_waves(c, b), most = std::max(b.most, 1), units = tile_units(c, b);
  const int64_t whole = ((b.n - 1) / most + 1) * ((most * (b.heads / c.kv_heads) - 1) / rows + 1);
  const int64_t longest = (static_cast<int64_t>(c.row_pages) * c.P + kLeastTokens - 1) / kLeastTokens;
  if (std::min(units, whole) * c.kv_heads > kSlots / 2 || longest < 2 || units > kMaxUnits) return 0;
  const int64_t working = unit_base(b.n, b.heads / c.kv_heads, row_shift(row_waves(c, b)), std::min(c.rows, b.n), 1);
  const int64_t useful = working * std::min<int64_t>(longest, kMaxParts);
  return static_cast<int32_t>(std::max(working, std::min<int64_t>(kSlots / c.kv_heads, useful)));
}

int32_t part_rows(const Cache& c, const BlockAttend& b) {
  return static_cast<int32_t>(std::min<int64_t>(32 * row_waves(c, b), static_cast<int64_t>(b.n) * (b.heads / c.kv_heads)));
}

template <int D, int TK, int RW>
hipError_t launch_tiles_dim(const TileArgs& a, uint32_t grid, hipStream_t st) {
  attend_tiles_kernel<D, TK, RW><<<grid, kThreads, 0, st>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.slots == 0) return e;
  const int per = 1024 / D;
  join_tiles_kernel<D, RW><<<dim3(a.rows.n, (a.heads + per - 1) / per), 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t attend_tiles_ws_bytes(const Cache& c, const BlockAttend& b) {
  const int32_t slots = tile_slots(c, b);
  if (slots == 0) return 0;
  const size_t parts = static_cast<size_t>(slots) * c.kv_heads * part_rows(c, b);
  return align_up(parts * sizeof(float2)) + align_up(parts * c.dv * sizeof(float)) + tile_units(c, b) * sizeof(int2);
}

hipError_t launch_attend_tiles(const Cache& c, const BlockAttend& b, hipStream_t st) {
  TileArgs a{};
  a.q = static_cast<const uint16_t*>(b.q);
  a.k_pages = static_cast<const uint8_t*>(b.k_pages);
  a.v_pages = static_cast<const uint8_t*>(b.v_pages);
  a.k_scale = b.k_scale;
  a.v_scale = b.v_scale;
  a.table = b.table;
  a.lengths = b.lengths;
  a.rows = Packed{b.offsets, c.rows, b.n};
  a.out = static_cast<uint16_t*>(b.out);
  a.lse = b.lse;
  a.heads = b.heads;
  a.share = b.heads / c.kv_heads;
  a.kv_heads = c.kv_heads;
  a.slots = tile_slots(c, b);
  a.full = kSlots / c.kv_heads;
  a.part_rows = part_rows(c, b);
  const size_t parts = static_cast<size_t>(a.slots) * c.kv_heads * a.part_rows;
  uint8_t* ws = static_cast<uint8_t*>(b.ws);
  a.part_ml = reinterpret_cast<float2*>(ws);
  a.part_o = reinterpret_cast<float*>(ws + align_up(parts * sizeof(float2)));
  a.where = reinterpret_cast<int2*>(ws + align_up(parts * sizeof(float2)) + align_up(parts * c.dv * sizeof(float)));
  a.row_pages = c.row_pages;
  a.pages = c.pages;
  a.shift = __builtin_ctz(static_cast<uint32_t>(b.block));
  a.q_and = b.scale == 0.f ? 0u : 0xFFFFFFFFu;
  a.q_xor = b.scale < 0.f ? 0x80008000u : 0u;
  a.scale2 = b.scale == 0.f ? 1.f : std::fabs(b.scale) * kLog2e;
  a.page = make_div(c.P);
  a.by_share = make_div(a.share);
  const uint32_t grid = static_cast<uint32_t>((a.slots ? a.slots : tile_units(c, b)) * c.kv_heads);
  const bool two = row_waves(c, b) == 2;
  switch (c.dk) {
    case 64: return two ? launch_tiles_dim<64, 64, 2>(a, grid, st) : launch_tiles_dim<64, 64, 4>(a, grid, st);
    case 128: return two ? launch_tiles_dim<128, 64, 2>(a, grid, st) : launch_tiles_dim<128, 64, 4>(a, grid, st);
    default: return launch_tiles_dim<256, 32, 4>(a, grid, st);
  }
}

}  // namespace misa
