// Attention over latent caches (misa_attend with dk 576, dv 512): one cached row
// per token serves every query head, and its first 512 elements are the value.
#include "attend.hpp"

namespace misa {

namespace {

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

constexpr int kLatentStage = 512;  // tokens whose slots are in LDS at a time: one per thread

// The end of a workgroup's work, for token group G (both meet in the barriers):
// the groups' sums are joined a quarter of the dimensions at a time; each group
// hands one quarter to the other through LDS and writes the other one.
template <int G, int NJ, int NB>
__device__ __forceinline__ void hand_over(const Args& a, const f32x4 (&acc)[NJ], uint4 (&even)[2][NB],
                                          uint4 (&odd)[2][NB], float (&top)[2][4][16],
                                          float (&sum)[2][4][16], float m, float l, int row, int split,
                                          int head0, int hw, int c, int g) {
  constexpr int kPart = NJ / 4;  // products of a quarter
  static_assert(kPart * 4 * kWave <= 2 * NB, "a quarter fits a buffer");
  const bool mine = head0 + c < a.heads;
  const int64_t at = static_cast<int64_t>(row) * a.heads + head0 + c;
  const int64_t part = at * a.splits + split;
  float4* give = reinterpret_cast<float4*>(G == 0 ? even : odd) + hw * kWave + lane_id();  // [product][wave][lane]
  const float4* take = reinterpret_cast<const float4*>(G == 0 ? odd : even) + hw * kWave + lane_id();
  float f_own = 0.f, f_other = 0.f;
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    if (pass > 0) __syncthreads();
#pragma unroll
    for (int j = 0; j < kPart; ++j) {
      const f32x4 y = acc[(2 * pass + 1 - G) * kPart + j];
      give[j * 4 * kWave] = make_float4(y[0], y[1], y[2], y[3]);
    }
    __syncthreads();
    if (pass == 0) {
      const float m1 = top[1 - G][hw][c], l1 = sum[1 - G][hw][c];
      const float mall = fmaxf(m, m1);
      f_own = part_factor(m, l, mall);
      f_other = part_factor(m1, l1, mall);
      const float lall = l * f_own + l1 * f_other;
      if (G == 0 && g == 0 && mine) {
        if (a.splits > 1)
          a.part_ml[part] = make_float2(mall, lall);
        else if (a.lse)
          a.lse[at] = lall == 0.f ? -INFINITY : final_lse(mall, lall);
      }
      if (a.splits == 1) {
        const float inv = lall == 0.f ? 0.f : 1.f / lall;
        f_own *= inv;
        f_other *= inv;
      }
    }
    if (!mine) continue;
#pragma unroll
    for (int j = 0; j < kPart; ++j) {
      const int d = 16 * ((2 * pass + G) * kPart + j) + 4 * g;
      const f32x4 y = acc[(2 * pass + G) * kPart + j];
      const float4 z = take[j * 4 * kWave];
      const float4 o = make_float4(y[0] * f_own + z.x * f_other, y[1] * f_own + z.y * f_other,
                                   y[2] * f_own + z.z * f_other, y[3] * f_own + z.w * f_other);
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

// One workgroup of eight waves per (split, 64 query heads, row): waves 0-3 and
// 4-7 are two token groups, and wave w of a group has the query heads 16 (w %
// 4) .. +15.  A group's tile of 32 cached rows goes to LDS once, by direct
// loads into one of two buffers while the other is worked on, and its four
// waves read it twice: as K for the scores, and its first 512 elements, by
// transposing reads, as V^T.  The products are those of attend_kernel, but that a
// weight's first part is its rounding (2^-17 together): a cached infinity makes its
// own token's scores infinite or NaN, so that it never meets a weight above zero.
//
// 32 rows of 128 heads over 2048 listed bf16 tokens, in 4 splits: 39 us and the
// join.  Of that a pair of tiles takes 2.77 us (eight of them), for 1.1 us of LDS
// cycles and 1.33 us of matrix cycles: with two waves a SIMD and all but a few of
// their 256 registers taken (O 128, queries 60), six reads are under way, too few
// to hide one behind the other.  The rest is the chain to the first tile (4 us
// for all 256 workgroups' first loads) and 34 MB of sums (3 us).  What it reads,
// 75 MB once from memory, would take 15.5 us.
//
// A tile is nine column blocks of 8 (fp8: 4) chunks of 16 bytes, each [32 rows]
// [chunks]: a direct load fills 64 consecutive chunks, here of 8 (16) rows, from
// whole 128- (64-) byte pieces of them.  Chunk x of row r sits at x ^ swz(r) of
// its block.  What has to be apart (measured: LDS serves a 16-byte read in four
// steps, of the lanes 0-3, 12-15 and 20-27, the rest of 0-31, and the same of
// 32-63, and an 8-byte transposing read in two, of 32 lanes; 256 bytes a step):
//   keys, bf16: 16 rows, with lane group g in rows 0-3, 12-15 and g ^ 1 in 4-11;
//     by t = r / 2, {swz(0, 1, 6, 7)} and {1 ^ swz(2 .. 5)} together are 0 .. 7;
//   values, bf16: 32 bytes of 8 rows: swz / 2 of t = 0 .. 3 (4 .. 7) are 0 .. 3;
//   fp8 by v = r / 4: {swz(0, 3)} and {1 ^ swz(1, 2)} are 0 .. 3, and so are
//     {swz(0, 1, 4, 5)} and {swz(2, 3, 6, 7)}.
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
  __shared__ float top[2][4][16], sum[2][4][16];

  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int hw = wave & 3, grp = wave >> 2;
  const int chunks = (a.heads + kLatentHeads - 1) / kLatentHeads;
  int unit, chunk;
  unit_chunk(chunks, unit, chunk);
  const int row = unit / a.splits, split = unit - row * a.splits;
  if (row >= a.rows) return;
  const int head0 = chunk * kLatentHeads + hw * 16;
  Query own;
  query_of<false>(a, row, own);
  const int32_t len = own.len;
  const int32_t todo = tokens_of(a, own);
  const int32_t per = tiles_per_split(a, todo) * kTileTokens;
  const int32_t t0 = split * per, t1 = min(t0 + per, todo);
  if (t0 >= t1 && split > 0) return;

  bf16x8 qf[KS - QL];
  auto keep_query = [&](int s, uint4 x) {
    if (s < KS - QL)
      qf[s] = as_bf16x8(x);
    else if (grp == 0)
      q_lds[hw][s - (KS - QL)][lane] = x;
  };
  auto query = [&](int s) {
    return s < KS - QL ? qf[s < KS - QL ? s : 0] : as_bf16x8(q_lds[hw][s < KS - QL ? 0 : s - (KS - QL)][lane]);
  };
  f32x4 acc[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;

  auto swz = [](int r) {
    if constexpr (kFp8) {
      const int v = r >> 2;
      return ((v & 1) << 1) ^ ((v >> 1 & 1) * 3) ^ (v >> 2);
    } else {
      const int t = r >> 1;
      return ((t & 3) ^ (t >> 1 & 2)) << 1 | (t >> 2 & 1);
    }
  };
  // The group's four waves load its tile of a pair.  A direct load takes one
  // column block of 8 (fp8: 16) rows; this lane always has the same row, r, and
  // the same chunk of it, so a tile costs it one slot, its address in `src`.
  constexpr int RL = kWave / CB;                  // rows of a load
  const int r = (kFp8 ? hw % 2 : hw) * RL + lane / CB;
  const int block0 = kFp8 ? hw / 2 : 0;           // this wave's column blocks: every other one for fp8
  constexpr int BS = kFp8 ? 2 : 1;
  constexpr int NI = (9 + BS - 1) / BS;           // its loads
  const int lds0 = (kFp8 ? hw % 2 : hw) * kWave;  // first chunk of a load in its block
  auto row_at = [&](int it, const uint8_t*& src) {
    const uint32_t s = slots[(2 * it + grp) * 32 + r];
    src = a.k_pages + static_cast<uint64_t>(s == kHidden ? 0 : s) * (kLatentK * EB) + block0 * (CB * 16) +
          (lane % CB ^ swz(r)) * 16;
    return static_cast<bool>(__any(s == kHidden));
  };
  auto issue = [&](int n, const uint8_t* src, uint4 (&tile)[2][32 * CH]) {
    uint4* buf = tile[grp] + block0 * (32 * CB) + lds0;
    if (n * BS + block0 < 9)
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(src + n * BS * (CB * 16)),
                                       (__attribute__((address_space(3))) void*)(buf + n * BS * (32 * CB)), 16, 0, 0);
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

  // The queries.  Beside a bf16 cache they have the shape of two tiles of 32 rows,
  // one for each group to load, into the buffer that the first pair leaves free;
  // a wave's fragments are those of a key.
  if constexpr (!kFp8) {
    const int h = min(chunk * kLatentHeads + grp * 32 + r, a.heads - 1);
    const uint8_t* src = reinterpret_cast<const uint8_t*>(a.q) +
                         (static_cast<int64_t>(row) * a.heads + h) * (kLatentK * 2) + (lane % CB ^ swz(r)) * 16;
#pragma unroll
    for (int n = 0; n < NI; ++n) issue(n, src, odd);
  } else {
    const int h = min(head0 + c, a.heads - 1);
    const uint16_t* src = a.q + (static_cast<int64_t>(row) * a.heads + h) * kLatentK;
#pragma unroll
    for (int s = 0; s < KS; ++s)
      keep_query(s, *reinterpret_cast<const uint4*>(src + 64 * (s / 2) + 16 * g + 8 * (s % 2)));
  }
  auto fill = [&](int32_t base) {  // slots (and scales) of the stage at `base`: one per thread
    const int32_t i = threadIdx.x, count = min(kLatentStage, t1 - base);
    const uint32_t s = i < count ? slot_of(a, row, row, 0, len, base + i) : kHidden;
    slots[i] = s;
    if constexpr (kFp8) scales[i] = s == kHidden ? 0.f : a.k_scale[s];
  };
  fill(t0);
  if constexpr (!kFp8) {
    landed();
    __syncthreads();
    const uint8_t* buf = reinterpret_cast<const uint8_t*>(odd[hw / 2]) + 16 * (hw % 2) * kRow;
#pragma unroll
    for (int s = 0; s < KS; ++s)
      keep_query(s, *reinterpret_cast<const uint4*>(buf + (koff ^ (s % 2 * 64)) + s / 2 * kBlock));
  }

  bool hidden = false;
  auto step = [&](int it, int pairs, uint4 (&tile)[2][32 * CH], uint4 (&next)[2][32 * CH]) __attribute__((always_inline)) {
    landed();  // this wave's loads ...
    if (hidden) clear_hidden(it, tile);
    barrier();  // ... and every wave's, and the other buffer is free
    const bool more = it + 1 < pairs;
    const uint8_t* src;
    hidden = row_at(more ? it + 1 : it, src);
    const uint8_t* buf = reinterpret_cast<const uint8_t*>(tile[grp]);
    const int first = (2 * it + grp) * 32;
    // Scores.  Fragment f = 2u + h: 16 bytes of token half h; kAhead reads are
    // under way (the barriers keep the compiler from undoing that).
    auto key = [&](int f) {
      const int u = f / 2, h = f % 2;
      const int x = kFp8 ? 16 * h : u % 2 * 64;  // fp8: the swizzle of rows 16 and up
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
      if (f % 4 == 0 && more) issue(f / 4, src, next);  // between the products: nine in a row would wait
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
    const int32_t pairs = (min(kLatentStage, t1 - base) + 63) / 64;
    if (base != t0) {
      __syncthreads();
      fill(base);
    }
    __syncthreads();
    const uint8_t* src;
    hidden = row_at(0, src);
#pragma unroll
    for (int n = 0; n < NI; ++n) issue(n, src, even);
    for (int32_t it = 0; it < pairs; it += 2) {
      step(it, pairs, even, odd);
      if (it + 1 < pairs) step(it + 1, pairs, odd, even);
    }
  }

  l = groups_sum(l);
  __syncthreads();
  if (g == 0) {
    top[grp][hw][c] = m;
    sum[grp][hw][c] = l;
  }
  if (grp == 0)
    hand_over<0>(a, acc, even, odd, top, sum, m, l, row, split, head0, hw, c, g);
  else
    hand_over<1>(a, acc, even, odd, top, sum, m, l, row, split, head0, hw, c, g);
}

}  // namespace

hipError_t launch_attend_latent(int32_t dtype, const Args& a, uint32_t grid, hipStream_t st) {
  if (dtype == kFP8)
    attend_latent_kernel<kFP8><<<grid, 512, 0, st>>>(a);
  else
    attend_latent_kernel<kBF16><<<grid, 512, 0, st>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  attend_join_kernel<kLatentV, false><<<dim3(a.heads, a.rows), 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace misa
