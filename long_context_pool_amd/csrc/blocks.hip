// The cache with one scale per block of tokens and head (misa_block_write and
// misa_block_read in misa.h).  Every id read from device memory (rows' ranges,
// lengths, pages) is range-checked before it becomes an address.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "packed.hpp"
#include "quant.hpp"

namespace misa {

namespace {

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

constexpr int kLeastScale = -100;  // exponent of the scale of a block of zeros

// The smallest 2^k, k >= -100, with amax <= 448 * 2^k = 1.75 * 2^(8 + k), for a
// finite amax >= 0.
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127;
  const int k = e - 8 + ((u & 0x7FFFFFu) > 0x600000u);
  return __uint_as_float(static_cast<uint32_t>(max(k, kLeastScale) + 127) << 23);
}

struct WriteArgs {
  Packed rows;
  const int32_t* lengths;
  const uint16_t* fresh[2];  // k_new, v_new
  uint8_t* pages_of[2];
  float* scale[2];
  const int32_t* table;
  int32_t row_pages, pages, P, kv_heads, shift;  // 2^shift tokens a block
  int32_t by_token;  // units are packed entries, not blocks
};

// One workgroup per (block with new tokens, kv head), for its keys and its values:
// D / 8 lanes hold eight values each of a token, and NP rounds of tokens a block, so
// that the block's values are read once, before its scale is known, and stay in
// registers.  (KV = 1: one of the two, by blockIdx.z, where both would take more
// registers than are there, or keys alone.)
//
// Units go by blocks (a row's c tokens touch at most floor(c / B) + 2) or, where
// there are fewer of them, by tokens: the first of a row and those that begin a
// block are at work, the other workgroups leave (32 rows with a token each: 32
// units for 64, 6.3 us for 7.1 a call; 1024 rows 30.6 us for 36.7; 256 rows with four each go by
// blocks, 13.0 us, by tokens 30.9; 8192 tokens of three rows 12.1 and 101).
//
// Bound by memory traffic: 8192 tokens of 8 heads of 128 (50 MB) 11.8 us, 4.3 TB/s (13
// us with keys and values in workgroups of their own); 32 rows with a token each 4.5 us,
// a launch and four dependent loads.
template <int D, int NP, int KV>
__global__ __launch_bounds__(256) void block_write_kernel(WriteArgs a) {
  constexpr int LPR = D / 8, TP = 256 / LPR;  // lanes of a token, tokens of a round
  __shared__ float tops[KV][4];
  const int head = blockIdx.y, B = 1 << a.shift;
  int32_t r, begin, end;
  int64_t block;  // of the row
  const int64_t u = blockIdx.x;
  if (a.by_token) {
    if (!row_of_entry(a.rows, static_cast<int32_t>(u), r, begin, end)) return;
  } else {
    r = last_row(a.rows.rows, u, [&](int32_t x) { return unit_base(a.rows.at(x), 1, a.shift, x, 2); });
    begin = a.rows.at(r);
    end = a.rows.at(r + 1);
    if (begin >= end) return;
  }
  const int64_t stop = a.lengths[r], start = stop - (end - begin);  // positions of the new tokens
  const int64_t from = start > 0 ? start : 0;
  if (a.by_token) {
    const int64_t p = start + (u - begin);
    if (p < from || (p != from && (p & (B - 1)) != 0)) return;
    block = p >> a.shift;
  } else {
    const int64_t j = u - unit_base(begin, 1, a.shift, r, 2);
    if (j < 0) return;
    block = (from >> a.shift) + j;
  }
  const int64_t p0 = block << a.shift;  // the block's first position
  if (p0 >= stop || p0 >= static_cast<int64_t>(a.row_pages) * a.P) return;
  const int32_t e = static_cast<int32_t>(static_cast<uint32_t>(p0) / static_cast<uint32_t>(a.P));  // p0 < 2^30
  const int32_t page = a.table[static_cast<int64_t>(r) * a.row_pages + e];
  const int32_t low = static_cast<int32_t>(from > p0 ? from - p0 : 0);            // first new token
  const int32_t high = static_cast<int32_t>(stop - p0 < B ? stop - p0 : B);  // one past the last
  const int lane = threadIdx.x % LPR, tok = threadIdx.x / LPR;

  const int64_t entry0 = begin + (p0 - start);  // packed entry of the block's first token
  uint4 x[KV][NP];
#pragma unroll
  for (int v = 0; v < KV; ++v) {
    const uint16_t* src = a.fresh[KV == 1 ? blockIdx.z : v] + head * D + lane * 8;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int32_t t = i * TP + tok;
      x[v][i] = make_uint4(0, 0, 0, 0);
      if (t >= low && t < high) x[v][i] = *reinterpret_cast<const uint4*>(src + (entry0 + t) * a.kv_heads * D);
    }
  }
  if (page < 0 || page >= a.pages) return;
  const int64_t slot0 = (static_cast<int64_t>(page) * a.kv_heads + head) * a.P + (p0 - static_cast<int64_t>(e) * a.P);
  float had[KV];
#pragma unroll
  for (int v = 0; v < KV; ++v) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const uint32_t w[4] = {x[v][i].x, x[v][i].y, x[v][i].z, x[v][i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float y0 = fabsf(__uint_as_float(w[j] << 16)), y1 = fabsf(__uint_as_float(w[j] & 0xFFFF0000u));
        top = fmaxf(top, y0 < INFINITY ? y0 : 0.f);
        top = fmaxf(top, y1 < INFINITY ? y1 : 0.f);
      }
    }
    top = lanes_reduce<kWave, true>(top);
    if (lane_id() == 0) tops[v][threadIdx.x / kWave] = top;
    had[v] = low > 0 ? a.scale[KV == 1 ? blockIdx.z : v][slot0 >> a.shift] : 0.f;
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < KV; ++v) {
    const int which = KV == 1 ? blockIdx.z : v;
    float unit = block_scale(fmaxf(fmaxf(tops[v][0], tops[v][1]), fmaxf(tops[v][2], tops[v][3])));
    const bool grown = low > 0 && had[v] < unit;
    if (low > 0 && had[v] > unit) unit = had[v];
    const float inv = 1.f / unit;  // exact
    uint8_t* dst = a.pages_of[which] + slot0 * D + lane * 8;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int32_t t = i * TP + tok;
      if (t >= low && t < high) {
        const uint32_t w[4] = {x[v][i].x, x[v][i].y, x[v][i].z, x[v][i].w};
        float y[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[2 * j] = __uint_as_float(w[j] << 16);
          y[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = fabsf(y[j]) < INFINITY ? y[j] : NAN;
        *reinterpret_cast<uint2*>(dst + static_cast<int64_t>(t) * D) =
            make_uint2(e4m3_pack4(y[0], y[1], y[2], y[3], inv), e4m3_pack4(y[4], y[5], y[6], y[7], inv));
      }
      if (grown && t < low) {  // earlier tokens, to the larger scale
        uint2* old = reinterpret_cast<uint2*>(dst + static_cast<int64_t>(t) * D);
        const uint2 z = *old;
        const float f = had[v] * inv;
        uint32_t c[2] = {z.x, z.y};
#pragma unroll
        for (int j = 0; j < 2; ++j)
          c[j] = e4m3_pack4(fp8_to_f32(c[j]), __builtin_amdgcn_cvt_f32_fp8(c[j], 1),
                            __builtin_amdgcn_cvt_f32_fp8(c[j], 2), __builtin_amdgcn_cvt_f32_fp8(c[j], 3), f);
        *old = make_uint2(c[0], c[1]);
      }
    }
    if (threadIdx.x == 0) a.scale[which][slot0 >> a.shift] = unit;
  }
}

template <int D, int NP>
void launch_write_rounds(const WriteArgs& a, uint32_t units, int32_t parts, hipStream_t st) {
  if (NP <= 4 && parts == 2)
    block_write_kernel<D, NP, NP <= 4 ? 2 : 1><<<dim3(units, a.kv_heads), 256, 0, st>>>(a);
  else
    block_write_kernel<D, NP, 1><<<dim3(units, a.kv_heads, parts), 256, 0, st>>>(a);
}

template <int D>
hipError_t launch_write_dim(const WriteArgs& a, uint32_t units, int32_t parts, hipStream_t st) {
  const int rounds = std::max(1, (D / 8 << a.shift) / 256);
  if (rounds == 1) launch_write_rounds<D, 1>(a, units, parts, st);
  if (rounds == 2) launch_write_rounds<D, 2>(a, units, parts, st);
  if (rounds == 4) launch_write_rounds<D, 4>(a, units, parts, st);
  if constexpr (D >= 128)
    if (rounds == 8) launch_write_rounds<D, 8>(a, units, parts, st);
  if constexpr (D >= 256)
    if (rounds == 16) launch_write_rounds<D, 16>(a, units, parts, st);
  return hipGetLastError();
}

// ---------------------------------------------------------------- reading back

struct ReadArgs {
  Packed rows;
  const int32_t *first, *lengths, *table;
  const uint8_t* pages_of[2];
  const float* scale[2];
  void* out[2];
  float* out_scale[2];
  int32_t row_pages, pages, P, kv_heads, shift;  // 2^shift tokens a block
};

// A lane's load and store: as many codes as make 16 bytes of OUT, so that a wave's
// stores are whole runs of the output (with 16 codes a lane, and stores of a lane's 64
// bytes of fp32 one after the other, 200 MB took 130 us instead of 53).
template <int OUT>
constexpr int kPerLane = 16 / elem_bytes<OUT>();

template <int N, bool ONCE>
__device__ __forceinline__ void get(const uint8_t* p, uint32_t (&to)[N]) {
  typedef __attribute__((ext_vector_type(N))) uint32_t V;
  const V* q = reinterpret_cast<const V*>(p);
  const V x = ONCE ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
  for (int i = 0; i < N; ++i) to[i] = x[i];
}

// The codes of a lane -> 16 bytes of OUT at `dst`.
template <int OUT, bool ONCE>
__device__ __forceinline__ void put(void* dst, const uint32_t (&c)[kPerLane<OUT> / 4], float scale) {
  u32x4 x;
  if constexpr (OUT == kFP8) {
    x = u32x4{c[0], c[1], c[2], c[3]};
  } else {
    float y[kPerLane<OUT>];
#pragma unroll
    for (int j = 0; j < kPerLane<OUT> / 4; ++j) {
      y[4 * j] = fp8_to_f32(c[j]) * scale;
      y[4 * j + 1] = __builtin_amdgcn_cvt_f32_fp8(c[j], 1) * scale;
      y[4 * j + 2] = __builtin_amdgcn_cvt_f32_fp8(c[j], 2) * scale;
      y[4 * j + 3] = __builtin_amdgcn_cvt_f32_fp8(c[j], 3) * scale;
    }
    if constexpr (OUT == kF32) {
      x = __builtin_bit_cast(u32x4, make_float4(y[0], y[1], y[2], y[3]));
    } else {
      typedef __attribute__((ext_vector_type(8))) __bf16 B8;
      B8 b;
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] = static_cast<__bf16>(y[j]);
      x = __builtin_bit_cast(u32x4, b);
    }
  }
  if constexpr (ONCE)
    __builtin_nontemporal_store(x, static_cast<u32x4*>(dst));
  else
    *static_cast<u32x4*>(dst) = x;
}

// Rounds of a lane, whose loads are under way together (twice as many for bf16 and fp32:
// 9.5 and 16.1 us for 2 rows of 2000 tokens of 8 heads, 8.8 and 13.2 with these).
template <int OUT>
constexpr int kRounds = OUT == kF32 ? 4 : 2;

// Lanes of a (packed token, kv head) that have kPerLane codes each.  The row of a workgroup's tokens, mostly one,
// is looked up once: a lookup each cost 8 rows of 131072 keys (213 MB) 20 of 70 us.
// Bound by HBM traffic, 5.1 TB/s there.
//
// ONCE: much is moved, and marked as not to be kept (41.7 us there, 47.1 without; bf16
// rows, 98 MB 25.4 and 27.3 us, 31 MB 10.7 and 9.9; between 32 and 64 MB plain loads are still
// ahead where the cache is on the chip from the call before: 49 MB 14.6 and 12.6).
template <int D, int OUT, bool ONCE>
__global__ __launch_bounds__(256) void block_read_kernel(ReadArgs a) {
  constexpr int N = kPerLane<OUT>, kReadRounds = kRounds<OUT>;
  constexpr int LPR = D / N, IP = 256 / LPR;  // lanes of an item, items of a round
  const int which = blockIdx.y;
  const int lane = threadIdx.x % LPR;
  const int64_t items = static_cast<int64_t>(a.rows.n) * a.kv_heads;
  const int64_t item0 = static_cast<int64_t>(blockIdx.x) * (IP * kReadRounds);
  // The rows of the workgroup's first and last token; mostly the same.
  const int32_t t0 = static_cast<int32_t>(item0 / a.kv_heads);
  const int32_t t1 = static_cast<int32_t>((min(item0 + IP * kReadRounds, items) - 1) / a.kv_heads);
  const auto offset = [&](int32_t x) { return static_cast<int64_t>(a.rows.at(x)); };
  const int32_t r0 = last_row(a.rows.rows, t0, offset);
  int32_t r1 = r0;
  if (a.rows.at(r0 + 1) <= t1) r1 = last_row(a.rows.rows, t1, offset);
  uint32_t code[kReadRounds][N / 4];
  float unit[kReadRounds];
  int64_t item[kReadRounds];
  const auto fetch = [&](int i, int32_t r, int32_t t, int32_t head, int32_t begin, int32_t end, int32_t first, int32_t len)
                         __attribute__((always_inline)) {
    if (t < begin || t >= end) {  // padding
      item[i] = -1;
      return;
    }
    const int64_t p = static_cast<int64_t>(first) + (t - begin);
    if (p < 0 || p >= len || p >= static_cast<int64_t>(a.row_pages) * a.P) return;
    const uint32_t e = static_cast<uint32_t>(p) / static_cast<uint32_t>(a.P);
    const int32_t page = a.table[static_cast<int64_t>(r) * a.row_pages + e];
    if (page < 0 || page >= a.pages) return;
    const int64_t slot = (static_cast<int64_t>(page) * a.kv_heads + head) * a.P + (p - static_cast<int64_t>(e) * a.P);
    get<N / 4, ONCE>(a.pages_of[which] + slot * D + lane * N, code[i]);
    unit[i] = a.scale[which][static_cast<uint32_t>(slot) >> a.shift];
  };
  const int32_t begin0 = a.rows.at(r0), end0 = a.rows.at(r0 + 1), first0 = a.first ? a.first[r0] : 0, len0 = a.lengths[r0];
#pragma unroll
  for (int i = 0; i < kReadRounds; ++i) {
    item[i] = item0 + i * IP + threadIdx.x / LPR;
#pragma unroll
    for (int j = 0; j < N / 4; ++j) code[i][j] = 0;
    unit[i] = 1.f;
    if (item[i] >= items) {
      item[i] = -1;
      continue;
    }
    const int32_t t = static_cast<int32_t>(static_cast<uint32_t>(item[i]) / static_cast<uint32_t>(a.kv_heads));
    const int32_t head = static_cast<int32_t>(item[i] - static_cast<int64_t>(t) * a.kv_heads);
    if (r0 == r1) {  // uniform: the row's numbers are there already
      fetch(i, r0, t, head, begin0, end0, first0, len0);
      continue;
    }
    int32_t lo = r0, hi = r1;  // the last row whose entries begin at or before t
    while (lo < hi) {
      const int32_t mid = lo + (hi - lo + 1) / 2;
      if (a.rows.at(mid) <= t)
        lo = mid;
      else
        hi = mid - 1;
    }
    fetch(i, lo, t, head, a.rows.at(lo), a.rows.at(lo + 1), a.first ? a.first[lo] : 0, a.lengths[lo]);
  }
#pragma unroll
  for (int i = 0; i < kReadRounds; ++i) {
    if (item[i] < 0) continue;
    put<OUT, ONCE>(static_cast<uint8_t*>(a.out[which]) + (item[i] * D + lane * N) * elem_bytes<OUT>(), code[i], unit[i]);
    if (OUT == kFP8 && lane == 0) a.out_scale[which][item[i]] = unit[i];
  }
}

constexpr int64_t kReadOnceBytes = int64_t{32} << 20;

template <int D, int OUT>
hipError_t launch_read_out(const ReadArgs& a, int32_t parts, hipStream_t st) {
  const int64_t items = static_cast<int64_t>(a.rows.n) * a.kv_heads;  // at most 2^27
  const int per = 256 / (D / kPerLane<OUT>)*kRounds<OUT>;
  const dim3 grid(static_cast<uint32_t>((items + per - 1) / per), parts);
  if (items * D * parts * (1 + elem_bytes<OUT>()) >= kReadOnceBytes)
    block_read_kernel<D, OUT, true><<<grid, 256, 0, st>>>(a);
  else
    block_read_kernel<D, OUT, false><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

template <int D>
hipError_t launch_read_dim(const ReadArgs& a, int32_t out_dtype, int32_t parts, hipStream_t st) {
  switch (out_dtype) {
    case kF32: return launch_read_out<D, kF32>(a, parts, st);
    case kBF16: return launch_read_out<D, kBF16>(a, parts, st);
    default: return launch_read_out<D, kFP8>(a, parts, st);
  }
}

}  // namespace

hipError_t launch_block_write(const Cache& c, int32_t block, int32_t n, const int32_t* offsets,
                              const int32_t* lengths, const void* k_new, const void* v_new,
                              void* k_pages, float* k_scale, void* v_pages, float* v_scale,
                              const int32_t* table, hipStream_t st) {
  WriteArgs a{};
  a.rows = Packed{offsets, c.rows, n};
  a.lengths = lengths;
  a.fresh[0] = static_cast<const uint16_t*>(k_new);
  a.fresh[1] = static_cast<const uint16_t*>(v_new);
  a.pages_of[0] = static_cast<uint8_t*>(k_pages);
  a.pages_of[1] = static_cast<uint8_t*>(v_pages);
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.table = table;
  a.row_pages = c.row_pages;
  a.pages = c.pages;
  a.P = c.P;
  a.kv_heads = c.kv_heads;
  a.shift = __builtin_ctz(static_cast<uint32_t>(block));
  const int64_t blocks = unit_base(n, 1, a.shift, c.rows, 2);
  a.by_token = n <= blocks;
  const uint32_t units = static_cast<uint32_t>(a.by_token ? n : blocks);
  const int32_t parts = v_pages ? 2 : 1;
  switch (c.dk) {
    case 64: return launch_write_dim<64>(a, units, parts, st);
    case 128: return launch_write_dim<128>(a, units, parts, st);
    default: return launch_write_dim<256>(a, units, parts, st);
  }
}

hipError_t launch_block_read(const Cache& c, int32_t block, int32_t n, int32_t out_dtype,
                             const int32_t* offsets, const int32_t* first, const int32_t* lengths,
                             const void* k_pages, const float* k_scale, const void* v_pages,
                             const float* v_scale, const int32_t* table, void* k_out,
                             float* k_out_scale, void* v_out, float* v_out_scale, hipStream_t st) {
  ReadArgs a{};
  a.rows = Packed{offsets, c.rows, n};
  a.first = first;
  a.lengths = lengths;
  a.table = table;
  a.pages_of[0] = static_cast<const uint8_t*>(k_pages);
  a.pages_of[1] = static_cast<const uint8_t*>(v_pages);
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.out[0] = k_out;
  a.out[1] = v_out;
  a.out_scale[0] = k_out_scale;
  a.out_scale[1] = v_out_scale;
  a.row_pages = c.row_pages;
  a.pages = c.pages;
  a.P = c.P;
  a.kv_heads = c.kv_heads;
  a.shift = __builtin_ctz(static_cast<uint32_t>(block));
  const int32_t parts = v_pages ? 2 : 1;
  switch (c.dk) {
    case 64: return launch_read_dim<64>(a, out_dtype, parts, st);
    case 128: return launch_read_dim<128>(a, out_dtype, parts, st);
    default: return launch_read_dim<256>(a, out_dtype, parts, st);
  }
}

}  // namespace misa
