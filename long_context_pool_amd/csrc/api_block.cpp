// C ABI of rotary positions and of the cache with one scale per block of tokens
// (declared in include/misa.h): argument checks on the host and dispatch to the
// kernels on the caller's stream.  Nothing here allocates device memory.
#include "misa.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "cache_checks.hpp"
#include "launch.hpp"

namespace {

using misa::Cache;
using misa::check_out;
using misa::check_ws;
using misa::from_hip;

misa_status check_block_cache(const misa_cache* cache, int32_t block, Cache& c) {
  MISA_TRY(misa::check_cache(cache, c));
  if (block < 1) return MISA_ERR_INVALID_ARG;
  if (c.dtype != MISA_FP8_E4M3 || c.latent() || c.rows > 65535) return MISA_ERR_UNSUPPORTED;
  if ((block & (block - 1)) != 0 || block < 16 || block > 128) return MISA_ERR_UNSUPPORTED;
  return c.P % block == 0 ? MISA_OK : MISA_ERR_INVALID_ARG;
}

// Keys, and values or none at all: `more` is the values' other array.
misa_status check_block_pools(const void* k_pages, const float* k_scale, const void* v_pages,
                              const float* v_scale, const void* more) {
  MISA_TRY(check_out(k_pages, true));
  MISA_TRY(check_out(k_scale, true));
  const bool values = v_pages != nullptr;
  if (values != (v_scale != nullptr) || values != (more != nullptr)) return MISA_ERR_INVALID_ARG;
  MISA_TRY(check_out(v_pages, false));
  MISA_TRY(check_out(v_scale, false));
  return check_out(more, false);
}

// One query at a time where each has a list of its own, or a row has one new token (8
// rows of 131072 tokens, 64 heads on 8: 297 us, 310 in tiles; 32 rows of 8192 86 and 96
// us); otherwise tiles of a row's queries share its keys and values (two on 16 rows of
// 32768: 160 us, 278 one by one).
bool one_by_one(const misa::BlockAttend& b) { return b.k > 0 || b.most <= 1; }

misa_status check_block_attend(const misa_cache* cache, int32_t heads, misa::BlockAttend& b, Cache& c) {
  MISA_TRY(check_block_cache(cache, b.block, c));
  if (heads < 1 || b.k < 0 || b.n < 0 || b.most < 0 || heads % c.kv_heads != 0)
    return MISA_ERR_INVALID_ARG;
  if (heads > 1024 || b.k > (1 << 20) || b.n > (1 << 20) ||
      static_cast<int64_t>(b.n) * heads > (int64_t{1} << 26))
    return MISA_ERR_UNSUPPORTED;
  // A launch has fewer than 2^24 workgroups of 256: at most one for each query and
  // head, or 2^20 of whole tiles and one more for each row and kv head.
  if ((one_by_one(b) ? static_cast<int64_t>(b.n) * heads : static_cast<int64_t>(c.rows) * c.kv_heads) >
      (int64_t{1} << 23))
    return MISA_ERR_UNSUPPORTED;
  b.heads = heads;
  return MISA_OK;
}

size_t attend_need(const Cache& c, const misa::BlockAttend& b) {
  if (b.n == 0) return 0;
  return one_by_one(b) ? misa::attend_queries_ws_bytes(c, b) : misa::attend_tiles_ws_bytes(c, b);
}

}  // namespace

extern "C" {

misa_status misa_rope(const misa_rope_spec* spec, int32_t n, const void* x, const int32_t* pos,
                      const double* freq, void* out, float* out_scale, hipStream_t stream) {
  if (!spec || n < 0) return MISA_ERR_INVALID_ARG;
  const misa_rope_spec& s = *spec;
  if (s.heads < 1 || s.d < 1 || s.first < 0 || s.rot < 2 || s.rot % 2 != 0 || s.rot > s.d ||
      s.first > s.d - s.rot)
    return MISA_ERR_INVALID_ARG;
  if (s.pairs != MISA_ROPE_HALF && s.pairs != MISA_ROPE_INTERLEAVED) return MISA_ERR_INVALID_ARG;
  if (s.x_dtype < MISA_F32 || s.x_dtype > MISA_FP8_E4M3 || s.out_dtype < MISA_F32 ||
      s.out_dtype > MISA_FP8_E4M3 || !std::isfinite(s.amplitude))
    return MISA_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(s.heads) * s.d;
  if (s.x_stride < row || s.out_stride < row) return MISA_ERR_INVALID_ARG;
  if (s.x_dtype == MISA_FP8_E4M3 || row > misa::kMaxRopeRow || s.rot > misa::kMaxRot ||
      n >= (1 << 24) || s.x_stride >= (int64_t{1} << 31) || s.out_stride >= (int64_t{1} << 31))
    return MISA_ERR_UNSUPPORTED;
  if (s.out_dtype == MISA_FP8_E4M3 && s.out_stride != row) return MISA_ERR_INVALID_ARG;
  if (n == 0) return MISA_OK;
  MISA_TRY(check_out(x, true));
  MISA_TRY(check_out(pos, true));
  MISA_TRY(check_out(freq, true));
  MISA_TRY(check_out(out, true));
  if (s.out_dtype == MISA_FP8_E4M3) MISA_TRY(check_out(out_scale, true));
  if (x == out && (s.x_dtype != s.out_dtype || s.x_stride != s.out_stride)) return MISA_ERR_INVALID_ARG;
  return from_hip(misa::launch_rope(misa::Rope{s.heads, s.d, s.first, s.rot, s.pairs, s.x_dtype,
                                               s.out_dtype, s.amplitude, s.x_stride, s.out_stride},
                                    n, x, pos, freq, out, out_scale, stream));
}

misa_status misa_rope_frequencies(const misa_rope_scaling* scaling, double* freq,
                                  float* amplitude) {
  if (!scaling || !freq || !amplitude) return MISA_ERR_INVALID_ARG;
  const misa_rope_scaling& s = *scaling;
  if (s.kind < MISA_ROPE_PLAIN || s.kind > MISA_ROPE_PARTS || s.rot < 2 || s.rot % 2 != 0 ||
      !(s.base > 1.0) || !std::isfinite(s.base))
    return MISA_ERR_INVALID_ARG;
  if (s.kind != MISA_ROPE_PLAIN && (!(s.factor >= 1.0) || !std::isfinite(s.factor)))
    return MISA_ERR_INVALID_ARG;
  if (s.kind == MISA_ROPE_PARTS &&
      (!(s.original > 0.0) || !(s.slow > 0.0) || !(s.fast >= s.slow) || !std::isfinite(s.original) ||
       !std::isfinite(s.fast)))
    return MISA_ERR_INVALID_ARG;
  if (s.rot > misa::kMaxRot) return MISA_ERR_UNSUPPORTED;
  const int32_t pairs = s.rot / 2;
  // The pair that turns `turns` times in the original context: original * base^(-2i
  // / rot) = 2 pi turns.
  const auto pair_of = [&](double turns) {
    return s.rot * std::log(s.original / (2.0 * M_PI * turns)) / (2.0 * std::log(s.base));
  };
  // The ramp's ends.  Its upper one lies behind the last pair where that one turns often
  // enough, as far as the rotated size less one.
  double first = 0.0, last = 0.0, low = 0.0, high = 1.0;
  if (s.kind == MISA_ROPE_PARTS) {
    first = pair_of(s.fast);
    last = pair_of(s.slow);
    low = std::max(std::floor(first), 0.0);
    high = std::min(std::ceil(last), s.rot - 1.0);
  }
  for (int32_t i = 0; i < pairs; ++i) {
    const double f = std::pow(s.base, -2.0 * i / s.rot);
    double slowed = s.kind == MISA_ROPE_LINEAR ? 1.0 : 0.0;  // share of f / factor
    if (s.kind == MISA_ROPE_PARTS && i > first)  // i >= last: also where no pair turns `slow` times
      slowed = i >= last ? 1.0 : std::min(std::max((i - low) / std::max(high - low, 1e-3), 0.0), 1.0);
    freq[i] = s.kind == MISA_ROPE_PLAIN ? f : f * (1.0 - slowed + slowed / s.factor);
  }
  *amplitude = s.kind == MISA_ROPE_PARTS ? static_cast<float>(1.0 + 0.1 * std::log(s.factor)) : 1.f;
  return MISA_OK;
}

misa_status misa_block_write(const misa_cache* cache, int32_t block_tokens, int32_t n,
                             const int32_t* offsets, const int32_t* lengths, const void* k_new,
                             const void* v_new, void* k_pages, float* k_scale, void* v_pages,
                             float* v_scale, const int32_t* table, hipStream_t stream) {
  Cache c;
  MISA_TRY(check_block_cache(cache, block_tokens, c));
  if (n < 0) return MISA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(n) * c.kv_heads > (int64_t{1} << 25)) return MISA_ERR_UNSUPPORTED;
  if (n == 0) return MISA_OK;
  MISA_TRY(check_block_pools(k_pages, k_scale, v_pages, v_scale, v_new));
  MISA_TRY(check_out(offsets, true));
  MISA_TRY(check_out(lengths, true));
  MISA_TRY(check_out(k_new, true));
  MISA_TRY(check_out(table, true));
  return from_hip(misa::launch_block_write(c, block_tokens, n, offsets, lengths, k_new, v_new,
                                           k_pages, k_scale, v_pages, v_scale, table, stream));
}

misa_status misa_block_read(const misa_cache* cache, int32_t block_tokens, int32_t n,
                            int32_t out_dtype, const int32_t* offsets, const int32_t* first,
                            const int32_t* lengths, const void* k_pages, const float* k_scale,
                            const void* v_pages, const float* v_scale, const int32_t* table,
                            void* k_out, float* k_out_scale, void* v_out, float* v_out_scale,
                            hipStream_t stream) {
  Cache c;
  MISA_TRY(check_block_cache(cache, block_tokens, c));
  if (n < 0 || out_dtype < MISA_F32 || out_dtype > MISA_FP8_E4M3) return MISA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(n) * c.kv_heads > (int64_t{1} << 27)) return MISA_ERR_UNSUPPORTED;
  if (n == 0) return MISA_OK;
  MISA_TRY(check_block_pools(k_pages, k_scale, v_pages, v_scale, v_out));
  MISA_TRY(check_out(offsets, true));
  MISA_TRY(check_out(first, false));
  MISA_TRY(check_out(lengths, true));
  MISA_TRY(check_out(table, true));
  MISA_TRY(check_out(k_out, true));
  if (out_dtype == MISA_FP8_E4M3) {
    MISA_TRY(check_out(k_out_scale, true));
    MISA_TRY(check_out(v_out_scale, v_pages != nullptr));
  }
  return from_hip(misa::launch_block_read(c, block_tokens, n, out_dtype, offsets, first, lengths,
                                          k_pages, k_scale, v_pages, v_scale, table, k_out,
                                          k_out_scale, v_out, v_out_scale, stream));
}

size_t misa_block_attend_workspace_bytes(const misa_cache* cache, int32_t block_tokens,
                                         int32_t heads, int32_t n, int32_t most, int32_t k) {
  Cache c;
  misa::BlockAttend b{};
  b.block = block_tokens;
  b.n = n;
  b.most = most;
  b.k = k;
  return check_block_attend(cache, heads, b, c) == MISA_OK ? attend_need(c, b) : 0;
}

misa_status misa_block_attend(const misa_cache* cache, int32_t block_tokens, int32_t heads,
                              int32_t n, int32_t most, int32_t k, float scale,
                              const int32_t* offsets, const void* q, const void* k_pages,
                              const float* k_scale, const void* v_pages, const float* v_scale,
                              const int32_t* table, const int32_t* lengths, const int32_t* idx,
                              void* out, float* lse, void* ws, size_t ws_bytes,
                              hipStream_t stream) {
  Cache c;
  misa::BlockAttend b{block_tokens, heads, n,     most,    k,      scale,   offsets, q,  k_pages, k_scale,
                      v_pages,      v_scale, table, lengths, idx, out, lse, ws};
  MISA_TRY(check_block_attend(cache, heads, b, c));
  if (!std::isfinite(scale)) return MISA_ERR_INVALID_ARG;
  if (!std::isfinite(scale * misa::kLog2e)) return MISA_ERR_UNSUPPORTED;
  if ((k > 0) != (idx != nullptr)) return MISA_ERR_INVALID_ARG;
  if (n == 0) return MISA_OK;
  MISA_TRY(check_block_pools(k_pages, k_scale, v_pages, v_scale, v_pages));
  if (!v_pages) return MISA_ERR_INVALID_ARG;
  MISA_TRY(check_out(offsets, true));
  MISA_TRY(check_out(q, true));
  MISA_TRY(check_out(table, true));
  MISA_TRY(check_out(lengths, true));
  MISA_TRY(check_out(idx, false));
  MISA_TRY(check_out(out, true));
  MISA_TRY(check_out(lse, false));
  MISA_TRY(check_ws(ws, ws_bytes, attend_need(c, b)));
  return from_hip(one_by_one(b) ? misa::launch_attend_queries(c, b, stream)
                                : misa::launch_attend_tiles(c, b, stream));
}

}  // extern "C"
