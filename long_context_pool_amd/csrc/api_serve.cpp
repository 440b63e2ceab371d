// C ABI of the serving operators (declared in include/misa.h): argument checks
// on the host, workspace sizing, and dispatch to the kernels on the caller's
// stream.  Nothing here allocates device memory.
#include "misa.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "cache_checks.hpp"
#include "launch.hpp"

namespace {

using misa::Cache;
using misa::check_cache;
using misa::check_out;
using misa::check_table;
using misa::check_ws;
using misa::from_hip;

// The cache's pools: values and their scales only where the cache has them.
misa_status check_pools(const Cache& c, const void* k_pages, const float* k_scale,
                        const void* v_pages, const float* v_scale) {
  const bool fp8 = c.dtype == MISA_FP8_E4M3;
  MISA_TRY(check_out(k_pages, true));
  if (fp8) MISA_TRY(check_out(k_scale, true));
  if (c.latent()) return v_pages || (fp8 && v_scale) ? MISA_ERR_INVALID_ARG : MISA_OK;
  MISA_TRY(check_out(v_pages, true));
  if (fp8) MISA_TRY(check_out(v_scale, true));
  return MISA_OK;
}

misa_status check_list(int32_t n) {
  if (n < 0) return MISA_ERR_INVALID_ARG;
  return n > misa::kMaxList ? MISA_ERR_UNSUPPORTED : MISA_OK;
}

misa_status check_attend(const misa_cache* cache, int32_t heads, int32_t k, Cache& c) {
  MISA_TRY(check_cache(cache, c));
  if (heads < 1 || k < 0 || heads % c.kv_heads != 0) return MISA_ERR_INVALID_ARG;
  if (heads > 1024 || k > (1 << 20) || c.rows > 65535) return MISA_ERR_UNSUPPORTED;
  return MISA_OK;
}

}  // namespace

extern "C" {

size_t misa_attend_workspace_bytes(const misa_cache* cache, int32_t heads, int32_t k) {
  Cache c;
  if (check_attend(cache, heads, k, c) != MISA_OK) return 0;
  return misa::attend_ws_bytes(c, heads, k);
}

misa_status misa_attend(const misa_cache* cache, int32_t heads, int32_t k, float scale,
                        const void* q, const void* k_pages, const float* k_scale,
                        const void* v_pages, const float* v_scale, const int32_t* table,
                        const int32_t* lengths, const int32_t* idx, void* out, float* lse,
                        void* ws, size_t ws_bytes, hipStream_t stream) {
  Cache c;
  MISA_TRY(check_attend(cache, heads, k, c));
  if (!std::isfinite(scale)) return MISA_ERR_INVALID_ARG;
  if (!std::isfinite(scale * misa::kLog2e)) return MISA_ERR_UNSUPPORTED;
  MISA_TRY(check_pools(c, k_pages, k_scale, v_pages, v_scale));
  MISA_TRY(check_out(q, true));
  MISA_TRY(check_out(table, true));
  MISA_TRY(check_out(lengths, true));
  if ((k > 0) != (idx != nullptr)) return MISA_ERR_INVALID_ARG;
  MISA_TRY(check_out(idx, false));
  MISA_TRY(check_out(out, true));
  MISA_TRY(check_out(lse, false));
  MISA_TRY(check_ws(ws, ws_bytes, misa::attend_ws_bytes(c, heads, k)));
  return from_hip(misa::launch_attend(c, heads, k, scale, q, k_pages, k_scale, v_pages, v_scale,
                                      table, lengths, idx, out, lse, ws, stream));
}

misa_status misa_page_write(const misa_cache* cache, int32_t n, const int32_t* row,
                            const int32_t* pos, const void* k_new, const void* v_new,
                            void* k_pages, float* k_scale, void* v_pages, float* v_scale,
                            const int32_t* table, hipStream_t stream) {
  Cache c;
  MISA_TRY(check_cache(cache, c));
  if (n < 0) return MISA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(n) * c.kv_heads > (int64_t{1} << 25)) return MISA_ERR_UNSUPPORTED;
  MISA_TRY(check_pools(c, k_pages, k_scale, v_pages, v_scale));
  MISA_TRY(check_out(table, true));
  if (n == 0) return MISA_OK;
  MISA_TRY(check_out(row, true));
  MISA_TRY(check_out(pos, true));
  MISA_TRY(check_out(k_new, true));
  if (c.latent() ? v_new != nullptr : check_out(v_new, true) != MISA_OK)
    return MISA_ERR_INVALID_ARG;
  return from_hip(misa::launch_page_write(c, n, row, pos, k_new, v_new, k_pages, k_scale, v_pages,
                                          v_scale, table, stream));
}

misa_status misa_page_extend(const misa_cache* cache, int32_t n, const int32_t* row,
                             const int32_t* count, int32_t* table, int32_t* lengths,
                             int32_t* refs, int32_t* ok, hipStream_t stream) {
  Cache c;
  MISA_TRY(check_table(cache, c));
  MISA_TRY(check_list(n));
  MISA_TRY(check_out(table, true));
  MISA_TRY(check_out(lengths, true));
  MISA_TRY(check_out(refs, true));
  if (n == 0) return MISA_OK;
  MISA_TRY(check_out(row, true));
  MISA_TRY(check_out(count, true));
  MISA_TRY(check_out(ok, true));
  return from_hip(misa::launch_page_extend(c, n, row, count, table, lengths, refs, ok, stream));
}

misa_status misa_page_fork(const misa_cache* cache, int32_t n, const int32_t* parent,
                           const int32_t* child, int32_t* table, int32_t* lengths, int32_t* refs,
                           int32_t* src, int32_t* dst, int32_t* ok, hipStream_t stream) {
  Cache c;
  MISA_TRY(check_table(cache, c));
  MISA_TRY(check_list(n));
  MISA_TRY(check_out(table, true));
  MISA_TRY(check_out(lengths, true));
  MISA_TRY(check_out(refs, true));
  if (n == 0) return MISA_OK;
  MISA_TRY(check_out(parent, true));
  MISA_TRY(check_out(child, true));
  MISA_TRY(check_out(src, true));
  MISA_TRY(check_out(dst, true));
  MISA_TRY(check_out(ok, true));
  return from_hip(
      misa::launch_page_fork(c, n, parent, child, table, lengths, refs, src, dst, ok, stream));
}

misa_status misa_page_free(const misa_cache* cache, int32_t n, const int32_t* row, int32_t* table,
                           int32_t* lengths, int32_t* refs, hipStream_t stream) {
  Cache c;
  MISA_TRY(check_table(cache, c));
  MISA_TRY(check_list(n));
  MISA_TRY(check_out(table, true));
  MISA_TRY(check_out(lengths, true));
  MISA_TRY(check_out(refs, true));
  if (n == 0) return MISA_OK;
  MISA_TRY(check_out(row, true));
  return from_hip(misa::launch_page_free(c, n, row, table, lengths, refs, stream));
}

size_t misa_page_workspace_bytes(const misa_cache* cache) {
  Cache c;
  return check_table(cache, c) == MISA_OK ? misa::page_compact_ws_bytes(c) : 0;
}

misa_status misa_page_compact(const misa_cache* cache, const int32_t* table, const int32_t* refs,
                              int32_t* table_out, int32_t* refs_out, int32_t* map, int32_t* live,
                              int32_t* src, int32_t* dst, void* ws, size_t ws_bytes,
                              hipStream_t stream) {
  Cache c;
  MISA_TRY(check_table(cache, c));
  MISA_TRY(check_out(table, true));
  MISA_TRY(check_out(refs, true));
  MISA_TRY(check_out(table_out, true));
  MISA_TRY(check_out(refs_out, true));
  MISA_TRY(check_out(map, true));
  MISA_TRY(check_out(live, true));
  MISA_TRY(check_out(src, true));
  MISA_TRY(check_out(dst, true));
  MISA_TRY(check_ws(ws, ws_bytes, misa::page_compact_ws_bytes(c)));
  return from_hip(misa::launch_page_compact(c, table, refs, table_out, refs_out, map, live, src,
                                            dst, ws, stream));
}

misa_status misa_page_copy(const misa_page_buffer* buffers, int32_t n_buffers, int32_t pages,
                           int32_t n, const int32_t* src, const int32_t* dst, hipStream_t stream) {
  if (!buffers || n_buffers < 1 || pages < 1 || n < 0) return MISA_ERR_INVALID_ARG;
  if (n_buffers > misa::kMaxPageBuffers || pages > (1 << 24)) return MISA_ERR_UNSUPPORTED;
  misa::PageBuffers b{};
  b.n = n_buffers;
  for (int32_t i = 0; i < n_buffers; ++i) {
    const misa_page_buffer& x = buffers[i];
    MISA_TRY(check_out(x.data, true));
    if (x.page_bytes < 4 || x.page_bytes % 4 != 0 || x.planes < 1) return MISA_ERR_INVALID_ARG;
    if (x.page_bytes > (int64_t{1} << 31) || x.planes > 65536) return MISA_ERR_UNSUPPORTED;
    // Byte offsets inside a buffer stay below 2^62 (pages * planes is at most 2^40).
    if (x.page_bytes > (int64_t{1} << 62) / (static_cast<int64_t>(pages) * x.planes))
      return MISA_ERR_UNSUPPORTED;
    b.b[i] = {static_cast<uint8_t*>(x.data), x.page_bytes, x.planes};
  }
  if (n == 0) return MISA_OK;
  MISA_TRY(check_out(src, true));
  MISA_TRY(check_out(dst, true));
  if (!misa::page_copy_supported(b, n)) return MISA_ERR_UNSUPPORTED;
  return from_hip(misa::launch_page_copy(b, pages, n, src, dst, stream));
}

misa_status misa_rms_norm(int32_t rows, int32_t n, int32_t groups, int32_t x_dtype,
                          int32_t out_dtype, float eps, const void* x, const void* residual,
                          const float* weight, void* sum_out, void* out, float* out_scale,
                          hipStream_t stream) {
  if (rows < 0 || n < 1 || groups < 1 || n % groups != 0) return MISA_ERR_INVALID_ARG;
  if (x_dtype < MISA_F32 || x_dtype > MISA_FP8_E4M3 || out_dtype < MISA_F32 ||
      out_dtype > MISA_FP8_E4M3)
    return MISA_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return MISA_ERR_INVALID_ARG;
  if (x_dtype == MISA_FP8_E4M3 || n > misa::kMaxNorm || rows >= (1 << 24))
    return MISA_ERR_UNSUPPORTED;
  if (rows == 0) return MISA_OK;
  MISA_TRY(check_out(x, true));
  MISA_TRY(check_out(residual, false));
  MISA_TRY(check_out(weight, true));
  MISA_TRY(check_out(sum_out, false));
  MISA_TRY(check_out(out, true));
  if (out_dtype == MISA_FP8_E4M3) MISA_TRY(check_out(out_scale, true));
  return from_hip(misa::launch_rms_norm(rows, n, groups, x_dtype, out_dtype, eps, x, residual,
                                        weight, sum_out, out, out_scale, stream));
}

}  // extern "C"
