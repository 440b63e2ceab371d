// Checks of a paged cache's description (misa_cache in misa.h), shared by the C-ABI
// translation units.
#pragma once

#include "checks.hpp"
#include "launch.hpp"

namespace misa {

// The page table's half of a cache: sizes only.
inline misa_status check_table(const misa_cache* c, Cache& out) {
  if (!c) return MISA_ERR_INVALID_ARG;
  if (c->rows < 1 || c->row_pages < 1 || c->pages < 1 || c->page_tokens < 1)
    return MISA_ERR_INVALID_ARG;
  if (c->page_tokens > 4096 || c->rows > (1 << 20) || c->pages > (1 << 24) ||
      static_cast<int64_t>(c->rows) * c->row_pages >= (int64_t{1} << 31) ||
      static_cast<int64_t>(c->row_pages) * c->page_tokens > (int64_t{1} << 30))
    return MISA_ERR_UNSUPPORTED;
  out = Cache{c->rows, c->row_pages, c->pages,  c->page_tokens,
              c->kv_heads, c->dk, c->dv, c->kv_dtype};
  return MISA_OK;
}

// The whole cache: sizes, head dimensions and type.
inline misa_status check_cache(const misa_cache* c, Cache& out) {
  MISA_TRY(check_table(c, out));
  if (c->kv_heads < 1 || c->dk < 1 || c->dv < 1) return MISA_ERR_INVALID_ARG;
  if (c->kv_dtype < MISA_F32 || c->kv_dtype > MISA_FP8_E4M3) return MISA_ERR_INVALID_ARG;
  if (c->kv_dtype == MISA_F32 || c->kv_heads > 256) return MISA_ERR_UNSUPPORTED;
  // Slots (page, kv head, token) are 32-bit numbers.
  if (static_cast<int64_t>(c->pages) * c->kv_heads * c->page_tokens >= (int64_t{1} << 32) - 1)
    return MISA_ERR_UNSUPPORTED;
  if (out.latent()) return c->kv_heads == 1 ? MISA_OK : MISA_ERR_UNSUPPORTED;
  if (c->dk != c->dv || (c->dk != 64 && c->dk != 128 && c->dk != 256)) return MISA_ERR_UNSUPPORTED;
  return MISA_OK;
}

}  // namespace misa
