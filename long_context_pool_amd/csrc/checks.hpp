// Host-side argument checks shared by the C-ABI translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "misa.h"

#define MISA_TRY(expr)                   \
  do {                                   \
    const misa_status st_ = (expr);      \
    if (st_ != MISA_OK) return st_;      \
  } while (0)

namespace misa {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline misa_status check_out(const void* p, bool required) {
  if (!p) return required ? MISA_ERR_INVALID_ARG : MISA_OK;
  return aligned16(p) ? MISA_OK : MISA_ERR_INVALID_ARG;
}

inline misa_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return MISA_OK;
  if (!ws || ws_bytes < need) return MISA_ERR_WORKSPACE;
  if (!aligned16(ws)) return MISA_ERR_INVALID_ARG;
  return MISA_OK;
}

inline misa_status from_hip(hipError_t e) { return e == hipSuccess ? MISA_OK : MISA_ERR_HIP; }

}  // namespace misa
