// Packed batches of rows (offsets [rows + 1] in misa.h): which row an entry, or
// a unit of a row's work, belongs to.
#pragma once

#include "common.hpp"

namespace misa {

struct Packed {
  const int32_t* offsets;
  int32_t rows, n;
  // Whatever the array holds, entries stay in [0, n].
  __device__ __forceinline__ int32_t at(int32_t r) const { return min(max(offsets[r], 0), n); }
};

// The last row r with f(r) <= u, for an f that grows with r, or 0; a wave looks
// at 64 rows at a time.  An f that does not grow (offsets that do not ascend)
// gives some row.
template <typename F>
__device__ __forceinline__ int32_t last_row(int32_t rows, int64_t u, F f) {
  int32_t lo = 0, size = rows;
  while (size > 1) {  // at most four times: rows < 2^24
    const int32_t step = (size + kWave - 1) / kWave;
    const int32_t i = lane_id() * step;
    const uint64_t below = __ballot(i < size && f(lo + i) <= u);
    const int32_t k = below ? 63 - __builtin_clzll(below) : 0;
    lo += k * step;
    size = min(step, size - k * step);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// The row of packed entry i and its range; false if no row has it.
__device__ __forceinline__ bool row_of_entry(const Packed& p, int32_t i, int32_t& r, int32_t& begin,
                                             int32_t& end) {
  r = last_row(p.rows, i, [&](int32_t x) { return static_cast<int64_t>(p.at(x)); });
  begin = p.at(r);
  end = p.at(r + 1);
  return i >= begin && i < end;
}

// Units of 2^shift entries each (entries times `times`), where a row whose c entries
// touch at most floor(c * times / 2^shift) + spare units has unit_base(r + 1) -
// unit_base(r) of them, and the rows' units follow one another: no prefix sum is
// needed.
__host__ __device__ __forceinline__ int64_t unit_base(int64_t entries, int32_t times, int32_t shift,
                                                      int32_t r, int32_t spare) {
  return (entries * times >> shift) + static_cast<int64_t>(r) * spare;
}

}  // namespace misa
