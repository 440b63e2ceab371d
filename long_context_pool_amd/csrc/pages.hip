// The paged cache of keys and values: token writes, page bookkeeping (extend,
// fork, free, compact) and page copies.  Layouts are those of misa_cache in
// include/misa.h.  Every id read from device memory (rows, pages, positions)
// is range-checked before it becomes an address.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "quant.hpp"

namespace misa {

namespace {

// ---------------------------------------------------------------- token writes

// One subgroup of LPR lanes per (token, kv head), which writes its K and its V
// (LATENT: K alone): D elements, 8 per lane and step, one 16-byte load each; fp8
// reduces the largest magnitude over the subgroup first.  Both rows' loads are
// under way while three dependent loads find the slot.  Bound by memory
// traffic: 8192 tokens of 8 heads of 128 to fp8 (47 MB) 12.2 us, 3.9 TB/s; 32
// tokens in bf16 3.0 us, a launch and four dependent loads.
template <int D, bool FP8, bool LATENT>
__global__ __launch_bounds__(256) void page_write_kernel(
    uint32_t items, int32_t kv_heads, int32_t rows, int32_t row_pages, int32_t pages, int32_t P,
    const int32_t* __restrict__ row, const int32_t* __restrict__ pos,
    const uint16_t* __restrict__ k_new, const uint16_t* __restrict__ v_new, void* __restrict__ k_pages,
    float* __restrict__ k_scale, void* __restrict__ v_pages, float* __restrict__ v_scale,
    const int32_t* __restrict__ table) {
  constexpr int kChunks = D / 8;
  constexpr int LPR = kChunks >= 64 ? 64 : kChunks;
  constexpr int NV = (kChunks + LPR - 1) / LPR;
  constexpr int KV = LATENT ? 1 : 2;
  const int sub = threadIdx.x % LPR;
  const uint32_t item = blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  if (item >= items) return;  // whole subgroups leave together
  const uint32_t token = item / kv_heads;
  const int32_t head = static_cast<int32_t>(item - token * kv_heads);
  uint4 x[KV][NV];
#pragma unroll
  for (int w = 0; w < KV; ++w) {
    const uint16_t* src = (w ? v_new : k_new) + static_cast<int64_t>(item) * D;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = u * LPR + sub;
      x[w][u] = make_uint4(0, 0, 0, 0);
      if (c < kChunks) x[w][u] = *reinterpret_cast<const uint4*>(src + c * 8);
    }
  }
  const int32_t r = row[token], s = pos[token];
  if (r < 0 || r >= rows || s < 0 || s / P >= row_pages) return;
  const int32_t page = table[static_cast<int64_t>(r) * row_pages + s / P];
  if (page < 0 || page >= pages) return;
  const int64_t slot = (static_cast<int64_t>(page) * kv_heads + head) * P + s % P;
#pragma unroll
  for (int w = 0; w < KV; ++w) {
    void* pool = w ? v_pages : k_pages;
    if constexpr (!FP8) {
      uint16_t* dst = static_cast<uint16_t*>(pool) + slot * D;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const int c = u * LPR + sub;
        if (c < kChunks) *reinterpret_cast<uint4*>(dst + c * 8) = x[w][u];
      }
    } else {
      float y[NV][8], amax = 0.f;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const uint32_t q[4] = {x[w][u].x, x[w][u].y, x[w][u].z, x[w][u].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[u][2 * e] = __uint_as_float(q[e] << 16);
          y[u][2 * e + 1] = __uint_as_float(q[e] & 0xFFFF0000u);
          amax = amax_step(amax_step(amax, y[u][2 * e]), y[u][2 * e + 1]);
        }
      }
      float scale, mult;
      amax = lanes_reduce<LPR, true>(amax);
      e4m3_scale(amax, scale, mult);
      const float rest = e4m3_rest(amax, mult);
      uint8_t* dst = static_cast<uint8_t*>(pool) + slot * D;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const int c = u * LPR + sub;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[u][e] = __builtin_fmaf(y[u][e], mult, y[u][e] * rest);
        if (c < kChunks)
          *reinterpret_cast<uint2*>(dst + c * 8) = make_uint2(e4m3_pack4(y[u][0], y[u][1], y[u][2], y[u][3], 1.f),
                                                              e4m3_pack4(y[u][4], y[u][5], y[u][6], y[u][7], 1.f));
      }
      if (sub == 0) (w ? v_scale : k_scale)[slot] = scale;
    }
  }
}

template <int D, bool LATENT>
hipError_t launch_write(const Cache& c, int32_t n, const int32_t* row, const int32_t* pos,
                        const void* k_new, const void* v_new, void* k_pages, float* k_scale,
                        void* v_pages, float* v_scale, const int32_t* table, hipStream_t st) {
  constexpr int LPR = D / 8 >= 64 ? 64 : D / 8;
  const uint32_t items = n * c.kv_heads;  // at most 2^25: the grid has below 2^32 threads
  const uint32_t blocks = (items - 1) / (256 / LPR) + 1;
  const auto f = c.dtype == kFP8 ? page_write_kernel<D, true, LATENT> : page_write_kernel<D, false, LATENT>;
  f<<<blocks, 256, 0, st>>>(items, c.kv_heads, c.rows, c.row_pages, c.pages, c.P, row, pos,
                            static_cast<const uint16_t*>(k_new), static_cast<const uint16_t*>(v_new),
                            k_pages, k_scale, v_pages, v_scale, table);
  return hipGetLastError();
}

// ---------------------------------------------------------------- page bookkeeping

constexpr int kListThreads = 1024;  // one workgroup plans a list
constexpr int kPerThread = kMaxList / kListThreads;
static_assert(kPerThread * kListThreads == kMaxList, "every entry of the longest list has a thread");
constexpr int32_t kNone = -1;

// Pages a row of `len` tokens holds, and its length as the table can hold it.
__device__ __forceinline__ int32_t held_tokens(int32_t len, int32_t row_pages, int32_t P) {
  return min(max(len, 0), row_pages * P);
}
__device__ __forceinline__ int32_t pages_of(int32_t tokens, int32_t P) {
  return tokens / P + (tokens % P != 0);
}

__device__ __forceinline__ int32_t per_thread(int32_t n) { return (n + kListThreads - 1) / kListThreads; }

// The rows of a list and the first entry that names each, in LDS: open
// addressing over at least twice as many places as entries, so that a search
// ends.  The first entry is a minimum: the order of the threads does not matter.
struct Rows {
  int32_t key[2 * kMaxList];
  int32_t first[2 * kMaxList];
};

__device__ __forceinline__ uint32_t rows_size(int32_t n) {
  uint32_t size = 64;
  while (size < 2u * n) size *= 2;  // at most 2 * kMaxList
  return size;
}

// A barrier must follow.
__device__ __forceinline__ void rows_clear(Rows& h, uint32_t size) {
  for (uint32_t i = threadIdx.x; i < size; i += kListThreads) {
    h.key[i] = kNone;
    h.first[i] = kMaxList;
  }
}

// Enters row r >= 0 of entry i; returns its place.  A barrier must follow
// before first[place] is read.
__device__ __forceinline__ uint32_t rows_enter(Rows& h, uint32_t size, int32_t r, int32_t i) {
  uint32_t at = (static_cast<uint32_t>(r) * 2654435761u >> 16) & (size - 1);
  for (;;) {
    const int32_t old = atomicCAS(&h.key[at], kNone, r);
    if (old == kNone || old == r) break;
    at = (at + 1) & (size - 1);
  }
  atomicMin(&h.first[at], i);
  return at;
}

// Four entries of refs from p on; entries behind the last page count as used.
__device__ __forceinline__ int4 refs_at(const int32_t* refs, int32_t pages, int32_t p) {
  if (p + 4 <= pages) return *reinterpret_cast<const int4*>(refs + p);
  int4 x = make_int4(1, 1, 1, 1);
  if (p < pages) x.x = refs[p];
  if (p + 1 < pages) x.y = refs[p + 1];
  if (p + 2 < pages) x.z = refs[p + 2];
  return x;
}

constexpr int kScanPages = kListThreads * 4;  // pages of a scan's step

// Calls found(rank, page) for the free pages of rank < want, lowest id first,
// and returns how many there are of those (all threads).  `first` is what
// refs_at gives for this thread's first four pages; the next step's are loaded
// ahead.  The scan ends with the step that holds the last one wanted.
template <class F>
__device__ int scan_free(const int32_t* refs, int32_t pages, int32_t want, int4 first, int* tmp, F found) {
  int have = 0;
  int4 next = first;
  for (int32_t c0 = 0; c0 < pages && have < want; c0 += kScanPages) {
    const int32_t p = c0 + static_cast<int32_t>(threadIdx.x) * 4;
    const int4 v = next;
    next = refs_at(refs, pages, p + kScanPages);
    const int32_t x[4] = {v.x, v.y, v.z, v.w};
    int mine = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) mine += x[e] <= 0;
    int total;
    int rank = have + block_exclusive_sum<kListThreads>(mine, tmp, total);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (x[e] <= 0) {
        if (rank < want) found(rank, p + e);
        ++rank;
      }
    have += total;
  }
  return min(have, want);
}

// misa_page_extend: one workgroup.  need[i] pages for entry i, offsets by a
// prefix sum; one scan collects the free pages' ids in LDS, and thread j hands
// out the j-th.  Lists that need more than LDS holds scan again.  Bound by the
// latency of its chain (entries, lengths, refs, tables): 8 rows of a pool of 900
// pages 3.8 us, 128 rows of one of 14000 5.1 us.
__global__ __launch_bounds__(kListThreads) void page_extend_kernel(
    int32_t n, int32_t rows, int32_t row_pages, int32_t pages, int32_t P,
    const int32_t* __restrict__ row, const int32_t* __restrict__ count, int32_t* __restrict__ table,
    int32_t* __restrict__ lengths, int32_t* refs, int32_t* __restrict__ ok) {
  __shared__ Rows seen;
  __shared__ int32_t list[kMaxList];
  __shared__ int32_t offset[kMaxList];  // pages needed by the entries before this one
  __shared__ int32_t held[kMaxList];    // pages of the entry's row before the call
  __shared__ int32_t taken[kMaxList];
  __shared__ int tmp[kListThreads / kWave];
  const int4 first_refs = refs_at(refs, pages, threadIdx.x * 4);
  const int32_t per = per_thread(n);  // thread t has the entries per * t + e, e < per
  const uint32_t places = rows_size(n);
  rows_clear(seen, places);
  int32_t r[kPerThread], more[kPerThread], len[kPerThread];
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    const int i = threadIdx.x * per + e;
    const bool inside = e < per && i < n;
    r[e] = inside ? row[i] : kNone;
    more[e] = inside ? count[i] : -1;
    if (r[e] >= rows) r[e] = kNone;
    if (inside) list[i] = r[e];
  }
  __syncthreads();
  uint32_t place[kPerThread];
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    len[e] = r[e] >= 0 ? lengths[r[e]] : -1;
    place[e] = r[e] >= 0 ? rows_enter(seen, places, r[e], threadIdx.x * per + e) : 0;
  }
  __syncthreads();
  int32_t need[kPerThread];
  bool valid[kPerThread];
  int sum = 0;
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    const int64_t to = static_cast<int64_t>(len[e]) + more[e];
    valid[e] = r[e] >= 0 && seen.first[place[e]] == static_cast<int32_t>(threadIdx.x * per + e) &&
               more[e] >= 0 && len[e] >= 0 && to <= static_cast<int64_t>(row_pages) * P;
    need[e] = valid[e] ? pages_of(static_cast<int32_t>(to), P) - pages_of(len[e], P) : 0;
    sum += need[e];  // at most rows * row_pages over distinct rows: below 2^31
  }
  int total;
  int at = block_exclusive_sum<kListThreads>(sum, tmp, total);
  int32_t first[kPerThread];
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    const int i = threadIdx.x * per + e;
    first[e] = at;
    if (e < per && i < n) {
      offset[i] = at;
      held[i] = valid[e] ? pages_of(len[e], P) : 0;
    }
    at += need[e];
  }
  const int have = scan_free(refs, pages, total, first_refs, tmp, [&](int rank, int32_t page) {
    if (rank < kMaxList) taken[rank] = page;
  });
  __syncthreads();
  auto hand_out = [&](int rank, int32_t page) {
    int lo = 0, hi = n - 1;  // the last entry with offset <= rank
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (offset[mid] <= rank) lo = mid; else hi = mid - 1;
    }
    const int end = lo + 1 < n ? offset[lo + 1] : total;
    if (end > have) return;  // that entry is not served
    table[static_cast<int64_t>(list[lo]) * row_pages + held[lo] + (rank - offset[lo])] = page;
    refs[page] = 1;
  };
  if (total <= kMaxList)
    for (int j = threadIdx.x; j < have; j += kListThreads) hand_out(j, taken[j]);
  else
    scan_free(refs, pages, have, first_refs, tmp, hand_out);
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    const int i = threadIdx.x * per + e;
    if (e >= per || i >= n) continue;
    const bool good = valid[e] && (need[e] == 0 || first[e] + need[e] <= have);
    if (good) lengths[r[e]] = len[e] + more[e];
    ok[i] = good;
  }
}

// Enters the parent's whole pages into a child's table row; this thread's part
// of them is begin, begin + step, ...  refs are integer sums: any order.
__device__ __forceinline__ void share_pages(int32_t* __restrict__ table, int32_t* refs, int64_t from,
                                            int64_t to, int32_t whole, int32_t pages, int begin,
                                            int step) {
  for (int32_t s = begin; s < whole; s += step) {
    const int32_t page = table[from + s];
    table[to + s] = page;
    if (page >= 0 && page < pages) atomicAdd(refs + page, 1);
  }
}

// misa_page_fork, by one workgroup: decide every entry, take the free pages,
// set the children's lengths and last pages.  APPLY: and share the whole pages,
// a wave per entry (short lists; longer ones take a second launch for that).
// A parent of a forked child that is not empty is no child of the call, so its
// row does not change.  Bound by latency like extend: 8 children 6.2 us, sharing
// up to 125 pages each included; 128 children 5.4 us, and 3.3 us for the second
// launch.
template <bool APPLY>
__global__ __launch_bounds__(kListThreads) void page_fork_kernel(
    int32_t n, int32_t rows, int32_t row_pages, int32_t pages, int32_t P,
    const int32_t* __restrict__ parent, const int32_t* __restrict__ child, int32_t* table,
    int32_t* __restrict__ lengths, int32_t* refs, int32_t* __restrict__ src,
    int32_t* __restrict__ dst, int32_t* __restrict__ ok) {
  __shared__ Rows seen;
  __shared__ int32_t taken[kMaxList];
  __shared__ int32_t whole[APPLY ? kMaxList : 1];   // pages to share
  __shared__ int32_t source[APPLY ? kMaxList : 1];  // the parents
  __shared__ int32_t target[APPLY ? kMaxList : 1];  // the children
  __shared__ int tmp[kListThreads / kWave];
  const int4 first_refs = refs_at(refs, pages, threadIdx.x * 4);
  const int32_t per = per_thread(n);  // thread t has the entries per * t + e, e < per
  const uint32_t places = rows_size(n);
  rows_clear(seen, places);
  int32_t p[kPerThread], c[kPerThread], len[kPerThread], from[kPerThread];
  bool valid[kPerThread];
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    const int i = threadIdx.x * per + e;
    const bool inside = e < per && i < n;
    p[e] = inside ? parent[i] : kNone;
    c[e] = inside ? child[i] : kNone;
    if (APPLY && inside) {
      source[i] = p[e];
      target[i] = c[e];
    }
  }
  __syncthreads();
  uint32_t place[kPerThread];
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    const bool named = c[e] >= 0 && c[e] < rows;
    place[e] = named ? rows_enter(seen, places, c[e], threadIdx.x * per + e) : 0;
    valid[e] = named && p[e] >= 0 && p[e] < rows && c[e] != p[e];
    len[e] = valid[e] ? held_tokens(lengths[p[e]], row_pages, P) : 0;
    if (valid[e]) valid[e] = lengths[c[e]] == 0;
    from[e] = kNone;
    if (valid[e] && len[e] % P != 0) {
      const int32_t last = table[static_cast<int64_t>(p[e]) * row_pages + len[e] / P];
      if (last >= 0 && last < pages) from[e] = last;
    }
  }
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    valid[e] = valid[e] && seen.first[place[e]] == static_cast<int32_t>(threadIdx.x * per + e);
    if (!valid[e]) from[e] = kNone;
    sum += from[e] != kNone;
  }
  int total;
  int at = block_exclusive_sum<kListThreads>(sum, tmp, total);
  const int have = scan_free(refs, pages, total, first_refs, tmp, [&](int rank, int32_t page) { taken[rank] = page; });
  __syncthreads();  // every read of refs and lengths, and taken's writes, before
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    const int i = threadIdx.x * per + e;
    if (e >= per || i >= n) continue;
    const bool part = from[e] != kNone;
    const bool good = valid[e] && (!part || at < have);
    const int32_t page = part && good ? taken[at] : kNone;
    if (page != kNone) refs[page] = 1;
    src[i] = page != kNone ? from[e] : kNone;
    dst[i] = page;
    ok[i] = good;
    if (APPLY) whole[i] = good ? len[e] / P : 0;
    if (good) {
      lengths[c[e]] = len[e];
      if (len[e] % P != 0) table[static_cast<int64_t>(c[e]) * row_pages + len[e] / P] = page;
    }
    at += part;
  }
  if constexpr (APPLY) {
    __syncthreads();
    for (int i = threadIdx.x / kWave; i < n; i += kListThreads / kWave)
      if (whole[i] > 0)
        share_pages(table, refs, static_cast<int64_t>(source[i]) * row_pages,
                    static_cast<int64_t>(target[i]) * row_pages, whole[i], pages, lane_id(), kWave);
  }
}

// misa_page_fork, second launch of long lists: workgroup (x, i) shares a part
// of the pages of entry i.
__global__ __launch_bounds__(256) void page_share_kernel(int32_t row_pages, int32_t pages, int32_t P,
                                                         const int32_t* __restrict__ parent,
                                                         const int32_t* __restrict__ child,
                                                         int32_t* __restrict__ table,
                                                         const int32_t* __restrict__ lengths,
                                                         int32_t* refs, const int32_t* __restrict__ ok) {
  const int i = blockIdx.y;
  if (!ok[i]) return;
  const int32_t c = child[i];
  share_pages(table, refs, static_cast<int64_t>(parent[i]) * row_pages,
              static_cast<int64_t>(c) * row_pages, lengths[c] / P, pages,
              blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
}

// misa_page_free: workgroup i clears the row of entry i, unless an earlier one
// names it.  8 or 128 rows of up to 128 pages: 3.5 us, a launch and three dependent
// loads.
__global__ __launch_bounds__(256) void page_free_kernel(int32_t rows, int32_t row_pages,
                                                        int32_t pages, int32_t P,
                                                        const int32_t* __restrict__ row,
                                                        int32_t* __restrict__ table,
                                                        int32_t* __restrict__ lengths,
                                                        int32_t* __restrict__ refs) {
  const int i = blockIdx.x;
  const int32_t r = row[i];
  if (r < 0 || r >= rows) return;
  bool before = false;
  for (int j = threadIdx.x; j < i; j += 256) before |= row[j] == r;
  if (__syncthreads_or(before)) return;
  const int32_t held = pages_of(held_tokens(lengths[r], row_pages, P), P);
  const int64_t at = static_cast<int64_t>(r) * row_pages;
#pragma unroll 4
  for (int32_t s = threadIdx.x; s < held; s += 256) {
    const int32_t page = table[at + s];
    table[at + s] = kNone;
    if (page >= 0 && page < pages) atomicSub(refs + page, 1);
  }
  __syncthreads();  // every thread has read the length
  if (threadIdx.x == 0) lengths[r] = 0;
}

// Workgroups per table row: four entries a thread, at most 64 (the kernels loop).
int32_t row_blocks(const Cache& c) {
  const int32_t blocks = (c.row_pages - 1) / 1024 + 1;
  return blocks < 64 ? blocks : 64;
}

// ---------------------------------------------------------------- compaction

constexpr int kCountPages = 1024;  // pages per workgroup: four per thread
// Up to so many, that every workgroup counts all pages is cheaper than a launch
// that counts them once (with the copies: 2500 pages 13.8 us against 16.2, 6000
// pages 15.4 against 16.7; 20000 pages would take 1.0 us more).
constexpr int kOwnChunks = 8;
constexpr int kSmallPages = 2048;  // pages and table entries of a compaction by one workgroup

__device__ __forceinline__ int used4(int4 x) { return (x.x > 0) + (x.y > 0) + (x.z > 0) + (x.w > 0); }

// refs_at, with entries behind the last page free.
__device__ __forceinline__ int4 refs_or_free(const int32_t* refs, int32_t pages, int32_t p) {
  if (p + 4 <= pages) return *reinterpret_cast<const int4*>(refs + p);
  int4 x = make_int4(0, 0, 0, 0);
  if (p < pages) x.x = refs[p];
  if (p + 1 < pages) x.y = refs[p + 1];
  if (p + 2 < pages) x.z = refs[p + 2];
  return x;
}

__global__ __launch_bounds__(256) void page_count_kernel(int32_t pages,
                                                         const int32_t* __restrict__ refs,
                                                         int32_t* __restrict__ counts) {
  __shared__ int tmp[4];
  int total;
  block_exclusive_sum<256>(used4(refs_or_free(refs, pages, blockIdx.x * kCountPages + threadIdx.x * 4)), tmp, total);
  if (threadIdx.x == 0) counts[blockIdx.x] = total;
}

// What becomes of four pages from p on, of which `x` are the refs: `rank` live
// pages lie before them, `live` in all, `stay` of them below `live`.  Holes and
// movers get their ranks; a mover's map entry holds -2 - rank until the tables
// are done.
__device__ __forceinline__ void place4(int4 x, int32_t p, int32_t pages, int rank, int live, int stay,
                                       int32_t* __restrict__ map, int32_t* __restrict__ src,
                                       int32_t* __restrict__ dst) {
  const int32_t v[4] = {x.x, x.y, x.z, x.w};
  const int holes = live - stay;
#pragma unroll
  for (int e = 0; e < 4; ++e, ++p) {
    if (p >= pages) break;
    const bool used = v[e] > 0;
    if (used && p >= live) {
      src[rank - stay] = p;
      map[p] = -2 - (rank - stay);
    } else {
      map[p] = used ? p : kNone;
      if (!used && p < live) dst[p - rank] = p;
    }
    if (p < max(1, pages / 2) && p >= holes) {
      src[p] = kNone;
      dst[p] = kNone;
    }
    rank += used;
  }
}

// Live pages of a wave's 256 pages of a chunk.
__device__ __forceinline__ int wave_used(int4 x) {
  return __popcll(__ballot(x.x > 0)) + __popcll(__ballot(x.y > 0)) + __popcll(__ballot(x.z > 0)) +
         __popcll(__ballot(x.w > 0));
}

// Second launch: ranks by prefix sums over the counts and a workgroup's pages.
// OWN: the first one; every workgroup counts the whole pool by itself, a count per
// chunk and wave.
template <bool OWN>
__global__ __launch_bounds__(256) void page_place_kernel(int32_t pages, int32_t chunks,
                                                         const int32_t* __restrict__ refs,
                                                         const int32_t* __restrict__ counts_in,
                                                         int32_t* __restrict__ map,
                                                         int32_t* __restrict__ live_out,
                                                         int32_t* __restrict__ src,
                                                         int32_t* __restrict__ dst) {
  constexpr int kEach = OWN ? 4 : 1;  // counts of a chunk
  __shared__ int tmp[4];
  __shared__ int own[OWN ? kOwnChunks * 4 : 1];
  const int32_t p = blockIdx.x * kCountPages + threadIdx.x * 4;
  const int4 x = refs_or_free(refs, pages, p);
  if constexpr (OWN) {
    const int wave = threadIdx.x / kWave, whole = pages / kCountPages;
    const int4* from = reinterpret_cast<const int4*>(refs) + threadIdx.x;
#pragma unroll 8
    for (int b = 0; b < whole; ++b) {
      const int n = wave_used(from[b * 256]);
      if (lane_id() == 0) own[4 * b + wave] = n;
    }
    if (whole < chunks) {
      const int n = wave_used(refs_or_free(refs, pages, whole * kCountPages + threadIdx.x * 4));
      if (lane_id() == 0) own[4 * whole + wave] = n;
    }
    __syncthreads();
  }
  const int32_t* counts = OWN ? own : counts_in;
  int all = 0, lower = 0;
  for (int b = threadIdx.x; b < chunks * kEach; b += 256) {
    const int c = counts[b];
    all += c;
    lower += b / kEach < static_cast<int>(blockIdx.x) ? c : 0;
  }
  int live, before, stay, total;
  block_exclusive_sum<256>(all, tmp, live);
  // Live pages below `live`: whole chunks, and the part of the one it is in.
  const int32_t edge = live / kCountPages;
  const int32_t q = edge * kCountPages + threadIdx.x * 4;
  const int4 y = q < pages ? refs_or_free(refs, pages, q) : make_int4(0, 0, 0, 0);
  int mine = 0;
  for (int b = threadIdx.x; b < edge * kEach; b += 256) mine += counts[b];
  mine += (y.x > 0 && q < live) + (y.y > 0 && q + 1 < live) + (y.z > 0 && q + 2 < live) +
          (y.w > 0 && q + 3 < live);
  block_exclusive_sum<256>(lower, tmp, before);
  block_exclusive_sum<256>(mine, tmp, stay);
  const int rank = before + block_exclusive_sum<256>(used4(x), tmp, total);
  place4(x, p, pages, rank, live, stay, map, src, dst);
  if (p == 0) live_out[0] = live;
}

// A table entry's page afterwards, from the map as place4 leaves it.  The map's entry
// is loaded once (an atomic load of a wave's scope is an ordinary one): another
// thread may resolve it meanwhile.
__device__ __forceinline__ int32_t moved_page(int32_t id, int32_t pages, const int32_t* map, const int32_t* dst) {
  if (id < 0 || id >= pages) return kNone;
  const int32_t to = __hip_atomic_load(map + id, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
  return to < kNone ? dst[-2 - to] : to;
}

// Small pools and tables: everything in one workgroup and one launch (1000 pages
// 4.7 us; the launches of larger pools take about that each, by latency).
__global__ __launch_bounds__(kListThreads) void page_compact_small_kernel(
    int32_t pages, int32_t entries, const int32_t* table, const int32_t* refs, int32_t* table_out,
    int32_t* refs_out, int32_t* map, int32_t* __restrict__ live_out, int32_t* src, int32_t* dst) {
  __shared__ int tmp[kListThreads / kWave];
  const int32_t p = threadIdx.x * 4;
  const int4 x = refs_or_free(refs, pages, p);
  int live, stay;
  const int rank = block_exclusive_sum<kListThreads>(used4(x), tmp, live);
  block_exclusive_sum<kListThreads>((x.x > 0 && p < live) + (x.y > 0 && p + 1 < live) +
                                        (x.z > 0 && p + 2 < live) + (x.w > 0 && p + 3 < live),
                                    tmp, stay);
  place4(x, p, pages, rank, live, stay, map, src, dst);
  if (p == 0) live_out[0] = live;
  __syncthreads();
  const int32_t v[4] = {x.x, x.y, x.z, x.w};
  for (int i = threadIdx.x; i < entries; i += kListThreads) table_out[i] = moved_page(table[i], pages, map, dst);
  int32_t to[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) to[e] = p + e < pages ? moved_page(p + e, pages, map, dst) : kNone;
  __syncthreads();  // every read of map before
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (p + e < pages) {
      map[p + e] = to[e];
      if (to[e] != kNone) refs_out[to[e]] = v[e];
      if (p + e >= live) refs_out[p + e] = 0;
    }
}

// Last launch: the movers' map entries, refs and the tables, which may be the same
// arrays before and after.  Threads that meet an entry of `map` before or after it
// is resolved find the same page.
__global__ __launch_bounds__(256) void page_finish_kernel(
    int32_t pages, int64_t entries, const int32_t* table, const int32_t* refs,
    int32_t* table_out, int32_t* refs_out, int32_t* map,
    const int32_t* __restrict__ live_out, const int32_t* __restrict__ src,
    const int32_t* __restrict__ dst) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int32_t live = live_out[0];
  if (i < pages / 2 && src[i] != kNone) {
    const int32_t s = src[i], d = dst[i];
    refs_out[d] = refs[s];
    refs_out[s] = 0;
    map[s] = d;
  }
  if (i < pages) {
    const int32_t x = refs[i];
    if (i < live) {
      if (map[i] == i) refs_out[i] = x;  // the holes belong to their movers' threads
    } else if (map[i] == kNone) {
      refs_out[i] = 0;
    }
  }
  if (i < entries) {
    table_out[i] = moved_page(table[i], pages, map, dst);
  }
}

// ---------------------------------------------------------------- copies

constexpr int kCopyBytes = 32768;  // bytes of a page in a piece
// Pages up to this size have a wave each, larger ones a workgroup per piece (a
// pool of 20000 pages compacted, pages of 1 KB: 18.0 us so, 29.0 us with
// workgroups; of 4 KB 28.2 and 32.0; of 8 KB 43.8 and 42.3.  A pool of 1000 pages
// of 8 KB: 13.8 and 11.2 us).
constexpr int64_t kWavePage = 4096;

struct CopyPlan {
  PageBuffers bufs;
  int64_t first[kMaxPageBuffers];  // first piece of each buffer
  int32_t parts[kMaxPageBuffers];  // pieces per page
};

// N dwords per thread and step, T threads on a piece, marked as not to be kept:
// pages go by once.  Four steps' loads are under way before the first store, which
// might otherwise be to what the next load reads (20000 pages of 32 KB, four
// planes, 1.3 GB: 230 us with the bookkeeping; 243 us with one load at a time, 261
// us with plain loads and stores, 274 us of those in pieces of 16 KB).
template <int T, int N>
__device__ __forceinline__ void copy_run(uint8_t* to, const uint8_t* from, int64_t bytes) {
  typedef __attribute__((ext_vector_type(N))) uint32_t V;
  constexpr int kStep = T * N * 4, kBatch = 4;
  int64_t o = threadIdx.x % T * (N * 4);
  for (; o + (kBatch - 1) * kStep < bytes; o += kBatch * kStep) {
    V x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      x[i] = __builtin_nontemporal_load(reinterpret_cast<const V*>(from + o + i * kStep));
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      __builtin_nontemporal_store(x[i], reinterpret_cast<V*>(to + o + i * kStep));
  }
  for (; o < bytes; o += kStep)
    __builtin_nontemporal_store(__builtin_nontemporal_load(reinterpret_cast<const V*>(from + o)),
                                reinterpret_cast<V*>(to + o));
}

// Piece `w` of the work over (buffer, pair, plane, part of the page).
template <int T>
__device__ __forceinline__ void copy_piece(const CopyPlan& plan, int64_t w, int32_t pages,
                                           const int32_t* __restrict__ src,
                                           const int32_t* __restrict__ dst) {
  int b = 0;
  while (b + 1 < plan.bufs.n && w >= plan.first[b + 1]) ++b;
  const PageBuffer buf = plan.bufs.b[b];
  w -= plan.first[b];
  const int32_t part = static_cast<int32_t>(w % plan.parts[b]);
  w /= plan.parts[b];
  const int32_t plane = static_cast<int32_t>(w % buf.planes);
  const int64_t pair = w / buf.planes;
  const int32_t s = src[pair], d = dst[pair];
  if (s < 0 || s >= pages || d < 0 || d >= pages || s == d) return;
  const int64_t at = static_cast<int64_t>(part) * kCopyBytes;
  const int64_t bytes = min<int64_t>(kCopyBytes, buf.page_bytes - at);
  uint8_t* base = buf.data + static_cast<int64_t>(plane) * pages * buf.page_bytes + at;
  uint8_t* to = base + d * buf.page_bytes;
  const uint8_t* from = base + s * buf.page_bytes;
  if (buf.page_bytes % 16 == 0)
    copy_run<T, 4>(to, from, bytes);
  else
    copy_run<T, 1>(to, from, bytes);
}

// A workgroup (T = 256) or a wave of it (T = 64) per piece.
template <int T>
__global__ __launch_bounds__(256) void page_copy_kernel(CopyPlan plan, int64_t pieces, int32_t pages,
                                                        const int32_t* __restrict__ src,
                                                        const int32_t* __restrict__ dst) {
  constexpr int kPieces = 256 / T;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / T);
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * kPieces + wave; w < pieces; w += static_cast<int64_t>(gridDim.x) * kPieces)
    copy_piece<T>(plan, w, pages, src, dst);
}

int32_t copy_parts(const PageBuffer& b) {
  return static_cast<int32_t>((b.page_bytes + kCopyBytes - 1) / kCopyBytes);
}

int64_t copy_blocks(const PageBuffer& b, int32_t n) {
  return static_cast<int64_t>(copy_parts(b)) * b.planes * n;
}

}  // namespace

hipError_t launch_page_write(const Cache& c, int32_t n, const int32_t* row, const int32_t* pos,
                             const void* k_new, const void* v_new, void* k_pages, float* k_scale,
                             void* v_pages, float* v_scale, const int32_t* table, hipStream_t st) {
  switch (c.dk) {
    case 64:
      return launch_write<64, false>(c, n, row, pos, k_new, v_new, k_pages, k_scale, v_pages, v_scale,
                              table, st);
    case 128:
      return launch_write<128, false>(c, n, row, pos, k_new, v_new, k_pages, k_scale, v_pages, v_scale,
                               table, st);
    case 256:
      return launch_write<256, false>(c, n, row, pos, k_new, v_new, k_pages, k_scale, v_pages, v_scale,
                               table, st);
    default:
      return launch_write<576, true>(c, n, row, pos, k_new, v_new, k_pages, k_scale, v_pages, v_scale,
                               table, st);
  }
}

hipError_t launch_page_extend(const Cache& c, int32_t n, const int32_t* row, const int32_t* count,
                              int32_t* table, int32_t* lengths, int32_t* refs, int32_t* ok,
                              hipStream_t st) {
  page_extend_kernel<<<1, kListThreads, 0, st>>>(n, c.rows, c.row_pages, c.pages, c.P, row, count,
                                                 table, lengths, refs, ok);
  return hipGetLastError();
}

hipError_t launch_page_fork(const Cache& c, int32_t n, const int32_t* parent, const int32_t* child,
                            int32_t* table, int32_t* lengths, int32_t* refs, int32_t* src,
                            int32_t* dst, int32_t* ok, hipStream_t st) {
  // Up to 2048 table entries one workgroup shares the pages too; beyond, a second
  // launch spreads them over the card.  A step of free, fork, copy and extend
  // with 8 children of 125 pages takes 21.4 us so, 24.1 us with two launches;
  // with 60 children of 128 pages it would take 37.1 us, against 29.8 us.
  const bool small = static_cast<int64_t>(n) * c.row_pages <= 2048;
  const auto f = small ? page_fork_kernel<true> : page_fork_kernel<false>;
  f<<<1, kListThreads, 0, st>>>(n, c.rows, c.row_pages, c.pages, c.P, parent, child, table, lengths,
                                refs, src, dst, ok);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || small) return e;
  page_share_kernel<<<dim3(row_blocks(c), n), 256, 0, st>>>(c.row_pages, c.pages, c.P, parent, child,
                                                            table, lengths, refs, ok);
  return hipGetLastError();
}

hipError_t launch_page_free(const Cache& c, int32_t n, const int32_t* row, int32_t* table,
                            int32_t* lengths, int32_t* refs, hipStream_t st) {
  page_free_kernel<<<n, 256, 0, st>>>(c.rows, c.row_pages, c.pages, c.P, row, table, lengths, refs);
  return hipGetLastError();
}

size_t page_compact_ws_bytes(const Cache& c) {
  return align_up((static_cast<size_t>(c.pages) + kCountPages - 1) / kCountPages * sizeof(int32_t));
}

hipError_t launch_page_compact(const Cache& c, const int32_t* table, const int32_t* refs,
                               int32_t* table_out, int32_t* refs_out, int32_t* map, int32_t* live,
                               int32_t* src, int32_t* dst, void* ws, hipStream_t st) {
  const int64_t entries = static_cast<int64_t>(c.rows) * c.row_pages;
  // Small pools and tables in one workgroup: with its copies, a pool of 1000
  // pages takes 12.2 us so, 15.1 us in two launches; one of 4000 pages with
  // 3000 table entries would take 24.2 us, against 22.5 us.
  static_assert(kSmallPages <= kScanPages, "four pages a thread");
  if (c.pages <= kSmallPages && entries <= kSmallPages) {
    page_compact_small_kernel<<<1, kListThreads, 0, st>>>(c.pages, static_cast<int32_t>(entries), table,
                                                          refs, table_out, refs_out, map, live, src, dst);
    return hipGetLastError();
  }
  const int32_t chunks = (c.pages + kCountPages - 1) / kCountPages;
  auto* counts = static_cast<int32_t*>(ws);
  hipError_t e;
  if (chunks <= kOwnChunks) {
    page_place_kernel<true><<<chunks, 256, 0, st>>>(c.pages, chunks, refs, counts, map, live, src, dst);
  } else {
    page_count_kernel<<<chunks, 256, 0, st>>>(c.pages, refs, counts);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    page_place_kernel<false><<<chunks, 256, 0, st>>>(c.pages, chunks, refs, counts, map, live, src, dst);
  }
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t most = entries > c.pages ? entries : c.pages;
  page_finish_kernel<<<static_cast<uint32_t>((most + 255) / 256), 256, 0, st>>>(
      c.pages, entries, table, refs, table_out, refs_out, map, live, src, dst);
  return hipGetLastError();
}

bool page_copy_supported(const PageBuffers& b, int32_t n) {
  for (int32_t i = 0; i < b.n; ++i)
    if (copy_blocks(b.b[i], n) >= (int64_t{1} << 40)) return false;
  return true;
}

hipError_t launch_page_copy(const PageBuffers& b, int32_t pages, int32_t n, const int32_t* src,
                            const int32_t* dst, hipStream_t st) {
  CopyPlan plan{};
  plan.bufs = b;
  int64_t pieces = 0;
  for (int32_t i = 0; i < b.n; ++i) {
    plan.first[i] = pieces;
    plan.parts[i] = copy_parts(b.b[i]);
    pieces += copy_blocks(b.b[i], n);
  }
  int64_t largest = 0;
  for (int32_t i = 0; i < b.n; ++i) largest = std::max(largest, b.b[i].page_bytes);
  // A grid's threads stay below 2^32: workgroups beyond 65536 loop.
  const bool waves = largest <= kWavePage;
  const int64_t blocks = waves ? (pieces + 3) / 4 : pieces;
  const uint32_t grid = static_cast<uint32_t>(std::min<int64_t>(blocks, 65536));
  const auto f = waves ? page_copy_kernel<kWave> : page_copy_kernel<256>;
  f<<<grid, 256, 0, st>>>(plan, pieces, pages, src, dst);
  return hipGetLastError();
}

}  // namespace misa
