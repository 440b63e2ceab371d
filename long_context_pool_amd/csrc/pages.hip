// The paged cache of keys and values: token writes, page bookkeeping (extend,
// fork, free, compact) and page copies.  Layouts are those of misa_cache in
// include/misa.h.  Every id read from device memory (rows, pages, positions)
// is range-checked before it becomes an address.
#include "common.hpp"
#include "launch.hpp"
#include "quant.hpp"

namespace misa {

namespace {

// ---------------------------------------------------------------- token writes

// One subgroup of LPR lanes per (token, kv head, K or V): D elements, 8 per
// lane and step, one 16-byte load each; fp8 reduces the largest magnitude over
// the subgroup first.  Bound by memory traffic.
template <int D, bool FP8>
__global__ __launch_bounds__(256) void page_write_kernel(
    int64_t items, int32_t per_token, int32_t kv_heads, int32_t rows, int32_t row_pages,
    int32_t pages, int32_t P, const int32_t* __restrict__ row, const int32_t* __restrict__ pos,
    const uint16_t* __restrict__ k_new, const uint16_t* __restrict__ v_new, void* __restrict__ k_pages,
    float* __restrict__ k_scale, void* __restrict__ v_pages, float* __restrict__ v_scale,
    const int32_t* __restrict__ table) {
  constexpr int kChunks = D / 8;
  constexpr int LPR = kChunks >= 64 ? 64 : kChunks;
  constexpr int NV = (kChunks + LPR - 1) / LPR;
  const int sub = threadIdx.x % LPR;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (256 / LPR) + threadIdx.x / LPR;
  if (item >= items) return;  // whole subgroups leave together
  const int64_t token = item / per_token;
  const int32_t which = static_cast<int32_t>(item - token * per_token);
  const bool is_v = which >= kv_heads;
  const int32_t head = is_v ? which - kv_heads : which;
  const int32_t r = row[token], s = pos[token];
  if (r < 0 || r >= rows || s < 0 || s / P >= row_pages) return;
  const int32_t page = table[static_cast<int64_t>(r) * row_pages + s / P];
  if (page < 0 || page >= pages) return;
  const uint16_t* src = (is_v ? v_new : k_new) + (token * kv_heads + head) * D;
  const int64_t slot = (static_cast<int64_t>(page) * kv_heads + head) * P + s % P;
  uint4 x[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int c = u * LPR + sub;
    x[u] = make_uint4(0, 0, 0, 0);
    if (c < kChunks) x[u] = *reinterpret_cast<const uint4*>(src + c * 8);
  }
  if constexpr (!FP8) {
    uint16_t* dst = static_cast<uint16_t*>(is_v ? v_pages : k_pages) + slot * D;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = u * LPR + sub;
      if (c < kChunks) *reinterpret_cast<uint4*>(dst + c * 8) = x[u];
    }
  } else {
    float amax = 0.f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        amax = amax_step(amax, __uint_as_float(w[e] << 16));
        amax = amax_step(amax, __uint_as_float(w[e] & 0xFFFF0000u));
      }
    }
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o, kWave));
    float scale, mult;
    e4m3_scale(amax, scale, mult);
    uint8_t* dst = static_cast<uint8_t*>(is_v ? v_pages : k_pages) + slot * D;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = u * LPR + sub;
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      uint2 code;
      code.x = e4m3_pack4(__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u),
                          __uint_as_float(w[1] << 16), __uint_as_float(w[1] & 0xFFFF0000u), mult);
      code.y = e4m3_pack4(__uint_as_float(w[2] << 16), __uint_as_float(w[2] & 0xFFFF0000u),
                          __uint_as_float(w[3] << 16), __uint_as_float(w[3] & 0xFFFF0000u), mult);
      if (c < kChunks) *reinterpret_cast<uint2*>(dst + c * 8) = code;
    }
    if (sub == 0) (is_v ? v_scale : k_scale)[slot] = scale;
  }
}

template <int D>
hipError_t launch_write(const Cache& c, int32_t n, const int32_t* row, const int32_t* pos,
                        const void* k_new, const void* v_new, void* k_pages, float* k_scale,
                        void* v_pages, float* v_scale, const int32_t* table, hipStream_t st) {
  constexpr int LPR = D / 8 >= 64 ? 64 : D / 8;
  const int32_t per_token = c.kv_heads * (c.latent() ? 1 : 2);
  const int64_t items = static_cast<int64_t>(n) * per_token;
  const int64_t blocks = (items + 256 / LPR - 1) / (256 / LPR);
  const auto* kn = static_cast<const uint16_t*>(k_new);
  const auto* vn = static_cast<const uint16_t*>(v_new);
  if (c.dtype == kFP8)
    page_write_kernel<D, true><<<static_cast<uint32_t>(blocks), 256, 0, st>>>(
        items, per_token, c.kv_heads, c.rows, c.row_pages, c.pages, c.P, row, pos, kn, vn, k_pages,
        k_scale, v_pages, v_scale, table);
  else
    page_write_kernel<D, false><<<static_cast<uint32_t>(blocks), 256, 0, st>>>(
        items, per_token, c.kv_heads, c.rows, c.row_pages, c.pages, c.P, row, pos, kn, vn, k_pages,
        k_scale, v_pages, v_scale, table);
  return hipGetLastError();
}

// ---------------------------------------------------------------- page bookkeeping

constexpr int kListThreads = 1024;  // one workgroup plans a list
constexpr int kMaxEntries = 4096;   // entries of a list; 4 per thread
constexpr int kPerThread = kMaxEntries / kListThreads;
constexpr int32_t kNone = -1;

// Pages a row of `len` tokens holds, and its length as the table can hold it.
__device__ __forceinline__ int32_t held_tokens(int32_t len, int32_t row_pages, int32_t P) {
  return min(max(len, 0), row_pages * P);
}
__device__ __forceinline__ int32_t pages_of(int32_t tokens, int32_t P) {
  return tokens / P + (tokens % P != 0);
}

// Whether an earlier entry of the list in LDS names the same row.
__device__ __forceinline__ bool listed_before(const int32_t* list, int i) {
  const int32_t r = list[i];
  bool hit = false;
  int j = 0;
  for (; j + 4 <= i; j += 4) {
    const int4 x = *reinterpret_cast<const int4*>(list + j);
    hit |= x.x == r || x.y == r || x.z == r || x.w == r;
  }
  for (; j < i; ++j) hit |= list[j] == r;
  return hit;
}

// Calls found(rank, page) for the free pages of rank < want, lowest id first,
// and returns how many there are of those (all threads).  The scan ends with
// the chunk that holds the last one wanted.
template <class F>
__device__ int scan_free(const int32_t* refs, int32_t pages, int32_t want, int* tmp,
                         F found) {
  constexpr int kChunk = kListThreads * 4;
  int have = 0;
  for (int32_t c0 = 0; c0 < pages && have < want; c0 += kChunk) {
    const int32_t p = c0 + static_cast<int32_t>(threadIdx.x) * 4;
    int32_t x[4] = {1, 1, 1, 1};
    if (p + 4 <= pages) {
      const int4 v = *reinterpret_cast<const int4*>(refs + p);
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (p + e < pages) x[e] = refs[p + e];
    }
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
// prefix sum, the free pages counted, then handed out by rank.
__global__ __launch_bounds__(kListThreads) void page_extend_kernel(
    int32_t n, int32_t rows, int32_t row_pages, int32_t pages, int32_t P,
    const int32_t* __restrict__ row, const int32_t* __restrict__ count, int32_t* __restrict__ table,
    int32_t* __restrict__ lengths, int32_t* __restrict__ refs, int32_t* __restrict__ ok) {
  __shared__ __attribute__((aligned(16))) int32_t list[kMaxEntries];
  __shared__ int32_t offset[kMaxEntries];  // pages needed by the entries before this one
  __shared__ int tmp[kListThreads / kWave];
  for (int i = threadIdx.x; i < n; i += kListThreads) list[i] = row[i];
  __syncthreads();
  int32_t len[kPerThread], need[kPerThread];
  bool valid[kPerThread];
  int sum = 0;
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    const int i = threadIdx.x * kPerThread + e;
    valid[e] = false;
    need[e] = 0;
    len[e] = 0;
    if (i < n) {
      const int32_t r = list[i], more = count[i];
      if (r >= 0 && r < rows && more >= 0 && !listed_before(list, i)) {
        len[e] = lengths[r];
        const int64_t to = static_cast<int64_t>(len[e]) + more;
        if (len[e] >= 0 && to <= static_cast<int64_t>(row_pages) * P) {
          valid[e] = true;
          need[e] = pages_of(static_cast<int32_t>(to), P) - pages_of(len[e], P);
        }
      }
    }
    // At most rows * row_pages pages over distinct rows: below 2^31.
    sum += need[e];
  }
  int total;
  int at = block_exclusive_sum<kListThreads>(sum, tmp, total);
  int32_t first[kPerThread];
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    first[e] = at;
    if (threadIdx.x * kPerThread + e < n) offset[threadIdx.x * kPerThread + e] = at;
    at += need[e];
  }
  __syncthreads();
  const int have = scan_free(refs, pages, total, tmp, [](int, int32_t) {});
  // The last entry whose pages are all there ends at `served`: ranks below it
  // are handed out.
  scan_free(refs, pages, have, tmp, [&](int rank, int32_t page) {
    int lo = 0, hi = n - 1;  // the last entry with offset <= rank
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (offset[mid] <= rank) lo = mid; else hi = mid - 1;
    }
    const int end = lo + 1 < n ? offset[lo + 1] : total;
    if (end > have) return;  // that entry is not served
    const int32_t r = list[lo];
    const int32_t at_page = pages_of(lengths[r], P) + (rank - offset[lo]);
    table[static_cast<int64_t>(r) * row_pages + at_page] = page;
    refs[page] = 1;
  });
  __syncthreads();  // the table entries above were placed by the old lengths
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    const int i = threadIdx.x * kPerThread + e;
    if (i >= n) continue;
    const bool good = valid[e] && (need[e] == 0 || first[e] + need[e] <= have);
    if (good) lengths[list[i]] = len[e] + count[i];
    ok[i] = good;
  }
}

// misa_page_fork, first launch: decide every entry, take the free pages, set
// the children's lengths.
__global__ __launch_bounds__(kListThreads) void page_fork_plan_kernel(
    int32_t n, int32_t rows, int32_t row_pages, int32_t pages, int32_t P,
    const int32_t* __restrict__ parent, const int32_t* __restrict__ child,
    const int32_t* __restrict__ table, int32_t* __restrict__ lengths, int32_t* __restrict__ refs,
    int32_t* __restrict__ src, int32_t* __restrict__ dst, int32_t* __restrict__ ok) {
  __shared__ __attribute__((aligned(16))) int32_t list[kMaxEntries];
  __shared__ int32_t taken[kMaxEntries];
  __shared__ int tmp[kListThreads / kWave];
  for (int i = threadIdx.x; i < n; i += kListThreads) list[i] = child[i];
  __syncthreads();
  int32_t len[kPerThread], from[kPerThread];
  bool valid[kPerThread];
  int sum = 0;
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    const int i = threadIdx.x * kPerThread + e;
    valid[e] = false;
    len[e] = 0;
    from[e] = kNone;
    if (i < n) {
      const int32_t c = list[i], p = parent[i];
      if (c >= 0 && c < rows && p >= 0 && p < rows && p != c && lengths[c] == 0 &&
          !listed_before(list, i)) {
        valid[e] = true;
        len[e] = held_tokens(lengths[p], row_pages, P);
        if (len[e] % P != 0) {
          const int32_t last = table[static_cast<int64_t>(p) * row_pages + len[e] / P];
          if (last >= 0 && last < pages) from[e] = last;
        }
      }
    }
    sum += from[e] != kNone;
  }
  int total;
  int at = block_exclusive_sum<kListThreads>(sum, tmp, total);
  const int have = scan_free(refs, pages, total, tmp, [&](int rank, int32_t page) { taken[rank] = page; });
  __syncthreads();  // every read of refs, lengths and taken's writes before
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    const int i = threadIdx.x * kPerThread + e;
    if (i >= n) continue;
    const bool part = from[e] != kNone;
    const bool good = valid[e] && (!part || at < have);
    const int32_t page = part && good ? taken[at] : kNone;
    if (page != kNone) refs[page] = 1;
    src[i] = page != kNone ? from[e] : kNone;
    dst[i] = page;
    ok[i] = good;
    if (good) lengths[list[i]] = len[e];
    at += part;
  }
}

// misa_page_fork, second launch: workgroup (x, i) enters a part of the
// parent's pages into child i's table row.  A parent of a forked child that is
// not empty is no child of the call, so its row does not change here.
__global__ __launch_bounds__(256) void page_fork_apply_kernel(
    int32_t rows, int32_t row_pages, int32_t pages, int32_t P, const int32_t* __restrict__ parent,
    const int32_t* __restrict__ child, int32_t* __restrict__ table,
    const int32_t* __restrict__ lengths, int32_t* __restrict__ refs,
    const int32_t* __restrict__ dst, const int32_t* __restrict__ ok) {
  const int i = blockIdx.y;
  if (!ok[i]) return;
  const int32_t c = child[i];
  const int32_t len = lengths[c];
  const int32_t whole = len / P;
  const int64_t to = static_cast<int64_t>(c) * row_pages;
  const int64_t from = static_cast<int64_t>(parent[i]) * row_pages;
  for (int32_t s = blockIdx.x * 256 + threadIdx.x; s < whole; s += gridDim.x * 256) {
    const int32_t page = table[from + s];
    table[to + s] = page;
    if (page >= 0 && page < pages) atomicAdd(refs + page, 1);  // integer: any order, same sum
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && len % P != 0) table[to + whole] = dst[i];
}

// misa_page_free: workgroup (x, i) clears a part of row i.  Lengths are read
// by every workgroup of the row, so they are cleared by a launch of their own.
__global__ __launch_bounds__(256) void page_free_kernel(int32_t rows, int32_t row_pages,
                                                        int32_t pages, int32_t P,
                                                        const int32_t* __restrict__ row,
                                                        int32_t* __restrict__ table,
                                                        const int32_t* __restrict__ lengths,
                                                        int32_t* __restrict__ refs) {
  const int i = blockIdx.y;
  const int32_t r = row[i];
  if (r < 0 || r >= rows) return;
  bool before = false;
  for (int j = threadIdx.x; j < i; j += 256) before |= row[j] == r;
  if (__syncthreads_or(before)) return;
  const int32_t held = pages_of(held_tokens(lengths[r], row_pages, P), P);
  const int64_t at = static_cast<int64_t>(r) * row_pages;
  for (int32_t s = blockIdx.x * 256 + threadIdx.x; s < held; s += gridDim.x * 256) {
    const int32_t page = table[at + s];
    table[at + s] = kNone;
    if (page >= 0 && page < pages) atomicSub(refs + page, 1);
  }
}

__global__ __launch_bounds__(256) void page_clear_lengths_kernel(int32_t n, int32_t rows,
                                                                 const int32_t* __restrict__ row,
                                                                 int32_t* __restrict__ lengths) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int32_t r = row[i];
  if (r >= 0 && r < rows) lengths[r] = 0;
}

// Workgroups per table row: four entries a thread, at most 64 (the kernels loop).
int32_t row_blocks(const Cache& c) {
  const int32_t blocks = (c.row_pages - 1) / 1024 + 1;
  return blocks < 64 ? blocks : 64;
}

// ---------------------------------------------------------------- compaction

constexpr int kCountPages = 4096;  // pages per counting workgroup

__global__ __launch_bounds__(256) void page_count_kernel(int32_t pages,
                                                         const int32_t* __restrict__ refs,
                                                         int32_t* __restrict__ counts) {
  __shared__ int tmp[4];
  int mine = 0;
  const int32_t c0 = blockIdx.x * kCountPages;
  for (int32_t p = c0 + threadIdx.x; p < min(c0 + kCountPages, pages); p += 256)
    mine += refs[p] > 0;
  int total;
  block_exclusive_sum<256>(mine, tmp, total);
  if (threadIdx.x == 0) counts[blockIdx.x] = total;
}

// Live pages in [0, end): the counts of the whole chunks below and the rest of
// the last one.  All threads; contains barriers.
__device__ int live_below(int32_t end, const int32_t* __restrict__ refs,
                          const int32_t* __restrict__ counts, int* tmp) {
  int mine = 0;
  const int32_t whole = end / kCountPages;
  for (int32_t b = threadIdx.x; b < whole; b += 256) mine += counts[b];
  for (int32_t p = whole * kCountPages + threadIdx.x; p < end; p += 256) mine += refs[p] > 0;
  int total;
  block_exclusive_sum<256>(mine, tmp, total);
  return total;
}

// Second launch: the rank of every hole (a free page below `live`) and mover
// (a live page behind it), by prefix sums over 256 pages per workgroup.  A
// mover's map entry holds -2 - rank until the last launch.
__global__ __launch_bounds__(256) void page_place_kernel(int32_t pages, int32_t chunks,
                                                         const int32_t* __restrict__ refs,
                                                         const int32_t* __restrict__ counts,
                                                         int32_t* __restrict__ map,
                                                         int32_t* __restrict__ live_out,
                                                         int32_t* __restrict__ src,
                                                         int32_t* __restrict__ dst) {
  __shared__ int tmp[4];
  int mine = 0;
  for (int b = threadIdx.x; b < chunks; b += 256) mine += counts[b];
  int live;
  block_exclusive_sum<256>(mine, tmp, live);
  const int stay = live_below(live, refs, counts, tmp);  // live pages that do not move
  const int32_t p0 = blockIdx.x * 256;
  const int before = live_below(p0, refs, counts, tmp);
  const int32_t p = p0 + threadIdx.x;
  const bool inside = p < pages;
  const bool used = inside && refs[p] > 0;
  int total;
  const int rank = before + block_exclusive_sum<256>(used, tmp, total);  // live pages before p
  const int holes = live - stay;
  if (inside) {
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
  }
  if (p == 0) live_out[0] = live;
}

// Last launch: the movers' map entries, refs and the tables.  Threads that
// meet an entry of `map` before or after it is resolved find the same page.
__global__ __launch_bounds__(256) void page_finish_kernel(
    int32_t pages, int64_t entries, const int32_t* __restrict__ table, const int32_t* refs,
    int32_t* __restrict__ table_out, int32_t* refs_out, int32_t* map,
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
    const int32_t id = table[i];
    int32_t to = kNone;
    if (id >= 0 && id < pages) {
      to = map[id];
      if (to < kNone) to = dst[-2 - to];
    }
    table_out[i] = to;
  }
}

// ---------------------------------------------------------------- copies

constexpr int kCopyBytes = 16384;  // bytes of a page that one workgroup copies

struct CopyPlan {
  PageBuffers bufs;
  int64_t first[kMaxPageBuffers];  // first workgroup of each buffer
  int32_t parts[kMaxPageBuffers];  // workgroups per page
};

template <class V>
__device__ __forceinline__ void copy_run(uint8_t* to, const uint8_t* from, int64_t bytes) {
  constexpr int kStep = 256 * sizeof(V);
  for (int64_t o = threadIdx.x * sizeof(V); o < bytes; o += kStep)
    *reinterpret_cast<V*>(to + o) = *reinterpret_cast<const V*>(from + o);
}

// Workgroups run over (buffer, pair, plane, part of the page).
__global__ __launch_bounds__(256) void page_copy_kernel(CopyPlan plan, int32_t pages,
                                                        const int32_t* __restrict__ src,
                                                        const int32_t* __restrict__ dst) {
  int b = 0;
  while (b + 1 < plan.bufs.n && static_cast<int64_t>(blockIdx.x) >= plan.first[b + 1]) ++b;
  const PageBuffer buf = plan.bufs.b[b];
  int64_t w = blockIdx.x - plan.first[b];
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
    copy_run<uint4>(to, from, bytes);
  else
    copy_run<uint32_t>(to, from, bytes);
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
      return launch_write<64>(c, n, row, pos, k_new, v_new, k_pages, k_scale, v_pages, v_scale,
                              table, st);
    case 128:
      return launch_write<128>(c, n, row, pos, k_new, v_new, k_pages, k_scale, v_pages, v_scale,
                               table, st);
    case 256:
      return launch_write<256>(c, n, row, pos, k_new, v_new, k_pages, k_scale, v_pages, v_scale,
                               table, st);
    default:
      return launch_write<576>(c, n, row, pos, k_new, v_new, k_pages, k_scale, v_pages, v_scale,
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
  page_fork_plan_kernel<<<1, kListThreads, 0, st>>>(n, c.rows, c.row_pages, c.pages, c.P, parent,
                                                    child, table, lengths, refs, src, dst, ok);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid(row_blocks(c), n);
  page_fork_apply_kernel<<<grid, 256, 0, st>>>(c.rows, c.row_pages, c.pages, c.P, parent, child,
                                               table, lengths, refs, dst, ok);
  return hipGetLastError();
}

hipError_t launch_page_free(const Cache& c, int32_t n, const int32_t* row, int32_t* table,
                            int32_t* lengths, int32_t* refs, hipStream_t st) {
  const dim3 grid(row_blocks(c), n);
  page_free_kernel<<<grid, 256, 0, st>>>(c.rows, c.row_pages, c.pages, c.P, row, table, lengths,
                                         refs);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  page_clear_lengths_kernel<<<(n + 255) / 256, 256, 0, st>>>(n, c.rows, row, lengths);
  return hipGetLastError();
}

size_t page_compact_ws_bytes(const Cache& c) {
  return align_up((static_cast<size_t>(c.pages) + kCountPages - 1) / kCountPages * sizeof(int32_t));
}

hipError_t launch_page_compact(const Cache& c, const int32_t* table, const int32_t* refs,
                               int32_t* table_out, int32_t* refs_out, int32_t* map, int32_t* live,
                               int32_t* src, int32_t* dst, void* ws, hipStream_t st) {
  const int32_t chunks = (c.pages + kCountPages - 1) / kCountPages;
  auto* counts = static_cast<int32_t*>(ws);
  page_count_kernel<<<chunks, 256, 0, st>>>(c.pages, refs, counts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  page_place_kernel<<<(c.pages + 255) / 256, 256, 0, st>>>(c.pages, chunks, refs, counts, map, live,
                                                           src, dst);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t entries = static_cast<int64_t>(c.rows) * c.row_pages;
  const int64_t most = entries > c.pages ? entries : c.pages;
  page_finish_kernel<<<static_cast<uint32_t>((most + 255) / 256), 256, 0, st>>>(
      c.pages, entries, table, refs, table_out, refs_out, map, live, src, dst);
  return hipGetLastError();
}

bool page_copy_supported(const PageBuffers& b, int32_t n) {
  int64_t blocks = 0;
  for (int32_t i = 0; i < b.n; ++i) {
    if (copy_blocks(b.b[i], n) >= (int64_t{1} << 31)) return false;
    blocks += copy_blocks(b.b[i], n);
  }
  return blocks < (int64_t{1} << 31);
}

hipError_t launch_page_copy(const PageBuffers& b, int32_t pages, int32_t n, const int32_t* src,
                            const int32_t* dst, hipStream_t st) {
  CopyPlan plan{};
  plan.bufs = b;
  int64_t blocks = 0;
  for (int32_t i = 0; i < b.n; ++i) {
    plan.first[i] = blocks;
    plan.parts[i] = copy_parts(b.b[i]);
    blocks += copy_blocks(b.b[i], n);
  }
  page_copy_kernel<<<static_cast<uint32_t>(blocks), 256, 0, st>>>(plan, pages, src, dst);
  return hipGetLastError();
}

}  // namespace misa
