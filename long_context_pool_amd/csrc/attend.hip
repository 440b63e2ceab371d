// Attention of one new token per row over a paged cache (misa_attend in
// misa.h): every cached token of the row, or those of an index list.
#include "common.hpp"
#include "launch.hpp"
#include "mfma.hpp"

namespace misa {

namespace {

constexpr int kTile = 256;  // tokens per pass: one per thread

// One workgroup per (head, row): scores of 256 tokens, one per thread, then
// the running maximum and sum, then the values, two dimensions per thread.
template <int DK, int DV, int DT, bool LATENT>
__global__ __launch_bounds__(256) void attend_kernel(
    Cache c, int32_t heads, int32_t k, float scale, const uint16_t* __restrict__ q,
    const void* __restrict__ k_pages, const float* __restrict__ k_scale,
    const void* __restrict__ v_pages, const float* __restrict__ v_scale,
    const int32_t* __restrict__ table, const int32_t* __restrict__ lengths,
    const int32_t* __restrict__ idx, uint16_t* __restrict__ out, float* __restrict__ lse) {
  __shared__ float qs[DK];
  __shared__ float ps[kTile];
  __shared__ int64_t slots[kTile];
  __shared__ float red[4];
  const int row = blockIdx.y, head = blockIdx.x;
  const int kvh = head / (heads / c.kv_heads);
  const int64_t qat = (static_cast<int64_t>(row) * heads + head);
  for (int e = threadIdx.x; e < DK; e += 256) qs[e] = bf16_bits_to_f32(q[qat * DK + e]);
  const int32_t len = min(lengths[row], c.row_pages * c.P);
  const int32_t todo = k > 0 ? k : len;
  float m = -INFINITY, l = 0.f, o[2] = {0.f, 0.f};
  for (int32_t t0 = 0; t0 < todo; t0 += kTile) {
    __syncthreads();
    const int32_t t = t0 + threadIdx.x;
    int32_t s = t < todo ? (k > 0 ? idx[static_cast<int64_t>(row) * k + t] : t) : -1;
    int64_t slot = -1;
    if (s >= 0 && s < len) {
      const int32_t page = table[static_cast<int64_t>(row) * c.row_pages + s / c.P];
      if (page >= 0 && page < c.pages)
        slot = (static_cast<int64_t>(page) * c.kv_heads + kvh) * c.P + s % c.P;
    }
    float score = -INFINITY;
    if (slot >= 0) {
      float dot = 0.f;
      for (int e = 0; e < DK; ++e) dot += qs[e] * load_elem<DT>(k_pages, slot * DK + e);
      if (DT == kFP8) dot *= k_scale[slot];
      score = dot * scale;
    }
    float top = score;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
    if (lane_id() == 0) red[threadIdx.x / kWave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float mn = fmaxf(m, top);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float a = expf(m - base);
    const float p = slot >= 0 ? expf(score - base) : 0.f;
    ps[threadIdx.x] = p;
    slots[threadIdx.x] = slot;
    float sum = p;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) sum += __shfl_xor(sum, d, kWave);
    __syncthreads();
    if (lane_id() == 0) red[threadIdx.x / kWave] = sum;
    __syncthreads();
    l = l * a + red[0] + red[1] + red[2] + red[3];
    m = mn;
    o[0] *= a;
    o[1] *= a;
    for (int i = 0; i < min(kTile, todo - t0); ++i) {
      const int64_t sl = slots[i];
      if (sl < 0) continue;
      float w = ps[i];
      if (DT == kFP8) w *= LATENT ? k_scale[sl] : v_scale[sl];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int e = u * 256 + threadIdx.x;
        if (e < DV)
          o[u] += w * (LATENT ? load_elem<DT>(k_pages, sl * DK + e) : load_elem<DT>(v_pages, sl * DV + e));
      }
    }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int e = u * 256 + threadIdx.x;
    if (e < DV)
      reinterpret_cast<__bf16*>(out)[qat * DV + e] = static_cast<__bf16>(l > 0.f || l != l ? o[u] / l : 0.f);
  }
  if (lse && threadIdx.x == 0) lse[qat] = m == -INFINITY ? -INFINITY : m + logf(l);
}

template <int DK, int DV, bool LATENT>
hipError_t launch_dims(const Cache& c, int32_t heads, int32_t k, float scale, const void* q,
                       const void* k_pages, const float* k_scale, const void* v_pages,
                       const float* v_scale, const int32_t* table, const int32_t* lengths,
                       const int32_t* idx, void* out, float* lse, hipStream_t st) {
  const dim3 grid(heads, c.rows);
  const auto* qq = static_cast<const uint16_t*>(q);
  auto* o = static_cast<uint16_t*>(out);
  if (c.dtype == kFP8)
    attend_kernel<DK, DV, kFP8, LATENT><<<grid, 256, 0, st>>>(
        c, heads, k, scale, qq, k_pages, k_scale, v_pages, v_scale, table, lengths, idx, o, lse);
  else
    attend_kernel<DK, DV, kBF16, LATENT><<<grid, 256, 0, st>>>(
        c, heads, k, scale, qq, k_pages, k_scale, v_pages, v_scale, table, lengths, idx, o, lse);
  return hipGetLastError();
}

}  // namespace

size_t attend_ws_bytes(const Cache&, int32_t, int32_t) { return 0; }

hipError_t launch_attend(const Cache& c, int32_t heads, int32_t k, float scale, const void* q,
                         const void* k_pages, const float* k_scale, const void* v_pages,
                         const float* v_scale, const int32_t* table, const int32_t* lengths,
                         const int32_t* idx, void* out, float* lse, void*, hipStream_t st) {
  switch (c.dk) {
    case 64:
      return launch_dims<64, 64, false>(c, heads, k, scale, q, k_pages, k_scale, v_pages, v_scale,
                                        table, lengths, idx, out, lse, st);
    case 128:
      return launch_dims<128, 128, false>(c, heads, k, scale, q, k_pages, k_scale, v_pages, v_scale,
                                          table, lengths, idx, out, lse, st);
    case 256:
      return launch_dims<256, 256, false>(c, heads, k, scale, q, k_pages, k_scale, v_pages, v_scale,
                                          table, lengths, idx, out, lse, st);
    default:
      return launch_dims<576, 512, true>(c, heads, k, scale, q, k_pages, k_scale, v_pages, v_scale,
                                         table, lengths, idx, out, lse, st);
  }
}

}  // namespace misa
