// Host-side launchers of the MISA kernels (internal; the public ABI is misa.h).
// Each returns the hipError_t of its launch(es).  Arguments were validated by
// the caller (api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace misa {

struct Shape {
  int32_t batch, L, T, H, d, B, dtype;
  int64_t M() const { return (static_cast<int64_t>(L) + B - 1) / B; }
};

hipError_t launch_pool(const Shape& s, int32_t block_begin, int32_t block_count, const void* k,
                       const float* k_scale, float* pooled, hipStream_t st);

// Router: E and top-h heads.  ws must hold route_ws_bytes(s).
size_t route_ws_bytes(const Shape& s);
hipError_t launch_route(const Shape& s, int32_t h, const void* q, const float* q_scale,
                        const float* w, const float* pooled, const void* k, const float* k_scale,
                        int32_t* heads, float* E_out, void* ws, hipStream_t st);

// Router on the matrix cores (bf16/fp8 inputs); no workspace.
bool route_mfma_supported(const Shape& s);
size_t route_mfma_ws_bytes(const Shape& s);
hipError_t launch_route_mfma(const Shape& s, int32_t h, const void* q, const float* q_scale,
                             const float* w, const float* pooled, const void* k,
                             const float* k_scale, int32_t* heads, float* E_out, void* ws,
                             hipStream_t st);

// Decode router (T == 1) on the vector ALU: chunked partial sums + finalize.
size_t route_decode_ws_bytes(const Shape& s);
hipError_t launch_route_decode(const Shape& s, int32_t h, const void* q, const float* q_scale,
                               const float* w, const float* pooled, const void* k,
                               const float* k_scale, int32_t* heads, float* E_out, void* ws,
                               hipStream_t st);

// Token scoring + top-k over each query's causal prefix.  heads == nullptr
// scores with all H heads (dense DSA); otherwise with the nh listed heads.
size_t score_ws_bytes(const Shape& s, int32_t nh, int32_t k);
hipError_t launch_score_topk(const Shape& s, int32_t nh, const int32_t* heads, int32_t k,
                             const void* q, const float* q_scale, const float* w, const void* kk,
                             const float* k_scale, int32_t* idx, float* scores_out, void* ws,
                             hipStream_t st);

// Decode (T == 1, bf16/fp8) token scoring + top-k: MFMA key streaming, then a
// per-sequence select.  ws must hold decode_ws_bytes(s).
size_t decode_ws_bytes(const Shape& s);
hipError_t launch_decode_score_topk(const Shape& s, int32_t nh, const int32_t* heads, int32_t k,
                                    const void* q, const float* q_scale, const float* w,
                                    const void* kk, const float* k_scale, int32_t* idx,
                                    float* scores_out, void* ws, hipStream_t st);

// Multi-query decode (2 <= T <= 8 queries at the end of each sequence,
// bf16/fp8, nh <= 16): every key read once for all T queries, then a row
// histogram and the decode select per (sequence, query).  ws must hold
// decode_mq_ws_bytes(s).
bool decode_mq_supported(const Shape& s, int32_t nh);
size_t decode_mq_ws_bytes(const Shape& s);
hipError_t launch_decode_mq_score_topk(const Shape& s, int32_t nh, const int32_t* heads, int32_t k,
                                       const void* q, const float* q_scale, const float* w,
                                       const void* kk, const float* k_scale, int32_t* idx,
                                       float* scores_out, void* ws, hipStream_t st);

// Fused decode step (T == 1, bf16/fp8): refresh the pooled key of the block
// holding key L-1, route (E, top-h) and score + top-k; two kernels.  ws must
// hold decode_ws_bytes(s).
hipError_t launch_decode_step(const Shape& s, int32_t h, int32_t k, const void* q,
                              const float* q_scale, const float* w, float* pooled, const void* kk,
                              const float* k_scale, int32_t* heads, float* E_out, int32_t* idx,
                              float* scores_out, void* ws, hipStream_t st);

// Prefill (T > 1, bf16/fp8) token scoring + top-k on 32x32 MFMA tiles with
// sampled thresholds, certified candidate selection and a repair path.
bool prefill_supported(const Shape& s);
size_t prefill_ws_bytes(const Shape& s, int32_t nh, int32_t k);
hipError_t launch_prefill_score_topk(const Shape& s, int32_t nh, const int32_t* heads, int32_t k,
                                     const void* q, const float* q_scale, const float* w,
                                     const void* kk, const float* k_scale, int32_t* idx,
                                     float* scores_out, void* ws, hipStream_t st);

// MISA-dagger fine stage.
size_t rerank_ws_bytes(const Shape& s, int32_t kprime);
hipError_t launch_rerank(const Shape& s, int32_t kprime, int32_t k, const void* q,
                         const float* q_scale, const float* w, const void* kk, const float* k_scale,
                         const int32_t* cand, int32_t* idx, float* scores_out, void* ws,
                         hipStream_t st);

// The re-rank with a list of heads per query (heads [batch*T, nh]; nullptr:
// every head) -- the routed scoring over a candidate list.  m > 0: `cand`
// holds m blocks per query ([batch*T, m]) whose B tokens each are the first
// m B of the kprime candidates (the rest padding); needs a head list of at
// most 16.  Head lists and blocks: bf16/fp8 keys within a buffer
// descriptor's reach only.
hipError_t launch_rerank_heads(const Shape& s, int32_t kprime, int32_t k, const void* q,
                               const float* q_scale, const float* w, const void* kk,
                               const float* k_scale, const int32_t* cand, int32_t m,
                               const int32_t* heads, int32_t nh, int32_t* idx, float* scores_out,
                               void* ws, hipStream_t st);

// Pooled keys -> bf16 hi and lo planes [batch*M, 128] (the router's B
// operand).
hipError_t launch_pooled_split(const Shape& s, const float* pooled, uint16_t* hi, uint16_t* lo,
                               hipStream_t st);

// MISA x HISA: block scores G (Eq. (7) affinities summed over heads), the
// top-m blocks, and the routed top-k over their tokens.
bool hisa_supported(const Shape& s, int32_t m);
size_t hisa_ws_bytes(const Shape& s, int32_t m, int32_t k);
hipError_t launch_hisa_score_topk(const Shape& s, int32_t nh, const int32_t* heads, int32_t m,
                                  int32_t k, const void* q, const float* q_scale, const float* w,
                                  const float* pooled, const void* kk, const float* k_scale,
                                  int32_t* blocks_out, float* block_scores_out, int32_t* idx,
                                  float* scores_out, void* ws, hipStream_t st);

// ---------------------------------------------------------------- serving

struct Cache {
  int32_t rows, row_pages, pages, P;  // P: tokens per page
  int32_t kv_heads, dk, dv, dtype;
  // One cached row per token serves every head; its first dv elements are the value.
  bool latent() const { return dk == 576 && dv == 512; }
};

constexpr float kLog2e = 1.4426950408889634f;  // scores are scaled to powers of two by scale * log2(e)
// Attention of one new token per row.  k > 0: over the listed tokens only.
size_t attend_ws_bytes(const Cache& c, int32_t heads, int32_t k);
hipError_t launch_attend(const Cache& c, int32_t heads, int32_t k, float scale, const void* q,
                         const void* k_pages, const float* k_scale, const void* v_pages,
                         const float* v_scale, const int32_t* table, const int32_t* lengths,
                         const int32_t* idx, void* out, float* lse, void* ws, hipStream_t st);

hipError_t launch_page_write(const Cache& c, int32_t n, const int32_t* row, const int32_t* pos,
                             const void* k_new, const void* v_new, void* k_pages, float* k_scale,
                             void* v_pages, float* v_scale, const int32_t* table, hipStream_t st);

constexpr int32_t kMaxList = 4096;  // entries of an extend, fork or free list (in LDS)
hipError_t launch_page_extend(const Cache& c, int32_t n, const int32_t* row, const int32_t* count,
                              int32_t* table, int32_t* lengths, int32_t* refs, int32_t* ok,
                              hipStream_t st);
hipError_t launch_page_fork(const Cache& c, int32_t n, const int32_t* parent, const int32_t* child,
                            int32_t* table, int32_t* lengths, int32_t* refs, int32_t* src,
                            int32_t* dst, int32_t* ok, hipStream_t st);
hipError_t launch_page_free(const Cache& c, int32_t n, const int32_t* row, int32_t* table,
                            int32_t* lengths, int32_t* refs, hipStream_t st);
size_t page_compact_ws_bytes(const Cache& c);
hipError_t launch_page_compact(const Cache& c, const int32_t* table, const int32_t* refs,
                               int32_t* table_out, int32_t* refs_out, int32_t* map, int32_t* live,
                               int32_t* src, int32_t* dst, void* ws, hipStream_t st);

constexpr int32_t kMaxPageBuffers = 8;
struct PageBuffer {
  uint8_t* data;
  int64_t page_bytes;
  int32_t planes;
};
struct PageBuffers {
  PageBuffer b[kMaxPageBuffers];
  int32_t n;
};
bool page_copy_supported(const PageBuffers& b, int32_t n);
hipError_t launch_page_copy(const PageBuffers& b, int32_t pages, int32_t n, const int32_t* src,
                            const int32_t* dst, hipStream_t st);

constexpr int32_t kMaxNorm = 32768;  // elements of a normed row (one row in LDS)
hipError_t launch_rms_norm(int32_t rows, int32_t n, int32_t groups, int32_t x_dtype,
                           int32_t out_dtype, float eps, const void* x, const void* residual,
                           const float* weight, void* sum_out, void* out, float* out_scale,
                           hipStream_t st);

inline size_t align_up(size_t x, size_t a = 256) { return (x + a - 1) / a * a; }

// The fixed device scratch of the no-allocation decode step: its size, and
// this device's address of it (looked up on the first call on each device).
constexpr size_t kStaticScratchBytes = size_t{64} << 20;
hipError_t static_scratch(void** ptr);

}  // namespace misa
