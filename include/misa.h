/*
 * misa.h -- C ABI of the MISA indexer library for AMD Instinct MI355X (gfx950).
 *
 * MISA (Mixture of Indexer Sparse Attention) replaces the DeepSeek Sparse
 * Attention (DSA) token indexer: a block-pooled router picks, per query, the
 * h most useful of the H indexer heads, and only those heads score the
 * query's causal prefix before the top-k token selection.  Source: the MISA
 * summary page ("MISA: Mixture of Indexer Sparse Attention for Long-Context
 * LLM Inference"), Eq. (1)-(2) in "Introduction and Theoretical Foundation",
 * Eq. (4), (7)-(10) in "Methodology" 1, Eq. (11)-(12) in "Methodology" 2.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Every pointer is a DEVICE pointer owned by the caller.  The library never
 *    allocates or frees device memory; scratch space is the caller's `ws`
 *    buffer of `ws_bytes` bytes (size it with misa_workspace_bytes()).
 *  - Arrays are dense row-major with the shapes given below and 16-byte
 *    aligned base addresses.  Element types: q and k are `shape->qk_dtype`
 *    (fp32, bf16, or OCP fp8 e4m3fn); w, scales, pooled keys, E and scores
 *    are fp32; indices are int32.
 *  - Sequence b holds L keys; its T queries sit at positions L-T .. L-1, and
 *    query t sees the causal prefix of keys 0 .. L-T+t (its own position
 *    included), n_t = L-T+t+1 keys.  Decode is T = 1.
 *  - fp8 inputs carry one fp32 scale per query token, q_scale [batch, T], and
 *    one per key token, k_scale [batch, L]: value = code * scale, scale > 0.
 *    For fp32/bf16 inputs the scale pointers are ignored and may be NULL.
 *  - Calls are asynchronous on `stream` (NULL = the default stream).  Argument
 *    checks run on the host before anything is launched; a failed check
 *    returns its status and launches nothing.  A launch failure returns
 *    MISA_ERR_HIP.  The library keeps no mutable global state: calls on
 *    different streams are independent when their workspaces are distinct.
 *    The only state carried between calls lives in the caller's `ws` (see
 *    misa_decode_step); no result ever depends on it.
 *  - Limits of this build: d = 128; 1 <= H <= 64; 1 <= h <= min(H, 16);
 *    1 <= k <= k' <= 8192; B >= 1; 1 <= T <= L < 2^31; batch*T*max(L,k')
 *    < 2^40.  Violations return MISA_ERR_UNSUPPORTED (a limit of this build)
 *    or MISA_ERR_INVALID_ARG (an argument no build accepts).
 *  - Selected-token outputs have SET semantics: the order of the k slots is
 *    unspecified; when n_t < k the trailing slots hold index -1 and score
 *    -INFINITY.  Among tokens with bit-identical fp32 scores the lower token
 *    index is kept.
 */
#ifndef MISA_H
#define MISA_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MISA_OK = 0,
  MISA_ERR_INVALID_ARG = -1, /* a null/misaligned pointer or an impossible size */
  MISA_ERR_UNSUPPORTED = -2, /* a valid request outside this build's limits   */
  MISA_ERR_WORKSPACE = -3,   /* ws is NULL or smaller than required            */
  MISA_ERR_HIP = -4          /* a HIP launch or runtime call failed            */
} misa_status;

typedef enum {
  MISA_F32 = 0,
  MISA_BF16 = 1,
  MISA_FP8_E4M3 = 2 /* OCP e4m3fn: bias 7, max 448, no infinities */
} misa_dtype;

/* Problem shape.  H is the number of indexer heads (H^I on the page), d the
 * head dimension, B the router block size, qk_dtype a misa_dtype. */
typedef struct {
  int32_t batch, L, T, H, d, B;
  int32_t qk_dtype;
} misa_shape;

/* Bytes of workspace that suffice for every entry point below called with
 * this shape and these h, k, k' (pass kprime = k when MISA-dagger is unused).
 * Returns 0 for an invalid shape. */
size_t misa_workspace_bytes(const misa_shape* shape, int32_t h, int32_t k, int32_t kprime);

/* Eq. (4): pooled[b, m, :] = mean of k[b, s, :] over the block
 * s in [m*B, min((m+1)*B, L)), for m < M = ceil(L/B).  The last block may be
 * partial (mean over its actual members).  fp8 keys are dequantised first.
 *   k        [batch, L, d]   qk_dtype
 *   k_scale  [batch, L]      fp32 (fp8 only)
 *   pooled   [batch, M, d]   fp32, written
 * In decode the pooled keys are a cache: call once per sequence and again
 * only for blocks that changed (see misa_pool_keys_range). */
misa_status misa_pool_keys(const misa_shape* shape, const void* k, const float* k_scale,
                           float* pooled, hipStream_t stream);

/* Eq. (4) restricted to blocks [block_begin, block_begin + block_count) of
 * every sequence: the incremental update of the decode cache when new keys
 * land in the last block.  Same layouts as misa_pool_keys; other blocks of
 * `pooled` are left untouched.  block_begin + block_count must be <= M. */
misa_status misa_pool_keys_range(const misa_shape* shape, int32_t block_begin, int32_t block_count,
                                 const void* k, const float* k_scale, float* pooled,
                                 hipStream_t stream);

/* Eq. (7)-(8), the block-pooled router.  For query t with n_t = L-T+t+1:
 *   E[b,t,j] = (1/M_t) * sum_{m < M_t} |w[b,t,j] * ReLU(q[b,t,j,:] . p_m)|,
 * M_t = ceil(n_t/B), where p_m = pooled[b,m,:] for the floor(n_t/B) blocks
 * lying wholly in the prefix and, when B does not divide n_t, the last p_m is
 * the mean of keys floor(n_t/B)*B .. n_t-1 (computed here from k).  Then
 * heads[b,t,:] = the h heads of largest E (ties: lower head), ascending.
 *   q        [batch, T, H, d]  qk_dtype      q_scale [batch, T] (fp8 only)
 *   w        [batch, T, H]     fp32
 *   pooled   [batch, M, d]     fp32 (from misa_pool_keys)
 *   k        [batch, L, d]     qk_dtype      k_scale [batch, L] (fp8 only)
 *   heads    [batch, T, h]     int32, written (ascending)
 *   E_out    [batch, T, H]     fp32, written if non-NULL */
misa_status misa_route(const misa_shape* shape, int32_t h, const void* q, const float* q_scale,
                       const float* w, const float* pooled, const void* k, const float* k_scale,
                       int32_t* heads, float* E_out, void* ws, size_t ws_bytes, hipStream_t stream);

/* Eq. (9)-(10) (Eq. (11) when called with k = k'):
 *   I[b,t,s] = sum_{j in heads[b,t,:]} w[b,t,j] * ReLU(q[b,t,j,:] . k[b,s,:])
 * for s in 0 .. n_t-1, then idx[b,t,:] = the k tokens of largest I.
 *   heads      [batch, T, h]  int32 head ids in [0, H) (e.g. from misa_route)
 *   idx        [batch, T, k]  int32, written (set semantics, -1 padding)
 *   scores_out [batch, T, k]  fp32 I of each idx slot, written if non-NULL */
misa_status misa_score_topk(const misa_shape* shape, int32_t h, int32_t k, const void* q,
                            const float* q_scale, const float* w, const void* kk,
                            const float* k_scale, const int32_t* heads, int32_t* idx,
                            float* scores_out, void* ws, size_t ws_bytes, hipStream_t stream);

/* Eq. (12), the fine stage of MISA-dagger: for every candidate s in
 * cand[b,t,:] (entries < 0 are padding and ignored), the full-head score
 *   I[b,t,s] = sum_{j < H} w[b,t,j] * ReLU(q[b,t,j,:] . k[b,s,:]),
 * then idx[b,t,:] = the k candidates of largest I.  Candidates must be
 * distinct token positions within query t's prefix.  Key rows are gathered
 * in list order, so a list sorted by token position runs faster (prefill
 * lists of misa_score_topk come out that way, apart from the few entries of
 * the threshold bin at their end); the result does not depend on the order.
 *   cand       [batch, T, kprime]  int32 (e.g. idx of misa_score_topk with k')
 *   idx        [batch, T, k]       int32, written
 *   scores_out [batch, T, k]       fp32, written if non-NULL */
misa_status misa_rerank(const misa_shape* shape, int32_t kprime, int32_t k, const void* q,
                        const float* q_scale, const float* w, const void* kk, const float* k_scale,
                        const int32_t* cand, int32_t* idx, float* scores_out, void* ws,
                        size_t ws_bytes, hipStream_t stream);

/* One decode step of MISA (T = 1; bf16 or fp8 only): Eq. (4) for the block
 * holding the newest key, then Eq. (7)-(8) and Eq. (9)-(10) -- the results of
 *   misa_pool_keys_range(shape, M-1, 1, ...); misa_route(...); misa_score_topk(...)
 * in two kernel launches (three when batch < 8).
 *   pooled   [batch, M, d]  fp32, read and written: blocks 0 .. M-2 must hold
 *            their Eq. (4) means (the cache kept by misa_pool_keys); block
 *            M-1 (keys (M-1)*B .. L-1, possibly partial) is recomputed from k
 *            and written.
 *   heads    [batch, h]     int32, written (ascending)
 *   E_out    [batch, H]     fp32, written if non-NULL
 *   idx, scores_out [batch, k] as misa_score_topk.
 * Other arguments and layouts as misa_route and misa_score_topk.  T != 1 or
 * fp32 inputs return MISA_ERR_UNSUPPORTED.
 *
 * State in `ws` (batch >= 8, the single-kernel form): the G workgroups of a
 * sequence share their router partial sums through `ws`, using one 64-bit
 * arrival word per sequence that this call's select kernel re-arms for the
 * NEXT call on the same `ws`.  A call whose `ws` is fresh (first call), was
 * used in between by another entry point, or was sized for another shape
 * finds no armed word: every workgroup then computes all router partials
 * itself (same additions in the same order, so the same result bits) and
 * the call is slower (about the router cost times G).  An armed word whose
 * peers are late makes a workgroup poll it up to 65536 times (with short
 * sleeps) before it takes the same local path, so one call never waits on
 * another.  Two calls that overlap on one `ws` race and are not allowed. */
misa_status misa_decode_step(const misa_shape* shape, int32_t h, int32_t k, const void* q,
                             const float* q_scale, const float* w, float* pooled, const void* kk,
                             const float* k_scale, int32_t* heads, float* E_out, int32_t* idx,
                             float* scores_out, void* ws, size_t ws_bytes, hipStream_t stream);

/* misa_decode_step for callers that cannot allocate device memory or pass a
 * workspace: code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc.  Same arguments (minus ws), checks and results as
 * misa_decode_step; the workspace is a fixed device array inside the library,
 * MISA_NOALLOC_SCRATCH_BYTES (64 MiB) per GPU, which each GPU the library
 * runs on holds until the process ends.  Nothing is allocated by the call
 * (no hipMalloc, no allocating library routine).
 *   - A shape whose decode workspace exceeds the array returns
 *     MISA_ERR_UNSUPPORTED and launches nothing.  The need is batch * L * 4
 *     bytes of scores, about 9 MB of digit histograms when batch >= 8 (34 KB
 *     per sequence below that) and about 17 KB per sequence: batch 32 x
 *     L 32768 takes 13.6 MB, batch 8 x L 131072 13.1 MB, batch 64 x
 *     L 131072 43.9 MB, batch 1 x L 2^20 4.3 MB.
 *   - Every call on one GPU shares that GPU's array, which keeps the last
 *     call's contents (including the router arrival words documented at
 *     misa_decode_step).  Calls that overlap in time on one GPU -- on
 *     different streams, or from different threads -- race and give wrong
 *     results: serialise them.
 *   - The first call on each device looks up the array's device address
 *     (hipGetSymbolAddress, no allocation); a failure returns MISA_ERR_HIP. */
#define MISA_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
misa_status misa_decode_step_noalloc(const misa_shape* shape, int32_t h, int32_t k, const void* q,
                                     const float* q_scale, const float* w, float* pooled,
                                     const void* kk, const float* k_scale, int32_t* heads,
                                     float* E_out, int32_t* idx, float* scores_out,
                                     hipStream_t stream);

/* Eq. (1)-(2), the dense DSA indexer baseline: Eq. (9)-(10) with every head
 * j < H, no router.  Layouts as misa_score_topk. */
misa_status dsa_index_dense(const misa_shape* shape, int32_t k, const void* q,
                            const float* q_scale, const float* w, const void* kk,
                            const float* k_scale, int32_t* idx, float* scores_out, void* ws,
                            size_t ws_bytes, hipStream_t stream);

/* MISA x HISA ("Methodology" 1, "Key distinction from HISA"; "Theoretical
 * and Practical Implications", "Scalability"): the Eq. (7) affinities
 * A = w * ReLU(q . p) reduced across the heads instead of the blocks pick the
 * query's top-m blocks, and the routed scoring of Eq. (9) runs only over their
 * tokens.  For query t (n_t = L-T+t+1, the same causal blocks as misa_route):
 *   G[b,t,blk] = sum_{j < H} w[b,t,j] * ReLU(q[b,t,j,:] . p_blk),  blk < M_t
 *   the m blocks of largest G (ties: lower block; all M_t when M_t <= m)
 *   I[b,t,s] = sum_{j in heads[b,t,:]} w[b,t,j] * ReLU(q[b,t,j,:] . k[b,s,:])
 *              for the tokens s <= L-T+t of those blocks
 *   idx[b,t,:] = the k of those tokens with the largest I (ties: lower token;
 *                -1 / -INFINITY padding when they are fewer than k).
 *   pooled            [batch, M, d]  fp32 (misa_pool_keys)
 *   heads             [batch, T, h]  int32 (misa_route)
 *   blocks_out        [batch, T, m]  int32, written if non-NULL: the blocks,
 *                     ascending, -1 padding
 *   block_scores_out  [batch, T, m]  fp32, written if non-NULL: G of each slot
 *   idx, scores_out   [batch, T, k]  as misa_score_topk
 * Limits: bf16 or fp8 inputs, h <= 16, k <= 8192, m * B <= 8192, one
 * sequence's keys below 2 GiB; otherwise MISA_ERR_UNSUPPORTED (h > H, m < 1,
 * k < 1 or a NULL/misaligned input: MISA_ERR_INVALID_ARG).  ws must hold
 * misa_hisa_workspace_bytes(shape, h, m, k) bytes (0 for invalid arguments);
 * it carries nothing from one call to the next. */
size_t misa_hisa_workspace_bytes(const misa_shape* shape, int32_t h, int32_t m, int32_t k);
misa_status misa_hisa_score_topk(const misa_shape* shape, int32_t h, int32_t m, int32_t k,
                                 const void* q, const float* q_scale, const float* w,
                                 const float* pooled, const void* kk, const float* k_scale,
                                 const int32_t* heads, int32_t* blocks_out,
                                 float* block_scores_out, int32_t* idx, float* scores_out,
                                 void* ws, size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------------ serving
 * What stands around the indexer in a serving step: the root-mean-square norm
 * that makes its 8-bit inputs, the paged cache of keys and values, and the
 * attention of the new token over the cached tokens the indexer selected (or
 * over all of them).
 *
 * Conventions on top of those above:
 *  - The limits on d, H, h and k above are the indexer's; each entry point
 *    below states its own.
 *  - Calls that read or change one cache are ordered by the caller (one stream,
 *    or events); calls on different caches are independent.
 *  - Integer arrays the calls read on the device (tables, lengths, lists) are
 *    checked there: an entry that names nothing (a row outside [0, rows), a
 *    page outside [0, pages), a position beyond the table) is skipped, and
 *    nothing outside the described arrays is read or written.
 *  - 8-bit codes are OCP e4m3fn, value = code * scale, rounded to nearest even
 *    from x * (448 / amax); scale = amax / 448, with amax the largest magnitude
 *    of the values that share the scale (NaN left out), and scale = 1 when
 *    amax < 2^-100 (zeros).  misa_page_write rounds that product as if it were
 *    exact, misa_rms_norm (whose x is an fp32 result) its fp32 value.  A NaN
 *    becomes a NaN code; an infinity makes its scale infinite and itself a NaN
 *    code.
 */

/* A paged cache.  Sequence r of `rows` owns row r of the page table: token s
 * of it lives in slot s % page_tokens of page table[r, s / page_tokens].
 *   table    [rows, row_pages]  int32, -1 = no page
 *   lengths  [rows]             int32, cached tokens of the row
 *   refs     [pages]            int32, table entries that name the page; a
 *                               page with refs <= 0 is free
 *   k_pages  [pages, kv_heads, page_tokens, dk]  kv_dtype
 *   v_pages  [pages, kv_heads, page_tokens, dv]  kv_dtype
 *   k_scale, v_scale  [pages, kv_heads, page_tokens]  fp32 (fp8 only, > 0)
 * Head dimensions: dk = dv in {64, 128, 256}; or the latent form dk = 576, dv
 * = 512, kv_heads = 1, where one cached row serves every head and the values
 * are its first 512 elements: v_pages, v_new and v_scale are then NULL.
 * kv_dtype is MISA_BF16 or MISA_FP8_E4M3.  Limits: rows, row_pages, pages and
 * page_tokens >= 1, page_tokens <= 4096, kv_heads <= 256, rows * row_pages <
 * 2^31, row_pages * page_tokens <= 2^30, rows <= 2^20, pages <= 2^24, pages *
 * kv_heads * page_tokens < 2^32 - 1.  The calls that touch only tables, lengths
 * and refs ignore kv_heads, dk, dv and kv_dtype. */
typedef struct {
  int32_t rows, row_pages, pages, page_tokens;
  int32_t kv_heads, dk, dv;
  int32_t kv_dtype;
} misa_cache;

/* Attention of one new token per row over its cached tokens:
 *   o[r, j, :] = sum_s p_s v[r, s, g, :],  p = softmax_s(scale * q[r,j,:] . k[r,s,g,:]),
 *   lse[r, j] = log sum_s exp(scale * q . k),   g = j / (heads / kv_heads),
 * over the visible tokens s: all s < lengths[r], or with k > 0 the entries of
 * idx[r, :] that lie in [0, lengths[r]) -- a list in any order, -1 padded, as
 * the indexer's entry points write it (a token listed twice counts twice).
 * Tokens whose table entry names no page are not visible.  A row without
 * visible tokens gets o = 0 and lse = -INFINITY.  What the cache holds at
 * invisible slots is never used, NaN or not.
 *   q    [rows, heads, dk]  bf16      out [rows, heads, dv]  bf16, written
 *   idx  [rows, k]  int32 (k > 0; k = 0: NULL)
 *   lse  [rows, heads]  fp32, written if non-NULL
 * Scores, softmax and sums are fp32: q . k and a score times log2(e) must be in
 * its range, and cached values below 2^90 in magnitude, or infinite (weights of
 * up to 2^8 are summed before the division by their sum).  A weight goes into
 * its products as two bf16 parts, which hold it to 2^-16.  Limits: heads a
 * multiple of kv_heads, heads <= 1024, rows <= 65535, 0 <= k <= 2^20, |scale| <=
 * 2^127.  ws must hold
 * misa_attend_workspace_bytes(cache, heads, k) bytes (0: invalid arguments or
 * no workspace needed); it carries nothing from one call to the next. */
size_t misa_attend_workspace_bytes(const misa_cache* cache, int32_t heads, int32_t k);
misa_status misa_attend(const misa_cache* cache, int32_t heads, int32_t k, float scale,
                        const void* q, const void* k_pages, const float* k_scale,
                        const void* v_pages, const float* v_scale, const int32_t* table,
                        const int32_t* lengths, const int32_t* idx, void* out, float* lse,
                        void* ws, size_t ws_bytes, hipStream_t stream);

/* Write n new tokens into their pages: token i goes to position pos[i] of row
 * row[i].  fp8 caches get codes and one scale per (token, kv head), from that
 * head's dk (dv) values.  Entries with row outside [0, rows), pos outside the
 * table or no page at that position are skipped (padding of a captured
 * batch); two entries must not name the same slot.  lengths is not looked at:
 * misa_page_extend keeps it, once per step for every layer.
 *   row, pos  [n]  int32
 *   k_new  [n, kv_heads, dk]  bf16        v_new  [n, kv_heads, dv]  bf16
 * n = 0 is a no-op; n * kv_heads <= 2^25. */
misa_status misa_page_write(const misa_cache* cache, int32_t n, const int32_t* row,
                            const int32_t* pos, const void* k_new, const void* v_new,
                            void* k_pages, float* k_scale, void* v_pages, float* v_scale,
                            const int32_t* table, hipStream_t stream);

/* Make room for count[i] more tokens of row[i], and count them: the pages
 * that positions lengths .. lengths + count - 1 newly need are taken from the
 * free ones, lowest ids first, in list order, entered into the table with
 * refs = 1, and lengths grows by count.  ok[i] = 1, or 0 with the row left as
 * it was: a row outside [0, rows) or listed before, a negative count, a table
 * row too short, or an entry that needs pages when the pages needed by the
 * list up to and including it exceed the free ones.  n <= 4096. */
misa_status misa_page_extend(const misa_cache* cache, int32_t n, const int32_t* row,
                             const int32_t* count, int32_t* table, int32_t* lengths,
                             int32_t* refs, int32_t* ok, hipStream_t stream);

/* Fork rows: child[i] becomes a sequence with the tokens of parent[i].  Pages
 * that the parent has filled are shared (refs + 1); a partly filled last page
 * is replaced by a free one (lowest ids first, in list order), and the pair to
 * copy is written to src[i], dst[i] for misa_page_copy (-1, -1: nothing to
 * copy), so that both rows can go on to write.  ok[i] = 1, or 0 with the child
 * left as it was: a row outside [0, rows), a child that is not empty (lengths
 * != 0), is listed before or is its own parent, or -- when a page is needed --
 * no free page left, counted as in misa_page_extend.  Parents are read as
 * they were before the call.
 *   parent, child, src, dst, ok  [n]  int32; n <= 4096 */
misa_status misa_page_fork(const misa_cache* cache, int32_t n, const int32_t* parent,
                           const int32_t* child, int32_t* table, int32_t* lengths, int32_t* refs,
                           int32_t* src, int32_t* dst, int32_t* ok, hipStream_t stream);

/* Free rows: refs of the pages that hold the row's tokens falls by one, their
 * table entries become -1 and lengths 0.  A row listed twice is freed once; n
 * <= 4096. */
misa_status misa_page_free(const misa_cache* cache, int32_t n, const int32_t* row, int32_t* table,
                           int32_t* lengths, int32_t* refs, hipStream_t stream);

/* Compact the pool: with `live` pages in use, the i-th live page with id >=
 * live (ascending) moves to the i-th free id < live, so that pages 0 .. live-1
 * are the ones in use and the pool can be cut there.
 *   map        [pages]  int32, written: each page's id afterwards, -1 = free
 *   live       [1]      int32, written
 *   src, dst   [max(1, pages / 2)]  int32, written: the moves, for
 *              misa_page_copy, then -1
 *   table_out, refs_out  written: table and refs with the new ids (they may
 *              be the same arrays as table and refs); entries that name a free
 *              page become -1
 * Rows and lengths stay as they are.  ws must hold
 * misa_page_workspace_bytes(cache) bytes. */
size_t misa_page_workspace_bytes(const misa_cache* cache);
misa_status misa_page_compact(const misa_cache* cache, const int32_t* table, const int32_t* refs,
                              int32_t* table_out, int32_t* refs_out, int32_t* map, int32_t* live,
                              int32_t* src, int32_t* dst, void* ws, size_t ws_bytes,
                              hipStream_t stream);

/* One buffer of pages: `planes` (layers, say) of `pages` pages of page_bytes
 * bytes each, [planes, pages, page_bytes]. */
typedef struct {
  void* data;
  int64_t page_bytes; /* a positive multiple of 4, at most 2^31 */
  int32_t planes;     /* 1 .. 65536 */
} misa_page_buffer;

/* Copy page src[i] onto page dst[i], i < n, in every plane of n_buffers (1 ..
 * 8) buffers of `pages` pages each.  `buffers` is a HOST array.  Pairs with an
 * id outside [0, pages) are skipped; a page written by one pair must not be
 * read or written by another. */
misa_status misa_page_copy(const misa_page_buffer* buffers, int32_t n_buffers, int32_t pages,
                           int32_t n, const int32_t* src, const int32_t* dst, hipStream_t stream);

/* Root-mean-square norm of rows, with the residual's addition before it and an
 * 8-bit output after it.  Per row of n elements in `groups` equal parts:
 *   y = x + residual,   z_part = y_part / sqrt(mean(y_part^2) + eps) * weight,
 *   out = z, or e4m3 codes of z with one scale per row.
 * groups = 1 is the norm of a residual stream or of the indexer's keys (n = d:
 * out and out_scale are misa_*'s k and k_scale); groups = H with n = H * d
 * norms each head by itself and gives the indexer's q and q_scale.
 *   x, residual  [rows, n]  x_dtype (MISA_F32 or MISA_BF16); residual may be NULL
 *   weight       [n / groups]  fp32
 *   sum_out      [rows, n]  x_dtype, y, written if non-NULL (may be x or residual)
 *   out          [rows, n]  out_dtype (any misa_dtype), written
 *   out_scale    [rows]     fp32, written (fp8 only, else ignored)
 * out must not overlap the inputs or sum_out.  fp32 throughout: a part's mean
 * square plus eps must be in fp32's normal range (an all-zero part with eps = 0
 * gives NaN), and results between 2^-110 and 2^112 in magnitude, or zero, have its
 * full precision.  0 <= rows < 2^24 (0: no-op), 1 <= n <= 32768, groups divides n,
 * eps >= 0. */
misa_status misa_rms_norm(int32_t rows, int32_t n, int32_t groups, int32_t x_dtype,
                          int32_t out_dtype, float eps, const void* x, const void* residual,
                          const float* weight, void* sum_out, void* out, float* out_scale,
                          hipStream_t stream);

/* ------------------------------------------------------------ rotary positions */

typedef enum {
  MISA_ROPE_HALF = 0,       /* pair i: elements i and i + rot/2 of the rotated part */
  MISA_ROPE_INTERLEAVED = 1 /* pair i: elements 2i and 2i + 1                       */
} misa_rope_pairs;

/* What misa_rope turns: heads of d elements, of which first .. first + rot - 1
 * are rotated in rot / 2 pairs; the others pass.  x_stride and out_stride are
 * elements from one token to the next, so that the heads may be a part of a
 * wider row (the queries and keys of a fused projection).  amplitude multiplies
 * the rotated part. */
typedef struct {
  int32_t heads, d, first, rot;
  int32_t pairs;             /* a misa_rope_pairs */
  int32_t x_dtype, out_dtype;
  float amplitude;
  int64_t x_stride, out_stride;
} misa_rope_spec;

/* Rotary positions.  Pair i of a head of token t, (a, b), becomes
 *   amplitude * (a cos - b sin, a sin + b cos)  of the angle pos[t] * freq[i].
 * The angle is a product in 64 bits, reduced to one turn there: 2^-50 of itself,
 * at any position.
 *   x     [n, heads, d], x_stride apart    MISA_F32 or MISA_BF16
 *   pos   [n]        int32, any sign
 *   freq  [rot / 2]  fp64, radians a position (misa_rope_frequencies)
 *   out   [n, heads, d], out_stride apart  MISA_F32, MISA_BF16 or MISA_FP8_E4M3,
 *         written; may be x itself (same type and stride)
 *   out_scale  [n]   fp32, written (fp8 only, else ignored): one scale per token
 *         over its heads, amax / 448, as misa_*'s q_scale and k_scale; a code is the
 *         value divided by it (in fp32), rounded to nearest even
 * 0 <= n < 2^24 (0: no-op); 1 <= heads, heads * d <= 32768; rot even, 0 < rot <=
 * 1024, first + rot <= d; strides of at least heads * d (out_stride of an fp8 out
 * exactly that) and below 2^31; rotated values in fp32's normal range. */
misa_status misa_rope(const misa_rope_spec* spec, int32_t n, const void* x, const int32_t* pos,
                      const double* freq, void* out, float* out_scale, hipStream_t stream);

typedef enum {
  MISA_ROPE_PLAIN = 0,  /* f_i = base^(-2i / rot)                                */
  MISA_ROPE_LINEAR = 1, /* f_i / factor: positions drawn together                */
  MISA_ROPE_PARTS = 2   /* by parts: slow pairs as LINEAR, fast ones as PLAIN    */
} misa_rope_kind;

/* Frequencies for contexts longer than the trained one.  MISA_ROPE_PARTS ("YaRN:
 * Efficient Context Window Extension of Large Language Models", section 3.2):
 * pairs that turn `fast` times and more in `original` positions keep f_i, those
 * that turn `slow` times and fewer have f_i / factor, with a linear ramp over i
 * between, from the last whole i that turns `fast` times (or 0) to the first that turns
 * `slow` times, beyond the last pair if need be (rot - 1 at most); and an amplitude of
 * 1 + 0.1 ln(factor). */
typedef struct {
  int32_t kind, rot; /* a misa_rope_kind; rot as in misa_rope_spec */
  double base;       /* > 1 */
  double factor;     /* >= 1; LINEAR and PARTS */
  double original;   /* > 0, positions; PARTS, like fast >= slow > 0 */
  double fast, slow;
} misa_rope_scaling;

/* Runs on the HOST: fills freq[0 .. rot/2 - 1] (host memory, to be copied to the
 * device once) and *amplitude. */
misa_status misa_rope_frequencies(const misa_rope_scaling* scaling, double* freq,
                                  float* amplitude);

/* ------------------------------------------- a cache with one scale per block
 * The paged cache above with e4m3 codes and ONE scale for each block of
 * block_tokens tokens of a page and kv head:
 *   k_pages, v_pages  [pages, kv_heads, page_tokens, d]   e4m3 codes
 *   k_scale, v_scale  [pages, kv_heads, page_tokens / block_tokens]  fp32
 * cache->kv_dtype is MISA_FP8_E4M3, dk = dv in {64, 128, 256}; block_tokens is 16,
 * 32, 64 or 128 and divides page_tokens; rows <= 65535.  The table, lengths and refs
 * and the calls that keep them (misa_page_extend, ..fork, ..free, ..compact,
 * ..copy) are those of misa_cache; codes and scales are buffers of misa_page_copy.
 *
 * A scale is a power of two: the smallest 2^e, e >= -100, with amax <= 448 * 2^e
 * over the finite values that the block got so far.  misa_block_write leaves such
 * scales, and misa_block_attend takes no others.  A code is x / scale rounded
 * to nearest even; infinities and NaN become NaN codes and set no scale.
 *
 * Batches of rows come packed: offsets [rows + 1] int32, ascending; entries
 * offsets[r] .. offsets[r+1] - 1 of the packed arrays belong to row r, whose
 * number may be zero.  Entries before offsets[0] and from offsets[rows] on
 * (padding of a captured batch) are not read and their outputs left as they were.
 * New tokens are the last ones of their row: with c of them, token i of row r is at
 * position lengths[r] - c + i (misa_page_extend has counted them). */

/* Write the rows' new tokens.  The first of them may go on in a block that holds
 * earlier tokens: the block keeps its scale, or, where the new ones are louder,
 * gets a larger one and its codes are rounded to that (exact but for codes that
 * become subnormal).  What the block held at and behind the new tokens'
 * positions counts for nothing but its scale.  Positions outside the table or
 * without a page are skipped.  Rows must not share a block that is written
 * (misa_page_fork sees to that).
 *   k_new, v_new  [n, kv_heads, d]  bf16; v_new, v_pages and v_scale all NULL: a
 *                 cache of keys alone (the indexer's)
 * n = 0 is a no-op; n * kv_heads <= 2^25. */
misa_status misa_block_write(const misa_cache* cache, int32_t block_tokens, int32_t n,
                             const int32_t* offsets, const int32_t* lengths, const void* k_new,
                             const void* v_new, void* k_pages, float* k_scale, void* v_pages,
                             float* v_scale, const int32_t* table, hipStream_t stream);

/* Read rows back: packed entry i of row r is its token first[r] + i - offsets[r]
 * (first NULL: from token 0).  Tokens outside [0, lengths[r]) or without a page
 * read as zeros (scale 1).
 *   first         [rows] int32 or NULL
 *   k_out, v_out  [n, kv_heads, d]  out_dtype (any misa_dtype), written: code *
 *                 scale, rounded once (exact in bf16 down to its subnormals); fp8:
 *                 the codes, with
 *   k_out_scale, v_out_scale  [n, kv_heads]  fp32, written (fp8 only, else
 *                 ignored).  With one kv head of 128 and rows of L tokens (offsets
 *                 r * L) these are misa_*'s k and k_scale.
 * Keys alone: v_pages, v_scale, v_out and v_out_scale NULL.  n = 0 is a no-op; n *
 * kv_heads <= 2^27. */
misa_status misa_block_read(const misa_cache* cache, int32_t block_tokens, int32_t n,
                            int32_t out_dtype, const int32_t* offsets, const int32_t* first,
                            const int32_t* lengths, const void* k_pages, const float* k_scale,
                            const void* v_pages, const float* v_scale, const int32_t* table,
                            void* k_out, float* k_out_scale, void* v_out, float* v_out_scale,
                            hipStream_t stream);

/* Attention of the rows' new tokens (one of each row, drafts, a prompt's chunk)
 * over the block-scaled cache that holds them already, causal:
 *   o[i, j, :] = sum_s p_s v[r, s, g, :],  p = softmax_s(scale * q[i,j,:] . k[r,s,g,:]),
 *   lse[i, j] = log sum_s exp(scale * q . k),   g = j / (heads / kv_heads),
 * over the tokens s of row r up to the query's own position, or with k > 0 those
 * of them that idx[i, :] lists (any order, -1 padded, as the indexer's entry points
 * write it).  Tokens whose table entry names no page are not visible.  A query
 * without visible tokens gets o = 0 and lse = -INFINITY.  What the cache holds at
 * invisible slots is never used, NaN or not.
 *   most  the largest number of new tokens of a row: it picks the kernel and sizes
 *         the workspace, and no result depends on it but by roundings
 *   q    [n, heads, d]  bf16         out [n, heads, d]  bf16, written
 *   idx  [n, k]  int32 (k > 0; k = 0: NULL)
 *   lse  [n, heads]  fp32, written if non-NULL
 * Scores, softmax and sums are fp32: q . k, q . codes and a score times log2(e) must
 * be in its range, and cached values below 2^90.  A weight goes into its products
 * in 16 bits where queries are worked on one by one (one new token a row, or lists);
 * where several share a pass in 11 bits, or to 2^-32 of the largest weight times the
 * largest value that the loudest block may hold of those that the query sees.  Limits: heads a multiple of
 * kv_heads, heads <= 1024, n <= 2^20, n * heads <= 2^26 (2^23 one by one; otherwise
 * rows * kv_heads <= 2^23), 0 <= k <= 2^20, |scale| <= 2^127.  ws must hold misa_block_attend_workspace_bytes(...) bytes (0: invalid
 * arguments or no workspace needed); it carries nothing from one call to the next. */
size_t misa_block_attend_workspace_bytes(const misa_cache* cache, int32_t block_tokens,
                                         int32_t heads, int32_t n, int32_t most, int32_t k);
misa_status misa_block_attend(const misa_cache* cache, int32_t block_tokens, int32_t heads,
                              int32_t n, int32_t most, int32_t k, float scale,
                              const int32_t* offsets, const void* q, const void* k_pages,
                              const float* k_scale, const void* v_pages, const float* v_scale,
                              const int32_t* table, const int32_t* lengths, const int32_t* idx,
                              void* out, float* lse, void* ws, size_t ws_bytes,
                              hipStream_t stream);

/* A static, human-readable name of a status code. */
const char* misa_status_string(misa_status status);

#ifdef __cplusplus
}
#endif

#endif /* MISA_H */
