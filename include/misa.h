/*
 * misa.h -- C ABI of the MISA (Mixture of Indexer Sparse Attention) indexer
 * for AMD Instinct MI355X (gfx950).
 *
 * The indexer picks, for every query token, the top-k prefix tokens that
 * DSA-style sparse attention will attend to.  MISA replaces the dense
 * all-head DSA indexer with four stages (gist.science technical summary of
 * "MISA: Mixture of Indexer Sparse Attention for Long-Context LLM Inference",
 * "Metodologia: MISA" items 1-2; agents-report summary, method overview):
 *
 *   misa_pool_keys          block mean-pooling of the shared indexer keys
 *   misa_route_heads        block-summary router: top-h indexer heads per query
 *   misa_sparse_head_logits token scoring with the routed heads only
 *   misa_topk               per-query top-k token selection
 *
 * plus the whole pipeline (misa_indexer, optionally the hierarchical
 * MISA-dagger variant of "Variante Hierárquica (MISA†)") and the dense DSA
 * indexer that MISA replaces (dsa_dense_logits; the baseline path named in
 * the GitHub issue "Clarification on the Figure 3 baseline ...").
 *
 * Token score (the DSA indexer score, DeepSeek-V3.2 lightning indexer):
 *     I[t, s] = sum_{j in heads(t)} w[t, j] * ReLU(q[t, j] . k[s] * sigma[s])
 * for every prefix key s <= t, and -inf for s > t.  sigma[s] is the per-token
 * scale of an fp8 key cache and 1 for bf16 keys.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Memory   All tensor pointers are DEVICE pointers owned by the caller.  The
 *          library never allocates, frees or synchronises; scratch space comes
 *          from a caller-provided workspace (misa_indexer_noalloc: from a fixed
 *          device buffer of the library).  Every tensor is densely
 *          packed in the layout given (row-major, last index fastest) and
 *          16-byte aligned.
 * Streams  `stream` is a hipStream_t passed as void* (NULL = the default
 *          stream).  Every call only enqueues work on it and returns.
 * Errors   Arguments are checked on the host before anything is enqueued; a
 *          bad argument returns a negative misa_status and enqueues nothing.
 *          A failed kernel launch returns MISA_ERR_HIP.  No C++ exception
 *          crosses this interface.  The only global state is the per-device
 *          address of misa_indexer_noalloc's fixed scratch (looked up once
 *          under a lock), so calls from several host threads are safe, except
 *          that misa_indexer_noalloc calls sharing one GPU must not overlap.
 * Numerics Preconditions that are documented, not checked: inputs are finite;
 *          fp8 scales are > 0.  Accumulation is fp32.
 * Shapes   A call covers n_seq independent sequences.  Sequence b has n_keys
 *          keys (positions 0..n_keys-1) and q_per_seq queries; query i of a
 *          sequence sits at absolute position t = q_pos0 + i and sees the keys
 *          0..t (causal).  Prefill chunk: n_seq = 1, q_pos0 = n_keys - M.
 *          Decode batch: q_per_seq = 1, q_pos0 = n_keys - 1.
 * Blocks   Block m covers key positions [m*B, (m+1)*B).  For query t the
 *          prefix holds floor((t+1)/B) complete blocks and, when (t+1) % B != 0,
 *          one partial block [floor((t+1)/B)*B, t] (its "tail").
 */
#ifndef MISA_H
#define MISA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MISA_OK = 0,
  MISA_ERR_INVALID_ARG = -1,   /* null pointer, bad size, bad alignment */
  MISA_ERR_UNSUPPORTED = -2,   /* a valid request outside what is implemented */
  MISA_ERR_WORKSPACE = -3,     /* workspace missing or too small */
  MISA_ERR_HIP = -4,           /* a HIP runtime call or kernel launch failed */
  MISA_ERR_SCRATCH = -5        /* misa_indexer_noalloc: more scratch needed than
                                  MISA_NOALLOC_SCRATCH_BYTES */
} misa_status;

typedef enum {
  MISA_K_BF16 = 0,             /* k: uint16 bf16 bits [n_seq][n_keys][128] */
  MISA_K_FP8_E4M3 = 1          /* k: uint8 OCP e4m3fn codes [n_seq][n_keys][128],
                                  k_scale: float [n_seq][n_keys], > 0 */
} misa_kdtype;

typedef struct {
  int32_t n_seq;      /* independent sequences, >= 1 */
  int32_t q_per_seq;  /* M: queries per sequence, >= 0 (0 = nothing to do) */
  int64_t n_keys;     /* N: keys per sequence, 1..2^26 (larger: MISA_ERR_UNSUPPORTED) */
  int64_t q_pos0;     /* position of query 0; 0 <= q_pos0 and q_pos0 + M <= N */
  int32_t n_heads;    /* H: indexer heads (H_I on the pages), 1..64 */
  int32_t head_dim;   /* d: must be 128 */
  int32_t block;      /* B: pooling block size, >= 1 */
} misa_shape;

#define MISA_HEAD_DIM 128
#define MISA_MAX_HEADS 64
#define MISA_MAX_TOPK 8192

/* Human-readable name of a status code (static string, never NULL). */
const char* misa_status_str(misa_status s);

/*
 * Block mean-pooling of the shared indexer keys (gist.science summary,
 * "Metodologia: MISA" item 1: mean-pooled indexer keys per block;
 * agents-report: one summary key per block of the prefix).
 *   pooled[b][m][:] = mean(key[b][m*B .. m*B+B-1][:])   for m < floor(N/B)
 *   tail[b][i][:]   = mean(key[b][floor((t+1)/B)*B .. t][:]),  t = q_pos0+i,
 *                     or all zeros when (t+1) % B == 0 (no partial block).
 * key = bf16 value, or e4m3 value * k_scale.  fp32 sums in key order.
 * k: see misa_kdtype.  k_scale: NULL for bf16, required for fp8.
 * pooled: float [n_seq][floor(N/B)][128] (not touched when floor(N/B) = 0).
 * tail:   float [n_seq][M][128].
 */
misa_status misa_pool_keys(const misa_shape* shape, const void* k, misa_kdtype kdtype,
                           const float* k_scale, float* pooled, float* tail, void* stream);

/*
 * Head router (gist.science summary, "Metodologia: MISA" item 1: per-head
 * affinities against the pooled keys, aggregated into a per-head importance,
 * top-h heads kept; agents-report: MISA aggregates along the blocks to pick
 * heads).  For query t of sequence b and head j:
 *   S[j] = sum_{m < floor((t+1)/B)} ReLU(q[t,j] . pooled[m]) + ReLU(q[t,j] . tail[t])
 *          (the tail term only when the partial block is non-empty)
 *   r[j] = w[t,j] * S[j]
 *   heads[b][i][:] = the h heads with the largest r (equal r -> lower head id),
 *                    stored in ascending head order.
 * q: uint16 bf16 bits [n_seq][M][H][128].  w: float [n_seq][M][H].
 * pooled, tail: as written by misa_pool_keys.  1 <= h <= H.
 * heads: int32 [n_seq][M][h].  scores: float [n_seq][M][H] receives r, or NULL.
 */
misa_status misa_route_heads(const misa_shape* shape, const uint16_t* q, const float* w,
                             const float* pooled, const float* tail, int32_t h,
                             int32_t* heads, float* scores, void* stream);

/*
 * Token scoring with the routed heads only (gist.science summary,
 * "Metodologia: MISA" item 2: only the h active heads score the whole prefix
 * token by token).
 *   logits[b][i][s] = sum_{j in heads[b][i]} w[t,j] * ReLU(q[t,j] . k[s] * sigma[s])
 *                     for s <= t,   -inf for t < s < N.   Columns N..roundup4(N)-1
 *                     may also be set to -inf; columns roundup4(N)..ld-1 are untouched.
 * heads: int32 [n_seq][M][h], ascending, distinct, each in [0, H).  1 <= h <= H.
 * logits: float [n_seq][M][ld]; ld >= N, ld % 4 == 0 and ld <= 2^27 (larger:
 *         MISA_ERR_UNSUPPORTED; row offsets of a 4-row group stay 32-bit).
 */
misa_status misa_sparse_head_logits(const misa_shape* shape, const uint16_t* q, const float* w,
                                    const void* k, misa_kdtype kdtype, const float* k_scale,
                                    const int32_t* heads, int32_t h, float* logits, int64_t ld,
                                    void* stream);

/*
 * The dense DSA indexer: the token score with all H heads (the baseline MISA
 * replaces; the abstract of arXiv 2605.07363 and the GitHub issue's dense
 * all-head path).
 * cand == NULL:  logits[b][i][s] over every key, exactly as
 *                misa_sparse_head_logits with heads = 0..H-1 (and bitwise equal
 *                to it); ld >= N, ld % 4 == 0, ld <= 2^27.
 * cand != NULL:  re-rank mode of MISA-dagger ("Variante Hierárquica (MISA†)":
 *                the original all-head indexer re-scores only the candidates).
 *                cand: int32 [n_seq][M][n_cand] token ids (any order; -1 = no
 *                candidate); logits[b][i][c] = score of token cand[b][i][c]
 *                (-inf where cand < 0); ld >= n_cand, ld % 4 == 0.  Every
 *                candidate id must be in [0, t].  Each value is bitwise equal
 *                to the cand == NULL value of the same (query, token).
 */
misa_status dsa_dense_logits(const misa_shape* shape, const uint16_t* q, const float* w,
                             const void* k, misa_kdtype kdtype, const float* k_scale,
                             const int32_t* cand, int32_t n_cand, float* logits, int64_t ld,
                             void* stream);

/*
 * Per-query top-k token selection (the selection step after scoring; the
 * issue's pipeline runs it as a separate top-k over the returned logits).
 * Order: value descending; equal values (with -0.0 == +0.0) -> lower token id.
 * cand == NULL:  row i of sequence b considers columns s in [0, min(n_cols, t+1));
 *                the token id is the column.
 * cand != NULL:  row considers columns c in [0, n_cols) with cand[b][i][c] >= 0;
 *                the token id is cand[b][i][c] (ids distinct within a row).
 * sorted != 0: idx lists the selection in that order.  sorted == 0: the same set in an
 *                unspecified order (enough for a candidate list), cheaper.
 * idx:  int32 [n_seq][M][k]; rows with fewer than k candidates are padded with -1 (the
 *       padding always comes last).
 * vals: float [n_seq][M][k] (the selected values, -inf padding), or NULL.
 * 1 <= k <= MISA_MAX_TOPK.  logits: float [n_seq][M][ld], ld % 4 == 0, ld >= n_cols.
 * ws / ws_bytes: workspace of at least misa_topk_workspace_bytes() bytes
 *                (may be NULL when that is 0).
 */
misa_status misa_topk(const misa_shape* shape, const float* logits, int64_t ld,
                      const int32_t* cand, int32_t n_cols, int32_t k, int32_t sorted,
                      int32_t* idx, float* vals, void* ws, size_t ws_bytes, void* stream);

size_t misa_topk_workspace_bytes(const misa_shape* shape, int32_t n_cols, int32_t k);

/*
 * Routed-head scoring and top-k token selection in one call, without
 * materialising the logits where that can be avoided (the fused scoring ->
 * top-k the GitHub issue asks for as a "fused MISA kernel").  The result is
 * exactly misa_topk(misa_sparse_head_logits(...), topk, sorted): same ids,
 * same values, same order (sorted != 0) or the same set (sorted == 0).
 * When h <= 8, topk <= 8192 and every query's prefix has at least
 * max(16384, 4 topk) keys, the scores of
 * a key sample (every kstride-th key, kstride >= 32) give each row a
 * threshold; the routed scoring keeps only the scores at or above it, as
 * candidates, and the exact top-k is taken over them.  A row whose
 * candidates fall short of topk (or overflow their buffers) is re-scored into
 * full logits in the workspace and selected from them, so the result does
 * not depend on the sample.  Otherwise the logits are materialised in the
 * workspace and misa_topk runs on them.
 * heads: int32 [n_seq][M][h], as misa_sparse_head_logits.  idx / vals: as
 * misa_topk.  1 <= topk <= MISA_MAX_TOPK.
 * ws / ws_bytes: at least misa_sparse_head_topk_workspace_bytes() bytes.
 */
misa_status misa_sparse_head_topk(const misa_shape* shape, const uint16_t* q, const float* w,
                                  const void* k, misa_kdtype kdtype, const float* k_scale,
                                  const int32_t* heads, int32_t h, int32_t topk, int32_t sorted,
                                  int32_t* idx, float* vals, void* ws, size_t ws_bytes, void* stream);

/* Workspace of misa_sparse_head_topk for keys of type kdtype (fp8 keys add a
 * bf16 copy of the keys, widened exactly once per call for the scoring's
 * direct global -> LDS staging); 0 for an invalid shape. */
size_t misa_sparse_head_topk_workspace_bytes(const misa_shape* shape, misa_kdtype kdtype, int32_t h,
                                             int32_t topk);

/*
 * fp8 path.  The pages' indexer runs on fp8 inputs, and the GitHub issue on
 * the vLLM kernel ("Clarification on the Figure 3 baseline and plans for an
 * optimized vLLM MISA kernel", second question) asks for an fp8 MISA kernel
 * that avoids widening fp8 to bf16.  These calls score with fp8 queries and
 * fp8 keys on the fp8 matrix cores; the result is the routed score of the
 * dequantised inputs (within the scoring tolerance: the fp8 MFMA accumulates
 * at slightly less than fp32 precision).
 *
 * misa_quantize_q: per (query, head) row of 128 values,
 *   q_scale = fp32(amax / 448), amax = max |q| over the row (1 for a zero row),
 *   q8      = e4m3fn round-to-nearest-even of fp32(q / q_scale),
 * both divisions correctly rounded (448 is the largest finite e4m3fn value).
 * q: bf16 [n_seq][M][H][128] (16-byte aligned); q8: uint8 [n_seq][M][H][128]
 * (16-byte aligned); q_scale: float [n_seq][M][H].
 */
misa_status misa_quantize_q(const misa_shape* shape, const uint16_t* q, uint8_t* q8, float* q_scale,
                            void* stream);

/*
 * misa_sparse_head_logits on fp8 queries (misa_quantize_q's q8 and q_scale):
 *   I[t,s] = sigma[s] * sum_{j in heads(t)} w[t,j] * q_scale[t,j] * ReLU(q8[t,j] . k8[s])
 * for s <= t, -inf after (the q and key codes taken as e4m3fn values).
 * kdtype must be MISA_K_FP8_E4M3 (MISA_ERR_UNSUPPORTED otherwise), and
 * 1 <= h <= 8 (MISA_ERR_UNSUPPORTED above 8).  Other arguments as
 * misa_sparse_head_logits; columns N .. roundup4(N)-1 may be set to -inf.
 */
misa_status misa_sparse_head_logits_q8(const misa_shape* shape, const uint8_t* q8, const float* q_scale,
                                       const float* w, const void* k, misa_kdtype kdtype, const float* k_scale,
                                       const int32_t* heads, int32_t h, float* logits, int64_t ld,
                                       void* stream);

/*
 * dsa_dense_logits on fp8 queries, every key (the fp8-query dense DSA
 * indexer, the production-style comparator of the GitHub issue's Figure 3
 * discussion, whose dense path scores fp8 queries and keys):
 *   D[t,s] = sigma[s] * sum_{j < H} w[t,j] * q_scale[t,j] * ReLU(q8[t,j] . k8[s])
 * for s <= t, -inf after.  kdtype must be MISA_K_FP8_E4M3
 * (MISA_ERR_UNSUPPORTED otherwise).  logits: float [n_seq][M][ld], ld >= N,
 * ld % 4 == 0, 16-byte aligned; columns N .. roundup4(N)-1 may be set to -inf.
 */
misa_status dsa_dense_logits_q8(const misa_shape* shape, const uint8_t* q8, const float* q_scale, const float* w,
                                const void* k, misa_kdtype kdtype, const float* k_scale, float* logits, int64_t ld,
                                void* stream);

/*
 * misa_sparse_head_topk on fp8 queries: exactly
 * misa_topk(misa_sparse_head_logits_q8(...), topk) (ids, values and order;
 * the set when sorted == 0), through the same fused path (logits only for
 * the rows the candidates cannot settle).  The second question of the GitHub
 * issue asks for an fp8 MISA kernel with the top-k overhead cut; this is it.
 * kdtype must be MISA_K_FP8_E4M3 and 1 <= h <= 8 (MISA_ERR_UNSUPPORTED
 * otherwise).  The workspace is misa_sparse_head_topk_workspace_bytes(shape,
 * MISA_K_FP8_E4M3, h, topk) bytes (16-byte aligned; the fp8 keys feed the
 * fp8 matrix cores as they are, so part of it stays unused).  Other arguments
 * as misa_sparse_head_topk.
 */
misa_status misa_sparse_head_topk_q8(const misa_shape* shape, const uint8_t* q8, const float* q_scale,
                                     const float* w, const void* k, misa_kdtype kdtype, const float* k_scale,
                                     const int32_t* heads, int32_t h, int32_t topk, int32_t sorted, int32_t* idx,
                                     float* vals, void* ws, size_t ws_bytes, void* stream);

/*
 * The whole indexer on the caller's stream: pool -> route -> routed scoring ->
 * top-k (k_prime == 0, MISA), or pool -> route -> routed scoring -> top-k' ->
 * all-head re-rank of the k' candidates -> top-k (k_prime >= topk, MISA-dagger;
 * "Variante Hierárquica (MISA†)" of the gist.science summary).
 * idx: int32 [n_seq][M][topk], vals: float [n_seq][M][topk] or NULL.
 * 1 <= h <= H; 1 <= topk <= MISA_MAX_TOPK; k_prime == 0 or topk <= k_prime <= MISA_MAX_TOPK.
 * ws / ws_bytes: the workspace (16-byte aligned) holds the pooled keys,
 * tails, routed heads, sampled scores, candidate regions and the logits rows
 * of rows the candidates cannot settle.  misa_indexer_workspace_bytes() bytes
 * is the fast plan (every such row re-scored in one pass); any size down to
 * misa_indexer_workspace_min_bytes() also works, with the same result: the
 * plan is taken from ws_bytes, the re-scoring then runs through a smaller
 * logits slab, a batch of query tiles at a time (two more launches per
 * batch), and candidate regions may be sized closer to the expected
 * candidates.  Below the minimum: MISA_ERR_WORKSPACE, nothing enqueued.
 */
misa_status misa_indexer(const misa_shape* shape, const uint16_t* q, const float* w, const void* k,
                         misa_kdtype kdtype, const float* k_scale, int32_t h, int32_t topk,
                         int32_t k_prime, int32_t* idx, float* vals, void* ws, size_t ws_bytes,
                         void* stream);

/* Workspace of misa_indexer's fast plan for keys of type kdtype; 0 for an
 * invalid shape. */
size_t misa_indexer_workspace_bytes(const misa_shape* shape, misa_kdtype kdtype, int32_t h, int32_t topk,
                                    int32_t k_prime);

/* The least workspace misa_indexer takes (its lean plan: a logits slab no
 * larger than the sampled scores, which it shares memory with, and tighter
 * candidate regions); 0 for an invalid shape.  E.g. about 0.94 GiB for
 * 8192 queries over 131072 fp8 keys, h = 8, topk = 2048, against 6 GiB for
 * the fast plan. */
size_t misa_indexer_workspace_min_bytes(const misa_shape* shape, misa_kdtype kdtype, int32_t h, int32_t topk,
                                        int32_t k_prime);

/*
 * misa_indexer for callers that cannot allocate device memory (code under HIP
 * graph capture, tight serving loops, harnesses that forbid allocation): the
 * same arguments and the same result as misa_indexer, but no workspace
 * argument.  Its scratch is a fixed device buffer of the library,
 * MISA_NOALLOC_SCRATCH_BYTES (256 MiB) per GPU, held until the process ends,
 * planned as a workspace of that size (see misa_indexer); a request whose
 * misa_indexer_workspace_min_bytes() exceeds it returns MISA_ERR_SCRATCH and
 * enqueues nothing (256 MiB holds, e.g., a decode batch of 64 sequences x
 * 131072 keys, or a prefill chunk of 512 queries over 65536 keys).  The call allocates, frees and synchronises nothing.  All
 * calls on one GPU share that GPU's buffer, which keeps the last call's
 * contents: calls that may overlap on one GPU (several streams, several host
 * threads) race, so the caller must order them (one stream, or events).
 * The first call on a device looks up the buffer's device address; later calls
 * reuse it.
 */
#define MISA_NOALLOC_SCRATCH_BYTES ((size_t)256 << 20)
misa_status misa_indexer_noalloc(const misa_shape* shape, const uint16_t* q, const float* w, const void* k,
                                 misa_kdtype kdtype, const float* k_scale, int32_t h, int32_t topk,
                                 int32_t k_prime, int32_t* idx, float* vals, void* stream);

/*
 * misa_indexer with fp8 queries for the routed scoring: pool -> route (bf16
 * q) -> misa_quantize_q into the workspace -> misa_sparse_head_topk_q8 (the
 * k' candidates when k_prime > 0, then the MISA-dagger re-rank with bf16 q
 * and all heads, as misa_indexer).  The result is exactly that sequence of
 * calls.  kdtype must be MISA_K_FP8_E4M3 and 1 <= h <= 8
 * (MISA_ERR_UNSUPPORTED otherwise); other arguments as misa_indexer; ws: at
 * least misa_indexer_q8_workspace_bytes() bytes.
 */
misa_status misa_indexer_q8(const misa_shape* shape, const uint16_t* q, const float* w, const void* k,
                            misa_kdtype kdtype, const float* k_scale, int32_t h, int32_t topk, int32_t k_prime,
                            int32_t* idx, float* vals, void* ws, size_t ws_bytes, void* stream);

size_t misa_indexer_q8_workspace_bytes(const misa_shape* shape, int32_t h, int32_t topk, int32_t k_prime);

/*
 * Paged key cache -> the contiguous keys every call here reads.  Serving
 * engines keep the indexer keys in pages of page_keys keys named by a
 * per-sequence block table (the GitHub issue's per-layer boundary includes
 * this cache handling).  Key s of sequence b is row s % page_keys of page
 * block_table[b * max_pages + s / page_keys]; the call writes keys
 * [0, n_keys) of every sequence to k_out [n_seq][n_keys][128] (16-byte
 * aligned) and, for fp8, their scales to scale_out [n_seq][n_keys].
 * k_pages: [n_pages][page_keys][128] bf16 or e4m3 codes (16-byte aligned),
 * scale_pages: [n_pages][page_keys] (fp8 only).  max_pages >=
 * ceil(n_keys / page_keys).  Page ids outside [0, n_pages) are a
 * precondition violation: those keys are written as zeros (scale 1), never
 * read.  HBM-bound: 2 x the keys' bytes.
 */
misa_status misa_gather_keys_paged(const misa_shape* shape, const void* k_pages, misa_kdtype kdtype,
                                   const float* scale_pages, const int32_t* block_table, int64_t max_pages,
                                   int64_t n_pages, int32_t page_keys, void* k_out, float* scale_out, void* stream);

/*
 * Pooled-key cache (chunked prefill and decode).  The GitHub issue measures
 * the indexer at a per-layer boundary that includes cache handling, under
 * chunked prefill of 8192 tokens up to a 128K prompt ("Clarification on the
 * Figure 3 baseline ...", the measured configuration).  Block means of keys
 * already pooled do not change as the sequence grows, so a caller-owned
 * cache keeps them across calls and each call pools only the blocks that
 * have become complete since (decode then reads K once per step instead of
 * twice).
 *
 * The cache of a shape's n_seq sequences, caller-owned device memory:
 *   pooled:       float    [n_seq][cap_blocks][128]     block means
 *   pooled_split: uint16_t [n_seq][2][cap_blocks][128]  their bf16 hi rows, then
 *                 lo rows (pooled - hi), which the router stages directly
 * both 16-byte aligned, cap_blocks >= n_keys / block.  n_cached: the number of
 * leading complete blocks whose rows already hold the means of these keys
 * (0 for an empty cache; after a call with n_keys keys the cache holds
 * n_keys / block blocks).  0 <= n_cached <= n_keys / block, else
 * MISA_ERR_INVALID_ARG.  The keys of the cached blocks are not read again,
 * so they must be the keys the cache was built from.
 */

/* misa_pool_keys into the cache: pools complete blocks [n_cached, N/B) and
 * the tails of the shape's queries (tail: float [n_seq][M][128], may be NULL
 * when M == 0). */
misa_status misa_pool_keys_cached(const misa_shape* shape, const void* k, misa_kdtype kdtype,
                                  const float* k_scale, int64_t n_cached, float* pooled,
                                  uint16_t* pooled_split, int64_t cap_blocks, float* tail, void* stream);

/* misa_indexer with the pooled keys in the cache (brought up to date first).
 * The result is exactly misa_indexer's on the same arguments.  ws: at least
 * misa_indexer_cached_workspace_bytes() bytes.  With M == 0 it only updates
 * the cache (q, w and idx may then be NULL). */
misa_status misa_indexer_cached(const misa_shape* shape, const uint16_t* q, const float* w, const void* k,
                                misa_kdtype kdtype, const float* k_scale, int32_t h, int32_t topk,
                                int32_t k_prime, int64_t n_cached, float* pooled, uint16_t* pooled_split,
                                int64_t cap_blocks, int32_t* idx, float* vals, void* ws, size_t ws_bytes,
                                void* stream);

size_t misa_indexer_cached_workspace_bytes(const misa_shape* shape, misa_kdtype kdtype, int32_t h,
                                           int32_t topk, int32_t k_prime);

/* misa_indexer_cached (k_prime = 0) on keys read in place from a paged cache
 * (the serving engine's KV pages; the GitHub issue's measured configuration
 * counts the cache handling inside the indexer): the pooling of the new
 * blocks and tails, and the routed scoring, read key t of sequence b from
 * page block_table[b * max_pages + t / page_keys], row t % page_keys, of the
 * pools k_pages (key rows of the kdtype, [n_pages][page_keys][128]) and, for
 * fp8 keys, scale_pages (float [n_pages][page_keys]).  No copy of the keys is
 * made (fp8 pages are widened on their way into LDS, never into the
 * workspace): the selection runs as misa_indexer_cached's does, its
 * sampled pass looking up each sampled key's page, its 64-key tiles one page
 * each, and the result equals misa_indexer_cached's on the keys
 * misa_gather_keys_paged would gather, bit for bit.
 * page_keys >= 64 and a multiple of 64 (a 64-key scoring tile then lies in
 * one page), n_pages >= 1, max_pages >= ceil(N / page_keys), else
 * MISA_ERR_INVALID_ARG; table entries are a precondition (in [0, n_pages);
 * out-of-range ones are clamped, never faulting); 1 <= h <= 8 (else
 * MISA_ERR_UNSUPPORTED).  Cache arguments as misa_indexer_cached; ws: at
 * least misa_indexer_paged_workspace_bytes() bytes.  With M == 0 it only
 * updates the cache (q, w and idx may then be NULL). */
misa_status misa_indexer_paged(const misa_shape* shape, const uint16_t* q, const float* w, const void* k_pages,
                               misa_kdtype kdtype, const float* scale_pages, const int32_t* block_table,
                               int64_t max_pages, int64_t n_pages, int32_t page_keys, int32_t h, int32_t topk,
                               int64_t n_cached, float* pooled, uint16_t* pooled_split, int64_t cap_blocks,
                               int32_t* idx, float* vals, void* ws, size_t ws_bytes, void* stream);

size_t misa_indexer_paged_workspace_bytes(const misa_shape* shape, misa_kdtype kdtype, int32_t h, int32_t topk);

/* Chunked prefill driver: the indexer over the shape's M queries (positions
 * q_pos0 .. q_pos0+M-1 of each sequence) in chunks of `chunk` queries, the way
 * a serving engine prefills a long prompt: chunk c sees the keys through its
 * own last query, and the pooled-key cache (kept in the workspace) grows from
 * chunk to chunk.  Sequences are processed one after another.  idx / vals as
 * misa_indexer over the whole shape, and equal to it: each query's top-k
 * depends only on its own prefix.  ws: at least misa_prefill_workspace_bytes()
 * bytes (the cache of one sequence plus the largest chunk's indexer
 * workspace).  chunk >= 1, else MISA_ERR_INVALID_ARG. */
misa_status misa_prefill_chunked(const misa_shape* shape, const uint16_t* q, const float* w, const void* k,
                                 misa_kdtype kdtype, const float* k_scale, int32_t h, int32_t topk,
                                 int32_t k_prime, int32_t chunk, int32_t* idx, float* vals, void* ws,
                                 size_t ws_bytes, void* stream);

size_t misa_prefill_workspace_bytes(const misa_shape* shape, misa_kdtype kdtype, int32_t h, int32_t topk,
                                    int32_t k_prime, int32_t chunk);

/*
 * ---------------------------------------------------------------------------
 * The paged serving step around misa_indexer_paged: page planning from request
 * lengths, rotary positions, the write of new keys and values into their
 * pages, and attention over the pages or over the tokens the indexer picked.
 *
 * Ragged batches.  These calls take the new tokens of n_seq sequences as rows
 * 0 .. q_start[n_seq]-1 of token-major tensors: sequence b's new tokens are
 * rows q_start[b] .. q_start[b+1]-1, in order, and are the last ones of its
 * kv_lens[b] tokens, so new token i of m sits at position kv_lens[b] - m + i.
 * Lengths live on the GPU and are read there.  Rows from q_start[n_seq] on (a
 * padded batch) are left as they were: in out and lse of the attention calls,
 * and in the pages, where their slot is -1.  misa_rope knows no sequences and
 * turns every row by its position, a padded one (-1) too.
 * Strided inputs.  Where a stride is given it counts elements; the last
 * dimension is dense.
 * Slots.  Row r of page p of a pool with page_keys rows a page is slot
 * p * page_keys + r.
 * ---------------------------------------------------------------------------
 */

/*
 * Block tables and slot maps from request lengths.  Sequence b holds
 * cached_lens[b] tokens in pages its table row already names, and gets
 * new_lens[b] more.  With have = ceil(cached / page_keys) and need =
 * ceil((cached + new) / page_keys) - have, the call takes `need` pages for
 * each sequence from free_pages, in sequence order, writes them to
 * block_table[b][have .. have+need-1] (the row's other entries stay as they
 * were), and writes
 *   q_start[0..n_seq]  first new token of each sequence (exclusive sums of new_lens)
 *   kv_lens[b]         cached + new
 *   slots[t]           slot of new token t, -1 for t >= q_start[n_seq]
 *   positions[t]       its position in its sequence, -1 for t >= q_start[n_seq]
 *   n_taken[0]         pages needed: free_pages[0 .. n_taken-1] are in use now
 * Negative lengths count as 0.  Where free_pages is too short (n_taken >
 * n_free) the entries without a page become -1 and so do the slots in them;
 * tokens past the table (max_pages * page_keys) get slot -1 and no page.
 * Tokens past n_tokens (slots / positions too short) get no slot.
 * cached_lens, new_lens: int32 [n_seq].  free_pages: int32 [n_free], NULL when
 * n_free = 0.  block_table: int32 [n_seq][max_pages].  slots: int64 [n_tokens],
 * positions: int32 [n_tokens].  1 <= n_seq <= 65535, page_keys >= 1,
 * max_pages >= 1, n_tokens <= 2^26 (larger: MISA_ERR_UNSUPPORTED).  Outputs
 * overlap neither inputs nor each other (MISA_ERR_INVALID_ARG): the kv_lens that
 * a call fills are the next step's cached_lens only once it has other outputs.
 */
misa_status misa_plan_pages(int32_t n_seq, const int32_t* cached_lens, const int32_t* new_lens, int32_t page_keys,
                            const int32_t* free_pages, int32_t n_free, int32_t* block_table, int64_t max_pages,
                            int32_t* q_start, int32_t* kv_lens, int64_t* slots, int32_t* positions,
                            int64_t n_tokens, int32_t* n_taken, void* stream);

typedef enum { MISA_T_BF16 = 0, MISA_T_FP16 = 1, MISA_T_FP32 = 2 } misa_dtype;
typedef enum {
  MISA_ROPE_HALF = 0,         /* pair j: elements j and j + rotary_dim/2 */
  MISA_ROPE_INTERLEAVED = 1   /* pair j: elements 2j and 2j + 1 */
} misa_rope_layout;

/* The rotation of a head's rotary part: elements rot_start ..
 * rot_start+rotary_dim-1; the rest of the head is copied.  Pair j of a token
 * at position p turns by the angle p * inv_freq[j] (radians) and is scaled by
 * mscale (the attention factor of a context-stretched model; 1 otherwise):
 *   (a, b) -> mscale * (a cos - b sin, a sin + b cos)
 * backward != 0: the transposed map (a cos + b sin, b cos - a sin) * mscale,
 * which takes the gradient of the output to the gradient of the input.
 * inv_freq: double [rotary_dim/2], positions: int32 [n_tokens], both on the
 * GPU.  Angles are formed and reduced in fp64, so far positions keep their
 * precision; the rotation runs in fp32 (or wider) and rounds once. */
typedef struct {
  const double* inv_freq;
  const int32_t* positions;
  int32_t rotary_dim;   /* even, 2 .. 1024 */
  int32_t rot_start;    /* >= 0, rot_start + rotary_dim <= head_dim */
  int32_t layout;       /* misa_rope_layout */
  int32_t backward;
  double mscale;
} misa_rope_spec;

/* Rotary positions of x [n_tokens][n_heads][head_dim] into out (same type).
 * out == x with the same strides rotates in place; any other overlap is a
 * precondition violation.  Strides must keep the heads apart. */
misa_status misa_rope(const misa_rope_spec* spec, const void* x, misa_dtype dtype, int64_t n_tokens, int32_t n_heads,
                      int32_t head_dim, int64_t x_stride_token, int64_t x_stride_head, void* out,
                      int64_t out_stride_token, int64_t out_stride_head, void* stream);

/*
 * New keys (and values) into their pages.  Row (t, h) of k goes to
 * k_pages[slot / page_keys][slot % page_keys][h][:], slot = slots[t]; v, when
 * given, to v_pages likewise.  spec != NULL rotates k first (v never; spec's
 * backward must be 0).
 * Rows are rounded (bf16) or quantised (e4m3) once, after the rotation:
 * scale_pages[...][h] = fp32(amax / 448) of the row (1 for a zero row) and
 * codes = e4m3fn round-to-nearest-even of fp32(row / scale), the rule of
 * misa_quantize_q.
 * Slots outside [0, n_pages * page_keys) write nothing (padding); slots are
 * distinct, else which of the rows a slot holds is not defined.  With
 * n_heads = 1 and head_dim = 128 the pages are those of misa_indexer_paged.
 * k, v: bf16, strides in elements and multiples of 8, 16-byte aligned.
 * head_dim: a multiple of 8 up to 512 (else MISA_ERR_UNSUPPORTED).
 */
misa_status misa_write_pages(int64_t n_tokens, int32_t n_heads, int32_t head_dim, const uint16_t* k,
                             int64_t k_stride_token, int64_t k_stride_head, const uint16_t* v,
                             int64_t v_stride_token, int64_t v_stride_head, const int64_t* slots,
                             const misa_rope_spec* spec, void* k_pages, void* v_pages, misa_kdtype kdtype,
                             float* k_scale_pages, float* v_scale_pages, int64_t n_pages, int32_t page_keys,
                             void* stream);

/* Paged keys and values: row (token t of sequence b, kv head g) is
 * k[block_table[b][t / page_keys]][t % page_keys][g][:], of kdtype, with fp8
 * rows' scales in k_scale [n_pages][page_keys][n_kv_heads] (v likewise).
 * page_keys >= 1, any; n_pages * page_keys < 2^31 (else
 * MISA_ERR_UNSUPPORTED).  Table entries of pages that hold visible keys are a
 * precondition (in [0, n_pages); out-of-range ones are clamped, never
 * faulting); rows behind a sequence's end may hold anything. */
typedef struct {
  const void* k;
  const void* v;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;   /* [n_seq][max_pages] */
  int64_t max_pages, n_pages;
  int32_t page_keys;
  int32_t kdtype;               /* misa_kdtype */
} misa_kv_pages;

typedef struct {
  int32_t n_seq;                /* 1..65535 */
  int32_t n_heads;              /* query heads, a multiple of n_kv_heads, <= 1024 */
  int32_t n_kv_heads;
  int32_t head_dim;             /* 64 or 128 */
  int64_t n_tokens;             /* rows of q and out, 0..2^26 */
  int64_t q_stride_token, q_stride_head;   /* multiples of 8 */
  int32_t max_new;              /* no sequence has more new tokens than this (rows past it may stay unwritten); 0:
                                   not known, and the call prepares for any mix: both kernels run, and there is
                                   a workspace where decodes alone need none (64 decodes over 2..4K keys, 32 / 8
                                   heads of 128: 166 us and 34 MB, with max_new = 1 155 us and none) */
  float scale;                  /* on q . k, usually 1/sqrt(head_dim) */
} misa_attn_shape;

/*
 * Causal attention of the new tokens of a ragged batch over their sequences'
 * pages (the new keys written already): query head h of a token at position p
 * reads kv head h / (n_heads / n_kv_heads),
 *   out = sum_{s <= p} softmax_s(scale * q . k[s]) v[s]
 *   lse = log sum_{s <= p} exp(scale * q . k[s])
 * A row that sees no key (or none with a score above -inf) gives out = 0, lse =
 * -inf.
 * One call takes decodes (one new token), chunks and both mixed.  Products
 * accumulate in fp32; softmax statistics are fp32; the softmax weights enter
 * the product with v as bf16 (in two parts where a kv head has few rows).
 * NaN in the keys and values that a row sees shows in its out (and, of keys, in
 * lse).  A score of +infinity gives NaN in both, one of -infinity a weight of 0;
 * an infinite value makes the elements it enters infinite or NaN (a weight, or
 * its second part, may round to 0).  NaN and infinity in a value among a
 * sequence's new tokens may reach its earlier new tokens too, never another
 * sequence; what a row of selected tokens does not list never reaches it.
 * q: bf16.  out: bf16 [n_tokens][n_heads][head_dim] dense, lse: float
 * [n_tokens][n_heads] or NULL; neither overlaps an input.  Where kv_lens[b] is
 * past max_pages * page_keys, positions are still those of the true length, as
 * in the page plan, and the keys without a table entry are not read.
 * ws: misa_attention_paged_workspace_bytes() bytes (16-byte aligned; may be NULL
 * when that is 0); nothing in it outlives the call.
 * Calls of more than 2^23 workgroups are MISA_ERR_UNSUPPORTED, and the workspace
 * query gives 0.  With G = n_heads / n_kv_heads and for each kv head these are
 * at most n_seq, and n_tokens * G / 64 + n_seq of chunks' rows (n_tokens * G /
 * 128 where more than 64 rows of a kv head may be one sequence's).
 */
misa_status misa_attention_paged(const misa_attn_shape* shape, const misa_kv_pages* pages, const uint16_t* q,
                                 const int32_t* q_start, const int32_t* kv_lens, uint16_t* out, float* lse, void* ws,
                                 size_t ws_bytes, void* stream);
size_t misa_attention_paged_workspace_bytes(const misa_attn_shape* shape, const misa_kv_pages* pages);

/*
 * The same over the tokens that the indexer picked: new token t reads only
 * tokens idx[t][0..topk-1] of its sequence (an indexer call's idx viewed as
 * [n_tokens][topk]).  Entries that are negative or lie behind the token's own
 * position count as absent; an id listed twice counts twice.
 * idx: int32 [n_tokens][topk], 1 <= topk <= MISA_MAX_TOPK.  Workgroups (see
 * above) for each kv head: n_tokens, times ceil(G / 128) where G > 64.
 */
misa_status misa_attention_selected(const misa_attn_shape* shape, const misa_kv_pages* pages, const uint16_t* q,
                                    const int32_t* q_start, const int32_t* kv_lens, const int32_t* idx, int32_t topk,
                                    uint16_t* out, float* lse, void* ws, size_t ws_bytes, void* stream);
size_t misa_attention_selected_workspace_bytes(const misa_attn_shape* shape, const misa_kv_pages* pages, int32_t topk);

/*
 * ---------------------------------------------------------------------------
 * Trees of drafted tokens.  A step that verifies drafts takes a sequence's new
 * tokens as a tree instead of a chain: a new token is a child of another one or
 * of the sequence's last cached token, and sees the cached prefix, its
 * ancestors and itself.  The new tokens' keys and values are written to the
 * places behind the prefix in the tokens' order (misa_plan_pages' slots, and
 * misa_write_pages with this plan's positions); once a path of the tree is
 * accepted, misa_keep_path moves its rows to where the prefix goes on.  A
 * sequence with one new token is a tree of one, and one whose every token is the
 * child of the token before it sees what misa_attention_paged's rows see.
 * ---------------------------------------------------------------------------
 */

/*
 * parents[t], of new token i of its sequence (row t = q_start[b] + i): the
 * index of its parent among the sequence's new tokens, in 0 .. i-1; -1, or any
 * other value, makes it a child of the last cached token.  Writes
 *   mask[t][..]   ancestor bits: bit j of the row is set where new token j is an
 *                 ancestor of token i or i itself (bit j % 32 of word j / 32).
 *                 Ancestors from 32 * words on have no bit.
 *   positions[t]  kv_lens[b] - m + depth, m the sequence's new tokens, depth the
 *                 number of the token's ancestors among them: its place in the
 *                 text that it is drafted for, which misa_rope turns it by
 * Rows that are no sequence's (in front of q_start[0], from q_start[n_seq] on)
 * get an empty mask and position -1.
 * A token takes a step for each of its ancestors: a chain of 256 tokens 23 us, of
 * 1024 85, of 8192 1070, and where a sequence has more than 32 * words tokens
 * a thread has several of its walks to make.  A prompt's chunk is not planned as a
 * chain: misa_attention_paged takes it as it is.
 * parents: int32 [n_tokens]; q_start, kv_lens as misa_plan_pages writes them.
 * mask: uint32 [n_tokens][words], positions: int32 [n_tokens]; they overlap
 * nothing else.  1 <= words <= 1024, 1 <= n_seq <= 65535, n_tokens <= 2^26.
 */
misa_status misa_plan_tree(int32_t n_seq, const int32_t* parents, const int32_t* q_start, const int32_t* kv_lens,
                           int64_t n_tokens, int32_t words, uint32_t* mask, int32_t* positions, void* stream);

/*
 * misa_attention_paged over trees: new token i of a sequence of m sees its
 * kv_lens[b] - m cached tokens, and new token j where bit j of its mask row is
 * set and j < m (any bits: the mask need not come from misa_plan_tree).  The
 * mask is read for the rows of sequences only.  A row that sees nothing gives
 * out = 0, lse = -inf.  All else is as in misa_attention_paged, its limits too.
 * NaN and infinity in a value among a sequence's new tokens may reach others of
 * its new tokens, never another sequence.
 * Over picked tokens there is no such call: misa_attention_selected takes no mask, and
 * a node's picks may name other branches' tokens, which the caller makes -1 first.
 * ws: misa_attention_tree_workspace_bytes() bytes, as misa_attention_paged's.
 * mask: uint32 [n_tokens][words], 1 <= words <= 1024 (MISA_ERR_UNSUPPORTED past it).
 */
misa_status misa_attention_tree(const misa_attn_shape* shape, const misa_kv_pages* pages, const uint16_t* q,
                                const int32_t* q_start, const int32_t* kv_lens, const uint32_t* mask, int32_t words,
                                uint16_t* out, float* lse, void* ws, size_t ws_bytes, void* stream);
size_t misa_attention_tree_workspace_bytes(const misa_attn_shape* shape, const misa_kv_pages* pages);

/*
 * The accepted path's rows to their places behind the cached prefix.  path[b][..]
 * names new tokens of sequence b in rising order (a path from a root down, as
 * parents come before their children); it ends at the first entry that does not
 * rise, is negative or is not below the sequence's count of new tokens.  With c
 * entries and first = kv_lens[b] - m, row first + path[b][i] of the keys (the
 * values, their scales) becomes row first + i, for i < c, and kept_lens[b] =
 * first + c: the next step's cached_lens.  Rows from kept_lens[b] on are left
 * as they are, to be written over.
 * Every layer's pages take a call of their own, the index keys' too (n_heads = 1,
 * v_pages = NULL).  Rows whose table entry is missing (past max_pages, or not in
 * [0, n_pages)) are not moved.  Sequences share no page that holds new tokens.
 * path: int32 [n_seq][max_path], max_path <= 2^20.  kept_lens: int32 [n_seq],
 * overlapping nothing else.  Pools as misa_write_pages takes them.
 */
misa_status misa_keep_path(int32_t n_seq, const int32_t* path, int32_t max_path, const int32_t* q_start,
                           const int32_t* kv_lens, const int32_t* block_table, int64_t max_pages, int32_t n_heads,
                           int32_t head_dim, void* k_pages, void* v_pages, misa_kdtype kdtype, float* k_scale_pages,
                           float* v_scale_pages, int64_t n_pages, int32_t page_keys, int32_t* kept_lens, void* stream);

/*
 * ---------------------------------------------------------------------------
 * Products with e4m3 weights that have a scale for each block of 128 x 128, and
 * activations with one for each 1 x 128: the projections around the indexer and
 * the attention (queries, index queries and keys, outputs).
 * ---------------------------------------------------------------------------
 */

/*
 * e4m3 codes of x [rows][cols] and the scales of its blocks of block_rows (1 or
 * 128) x 128; the last block of a row of blocks, and the last row of blocks, may be
 * smaller:
 *   scale = fp32(amax / 448), at least 2^-126; 1 for a block of zeros
 *   codes = e4m3fn round-to-nearest-even of fp32(x / scale)
 * the rule of misa_quantize_q, which this call equals bit for bit for heads of 128
 * (block_rows = 1) but where a row's values all lie below 448 * 2^-126.  NaN
 * becomes the NaN code and leaves its block's scale alone; a block with an
 * infinity has scale infinity, its infinities NaN codes, the rest 0.
 * x: bf16, fp16 or fp32, row stride x_stride (elements), 16-byte aligned rows.
 * codes: [rows][cols] dense, 16-byte aligned.  scale: float
 * [ceil(rows / block_rows)][ceil(cols / 128)].  cols: a multiple of 16, up to 2^20;
 * rows * ceil(cols / 128) <= 2^27 (else MISA_ERR_UNSUPPORTED).
 */
misa_status misa_quantize_blocks(const void* x, misa_dtype dtype, int64_t rows, int64_t cols, int64_t x_stride,
                                 int32_t block_rows, uint8_t* codes, float* scale, void* stream);

/*
 *   out[i][j] = sum_b x_scale[i][b] w_scale[j / 128][b] sum_{128 b <= c < 128 (b + 1)} x[i][c] w[j][c]
 * x: e4m3 codes [m][k], w: e4m3 codes [n][k] (a linear layer's weight), row strides
 * in bytes and multiples of 16, rows 16-byte aligned.  x_scale: float
 * [m][ceil(k / 128)], w_scale: float [ceil(n / 128)][ceil(k / 128)], dense.  out:
 * bf16 [m][n], row stride out_stride >= n (elements), overlapping no input.
 * A block's sum is formed by the matrix units, which cut each product at 2^-13 of the
 * largest of the eight (columns 8 c .. 8 c + 7) that it is summed with first, and is scaled
 * and added up in fp32; out is rounded once.  The order of the sums is fixed: the same
 * call gives the same bits.  NaN codes and scales show in the
 * rows and columns that they are in.
 * k: a multiple of 16, up to 2^20 (else MISA_ERR_UNSUPPORTED).
 * ws: misa_matmul_q8_workspace_bytes() bytes (16-byte aligned; may be NULL when
 * that is 0); nothing in it outlives the call.
 */
misa_status misa_matmul_q8(int64_t m, int64_t n, int64_t k, const uint8_t* x, int64_t x_stride, const float* x_scale,
                           const uint8_t* w, int64_t w_stride, const float* w_scale, uint16_t* out, int64_t out_stride,
                           void* ws, size_t ws_bytes, void* stream);
size_t misa_matmul_q8_workspace_bytes(int64_t m, int64_t n, int64_t k);

/*
 * Profiling.  The stages of misa_indexer (and of the calls that run parts of
 * it: misa_sparse_head_topk[_q8], misa_indexer_cached, misa_indexer_q8,
 * misa_indexer_noalloc, misa_prefill_chunked) whose kernels a caller can time
 * on their own with HIP events.  The fused-selection stages apply when that
 * path is taken (misa_sparse_head_topk above).
 */
typedef enum {
  MISA_STAGE_NONE = 0,
  MISA_STAGE_POOL = 1,               /* block pooling (inside the indexer calls) */
  MISA_STAGE_ROUTE = 2,              /* head routing (inside the indexer calls) */
  MISA_STAGE_SCORE_SAMPLE = 3,       /* scores of the key sample */
  MISA_STAGE_SAMPLE_THRESHOLD = 4,   /* per-row thresholds from the sample */
  MISA_STAGE_SCORE_CANDIDATES = 5,   /* routed scoring that keeps the candidates */
  MISA_STAGE_REGION_SELECT = 6,      /* exact top-k of the candidates */
  MISA_STAGE_RESCORE = 7,            /* re-scoring and top-k of the rows the candidates could not settle */
  MISA_STAGE_RERANK = 8,             /* MISA-dagger: all-head re-rank of the k' candidates */
  MISA_STAGE_FINAL_TOPK = 9,         /* MISA-dagger: top-k of the re-ranked candidates */
  MISA_STAGE_SCORE_LOGITS = 10,      /* routed scoring into whole logits rows (few queries, short prefixes, paged keys) */
  MISA_STAGE_LOGITS_TOPK = 11        /* top-k of those logits */
} misa_stage;

/*
 * Until the next misa_profile_stage call on the same host thread, every call
 * made on that thread records start_event on its stream just before it
 * enqueues the kernels of `stage`, and stop_event just after (hipEvent_t
 * passed as void*, created by the caller; the setting is per host thread).
 * A call that does not run the stage records nothing.  MISA_STAGE_NONE (events
 * may be NULL) turns it off.  An unknown stage or a null event:
 * MISA_ERR_INVALID_ARG.
 */
misa_status misa_profile_stage(int32_t stage, void* start_event, void* stop_event);

#ifdef __cplusplus
}
#endif

#endif /* MISA_H */
