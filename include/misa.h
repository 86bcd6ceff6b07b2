/*
 * misa.h — C ABI of the MISA routed token indexer for AMD Instinct MI355X (gfx950).
 *
 * The library implements the indexer of DeepSeek-Sparse-Attention-style
 * inference as described on the MISA pages (arXiv 2605.07363, "MISA: Mixture of
 * Indexer Sparse Attention for Long-Context LLM Inference": the abstract, and
 * gist.science's "Technische Samenvatting" with its sections "Probleemstelling",
 * "Methodologie: MISA" and "Hiërarchische Variant (MISA†)"):
 *
 *   1. mean-pool the indexer keys into blocks of B tokens      (misa_pool_keys)
 *   2. a router scores all H heads on the pooled keys and keeps
 *      the top-h heads of each query                           (misa_route)
 *   3. only the routed heads score every visible prefix token,
 *      S[t][s] = sum_{g in R_t} w[t][g] * max(q[t][g] . k[s], 0),
 *      and a per-query top-k keeps the selected tokens         (misa_score_topk)
 *   4. MISA†: the routed pass keeps k' candidates, the dense
 *      H-head indexer re-ranks them to the final k              (misa_hier_rerank)
 *   5. the dense DSA indexer, all H heads                      (dsa_index_dense)
 *
 * and, around the indexer, the key/value cache and the attention that reads it:
 *   6. new keys and values, rotated, into a paged cache        (misa_cache_append)
 *   7. attention over the selected tokens                      (misa_attend_selected)
 *   8. attention over the whole cache, also behind a prefix
 *      that the batch shares             (misa_attend, misa_attend_shared)
 *   9. how much weight attention gave each cached token        (misa_attend_mass)
 *  10. eviction: the tokens of most weight become the first
 *      rows of the cache              (misa_cache_evict, misa_cache_move)
 *  11. the next tokens from a step's logits                    (misa_sample)
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - All array arguments are DEVICE pointers to caller-owned memory. The library
 *    never retains, frees or allocates them, and allocates no device memory at
 *    run time: scratch space is the caller's workspace `ws` of at least
 *    misa_workspace_bytes(...) bytes (256-byte aligned). A workspace may be
 *    reused by later calls on the same stream; calls that overlap in time must
 *    not share one. (misa_hier_indexer_noalloc instead uses a fixed device
 *    array that the library holds per GPU; see there.)
 *  - `stream` is a hipStream_t passed as void* (NULL = the legacy default
 *    stream). Work is enqueued asynchronously on it; no call synchronizes.
 *  - Layouts (row-major, contiguous):
 *      q      bf16  [T][H][d]        per-head indexer queries
 *      w      fp32  [T][H]           per-head weights
 *      k      bf16  [nseq][Lmax][d]  one indexer key per token, shared by all heads
 *      kbar   fp32  [nseq][Lmax/B][d] means of the complete blocks of B tokens
 *      q_seq  int32 [T]              sequence of query t (0 <= q_seq < nseq)
 *      q_len  int32 [T]              visible prefix p of query t (tokens 0..p-1;
 *                                    a causal prefill query at position t has p = t+1)
 *      heads  int32 [T][h]           routed head ids, ascending
 *      idx    int32 [T][topk]        selected token ids, ascending, -1 padded
 *      score  fp32  [T][topk]        their scores (0 in padded slots); may be NULL
 *    q and k must be 16-byte aligned; other arrays 4-byte aligned.
 *  - Supported sizes: d in {32, 64, 128, 256}; 1 <= H <= 64; 1 <= h <= H;
 *    1 <= topk; T >= 0 (T = 0 is a no-op); 1 <= Lmax < 2^31; 1 <= B <= Lmax.
 *  - Ties: tokens of equal score go to the lower token index; heads of equal
 *    router importance go to the lower head id. Scores compare as reals (-0 == +0).
 *  - Device-side values the host cannot check: a query with q_seq outside
 *    [0, nseq) is treated as empty (idx all -1; routed heads 0..h-1); q_len is
 *    clamped to [0, Lmax]; a head id outside [0, H) contributes nothing.
 *  - Return value: MISA_OK (0) or a negative MISA_ERR_*. Arguments are checked
 *    before anything is enqueued; on error nothing is enqueued and
 *    misa_last_error() (thread-local) describes the problem.
 */
#ifndef MISA_H
#define MISA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__) || defined(__clang__)
#define MISA_API __attribute__((visibility("default")))
#else
#define MISA_API
#endif

#define MISA_OK 0
#define MISA_ERR_ARG (-1)        /* a size, range or null-pointer error            */
#define MISA_ERR_ALIGN (-2)      /* a pointer is not aligned as required            */
#define MISA_ERR_WORKSPACE (-3)  /* ws is NULL or smaller than misa_workspace_bytes */
#define MISA_ERR_HIP (-4)        /* the HIP runtime refused a launch                */

/* op codes of misa_workspace_bytes */
#define MISA_OP_ROUTE 1
#define MISA_OP_SCORE_TOPK 2
#define MISA_OP_HIER_RERANK 3
#define MISA_OP_DSA_DENSE 4
#define MISA_OP_INDEXER 5
#define MISA_OP_HIER_INDEXER 6
#define MISA_OP_BLOCK_FILTER 7     /* kc argument = m, the complete blocks kept */
#define MISA_OP_BLOCK_INDEXER 8    /* kc argument = m */
#define MISA_OP_PIVOT_INDEXER 9    /* B argument = G, the group size */

/* Library version, major * 10000 + minor * 100 + patch. */
MISA_API int32_t misa_version(void);

/* Human-readable name of a status code (static storage). */
MISA_API const char* misa_status_string(int32_t code);

/* Message describing the last error returned on the calling thread ("" if none). */
MISA_API const char* misa_last_error(void);

/*
 * Workspace bytes needed by one call of `op` (MISA_OP_*) with these sizes.
 * Arguments that an op does not use are ignored (kc matters for the MISA†
 * ops, and stands for m, the blocks kept, in the block ops; B for the ops that
 * route or pool). Returns 0 if none is needed.
 * The scoring ops hold fp32 score rows for at most 1 GiB of queries at a time
 * (min(T, 2^28 / Lmax) rows): a larger batch, such as a long causal prefill, is
 * scored and selected in consecutive slabs of queries on the stream, so the
 * workspace does not grow with T * Lmax beyond that bound. misa_indexer and
 * misa_hier_indexer run their fused decode pipeline (score rows for the whole
 * batch) only for batches of at most 4096 queries; larger batches take the
 * separate calls and their bound.
 */
MISA_API size_t misa_workspace_bytes(int32_t op, int64_t T, int32_t H, int64_t Lmax, int32_t B, int32_t topk,
                            int32_t kc);

/*
 * Block mean-pooling of the indexer keys (MISA pages, "Methodologie: MISA":
 * the prefix is split into blocks of B tokens and the router works on
 * mean-pooled keys).
 *   k     bf16 [nseq][Lmax][d]    in
 *   kbar  fp32 [nseq][Lmax/B][d]  out: kbar[n][j] = mean of k[n][jB .. jB+B-1]
 * Only complete blocks are written; a query's partial last block is pooled by
 * misa_route from k. Deterministic (fixed summation order).
 */
MISA_API int32_t misa_pool_keys(const void* k, int64_t nseq, int64_t Lmax, int32_t d, int32_t B, float* kbar,
                       void* stream);

/*
 * Incremental pooling for a decode loop. The router's O(H * M) cost
 * ("Methodologie: MISA") presumes that the pooled keys already exist; this call
 * keeps them current after tokens were appended to the key cache, by pooling
 * only the blocks that the append completed.
 *   k         bf16 [nseq][Lmax][d]    in, already holding the appended keys
 *   prev_len  int32 [nseq]            in: tokens of each sequence before the append
 *   new_len   int32 [nseq]            in: tokens after it
 *   max_new   bound on new_len[n] - prev_len[n] over the batch (0 .. Lmax)
 *   kbar      fp32 [nseq][Lmax/B][d]  in/out: kbar[n][j] is rewritten for every
 *             block j with prev_len[n] < (j + 1) B <= new_len[n]; every other
 *             block keeps its value
 * The written means are bit-identical to what misa_pool_keys writes for the
 * same blocks. A sequence whose pair is not an append (prev_len < 0,
 * new_len < prev_len or new_len > Lmax) is left alone; blocks completed
 * beyond max_new new tokens are not pooled (max_new must bound the append).
 * Errors: MISA_ERR_ARG (sizes, max_new outside [0, Lmax], null pointers),
 * MISA_ERR_ALIGN (k, kbar not 16-byte or the lengths not 4-byte aligned).
 */
MISA_API int32_t misa_pool_update(const void* k, int64_t nseq, int64_t Lmax, int32_t d, int32_t B,
                                  const int32_t* prev_len, const int32_t* new_len, int32_t max_new, float* kbar,
                                  void* stream);

/*
 * Block-pooled MoE router (MISA abstract; "Methodologie: MISA": per-head
 * affinities with pooled keys over M = ceil(p/B) blocks, aggregated into one
 * importance per head, top-h heads kept; cost O(H * M)).
 * Importance of head g for query t (the last block may be partial: its mean is
 * over the tokens the query sees):
 *     r[t][g] = w[t][g] * sum_{j < ceil(p/B)} max(q[t][g] . Kbar_j, 0)
 *   q, w, k, kbar, q_seq, q_len   in (kbar from misa_pool_keys with the same B)
 *   heads       int32 [T][h]  out: the h heads of largest r, ascending id
 *   router_key  fp32  [T][H]  out (may be NULL): r[t][g]
 *   ws / ws_bytes             workspace, misa_workspace_bytes(MISA_OP_ROUTE, T, H, Lmax, B, 0, 0)
 */
MISA_API int32_t misa_route(const void* q, const float* w, const void* k, const float* kbar, const int32_t* q_seq,
                   const int32_t* q_len, int64_t T, int32_t H, int32_t d, int64_t nseq, int64_t Lmax,
                   int32_t B, int32_t h, int32_t* heads, float* router_key, void* ws, size_t ws_bytes,
                   void* stream);

/*
 * Routed token scoring + per-query top-k (MISA abstract; "Methodologie: MISA",
 * sparse token scoring: only the h routed heads score every prefix token; the
 * final top-k comes from these reduced scores):
 *     S[t][s] = sum_{g in heads[t]} w[t][g] * max(q[t][g] . k[q_seq[t]][s], 0),  s < q_len[t]
 *   heads   int32 [T][h]   in (from misa_route, or any ids in [0, H))
 *   idx     int32 [T][topk] out: the topk best s (ties: lower s), ascending, -1 padded;
 *                           a query with q_len <= topk gets all of its prefix
 *   score   fp32  [T][topk] out (may be NULL)
 *   ws / ws_bytes           misa_workspace_bytes(MISA_OP_SCORE_TOPK, T, H, Lmax, 0, topk, 0)
 * With topk = k' this is the coarse pass of MISA† (its idx is the candidate set).
 */
MISA_API int32_t misa_score_topk(const void* q, const float* w, const void* k, const int32_t* heads, int32_t h,
                        const int32_t* q_seq, const int32_t* q_len, int64_t T, int32_t H, int32_t d,
                        int64_t nseq, int64_t Lmax, int32_t topk, int32_t* idx, float* score, void* ws,
                        size_t ws_bytes, void* stream);

/*
 * Fine stage of MISA† ("Hiërarchische Variant (MISA†)": the dense DSA indexer,
 * all H heads, re-scores only the k' candidates of the routed pass and keeps the
 * final top-k).
 *   cand   int32 [T][kc]  in: candidate token ids, ascending, -1 padded (the idx
 *                          output of misa_score_topk with topk = kc). Entries
 *                          outside [0, q_len) are not candidates; each valid
 *                          entry is scored once per occurrence.
 *   idx    int32 [T][topk] out: the topk candidates of best dense score (ties:
 *                          lower candidate slot, i.e. lower token id for an
 *                          ascending list), in candidate-slot order (ascending
 *                          token id), -1 padded when fewer than topk are valid
 *   score  fp32  [T][topk] out (may be NULL): their dense scores
 *   Requires kc >= topk.  ws: misa_workspace_bytes(MISA_OP_HIER_RERANK, T, H, Lmax, 0, topk, kc)
 */
MISA_API int32_t misa_hier_rerank(const void* q, const float* w, const void* k, const int32_t* cand, int32_t kc,
                         const int32_t* q_seq, const int32_t* q_len, int64_t T, int32_t H, int32_t d,
                         int64_t nseq, int64_t Lmax, int32_t topk, int32_t* idx, float* score, void* ws,
                         size_t ws_bytes, void* stream);

/*
 * Dense DSA indexer (MISA abstract; "Probleemstelling": the DSA indexer scores
 * every prefix token with all H_I heads and keeps the top-k, shared by all
 * heads). misa_score_topk with heads = {0..H-1}; the same summation order, so a
 * routed call with h = H and heads 0..H-1 returns bit-identical results.
 *   ws: misa_workspace_bytes(MISA_OP_DSA_DENSE, T, H, Lmax, 0, topk, 0)
 */
MISA_API int32_t dsa_index_dense(const void* q, const float* w, const void* k, const int32_t* q_seq,
                        const int32_t* q_len, int64_t T, int32_t H, int32_t d, int64_t nseq, int64_t Lmax,
                        int32_t topk, int32_t* idx, float* score, void* ws, size_t ws_bytes, void* stream);

/*
 * The whole MISA indexer in one call: misa_route followed by misa_score_topk
 * (MISA abstract; "Methodologie: MISA"), with bit-identical results. For decode
 * shapes (fewer than 8 queries per sequence on average) it runs as one pipeline
 * of four launches: router partials, head selection fused into the routed
 * scoring, and a two-launch top-k; otherwise it makes the separate calls.
 *   kbar     fp32 [nseq][Lmax/B][d] from misa_pool_keys (the pooled-key cache)
 *   heads    int32 [T][h] out, may be NULL: the routed heads
 *   idx / score as misa_score_topk
 *   ws: misa_workspace_bytes(MISA_OP_INDEXER, T, H, Lmax, B, topk, 0)
 */
MISA_API int32_t misa_indexer(const void* q, const float* w, const void* k, const float* kbar, const int32_t* q_seq,
                              const int32_t* q_len, int64_t T, int32_t H, int32_t d, int64_t nseq, int64_t Lmax,
                              int32_t B, int32_t h, int32_t topk, int32_t* heads, int32_t* idx, float* score,
                              void* ws, size_t ws_bytes, void* stream);

/*
 * The whole MISA† indexer in one call: misa_route, misa_score_topk with
 * topk = kc (the enlarged candidate set) and misa_hier_rerank to topk
 * ("Hiërarchische Variant (MISA†)"), with bit-identical results. For decode
 * shapes it runs as six launches, the candidates' dense re-scoring fused into
 * the coarse pass's compaction.
 *   heads  int32 [T][h] out, may be NULL;  cand  int32 [T][kc] out, may be NULL
 *   ws: misa_workspace_bytes(MISA_OP_HIER_INDEXER, T, H, Lmax, B, topk, kc)
 */
MISA_API int32_t misa_hier_indexer(const void* q, const float* w, const void* k, const float* kbar,
                                   const int32_t* q_seq, const int32_t* q_len, int64_t T, int32_t H, int32_t d,
                                   int64_t nseq, int64_t Lmax, int32_t B, int32_t h, int32_t kc, int32_t topk,
                                   int32_t* heads, int32_t* cand, int32_t* idx, float* score, void* ws,
                                   size_t ws_bytes, void* stream);

/*
 * misa_hier_indexer for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc. It
 * takes no workspace argument and allocates nothing; its scratch is a device
 * array of MISA_SCRATCH_BYTES that the library holds on every GPU it runs on
 * until the process ends. The caller still passes the inputs and outputs, with
 * the meaning, layout and results of misa_hier_indexer (same kernels, bit for
 * bit).
 *  - Sizes whose workspace (misa_workspace_bytes(MISA_OP_HIER_INDEXER, ...))
 *    exceeds MISA_SCRATCH_BYTES are refused with MISA_ERR_WORKSPACE before
 *    anything is enqueued (decode batches fit: 4 x 128K tokens need about
 *    9 MiB; a long causal prefill does not).
 *  - The scratch belongs to the GPU of `stream` (NULL: the current device). Its
 *    address is looked up once per device, on the first call there. Every call
 *    on a GPU shares that GPU's array and leaves its contents behind; each call
 *    clears, with its own kernels, the state it needs zeroed. Calls that overlap
 *    in time on one GPU (other streams, other host threads) race on the array
 *    and must be serialized by the caller.
 * Errors: as misa_hier_indexer; MISA_ERR_HIP if the scratch address cannot be
 * obtained.
 */
#define MISA_SCRATCH_BYTES (32u << 20)
MISA_API int32_t misa_hier_indexer_noalloc(const void* q, const float* w, const void* k, const float* kbar,
                                           const int32_t* q_seq, const int32_t* q_len, int64_t T, int32_t H,
                                           int32_t d, int64_t nseq, int64_t Lmax, int32_t B, int32_t h, int32_t kc,
                                           int32_t topk, int32_t* heads, int32_t* cand, int32_t* idx, float* score,
                                           void* stream);

/*
 * Block filter on the pooled keys, composed with head routing: the coarse stage
 * of a two-stage (block, then token) search. HISA (thelatestinai.com paper
 * cards, the HISA abstract) scores pooled block representations, drops the
 * weak blocks and runs the indexer only inside the retained ones; the
 * gist.science MISA summary presents head routing as combinable with such
 * token-axis schemes ("Betekenis en Claims"). The pages give no formula for the
 * coarse score; this library takes the routed indexer formula on the block's
 * mean key, b_j = sum over the routed heads g of w[t][g] * max(q[t][g] . kbar[j], 0),
 * for the complete visible blocks j < q_len[t] / B, keeps the m best (ties to
 * the lower block id; all of them when there are at most m) and always keeps
 * the partial last block.
 *   kbar    fp32 [nseq][Lmax/B][d]  from misa_pool_keys
 *   heads   int32 [T][h]            routed heads (an id outside [0, H) contributes nothing)
 *   m       complete blocks kept per query, 1 .. Lmax / B
 *   blocks  int32 [T][m] out: kept complete block ids, ascending, -1 padded
 *   cand    int32 [T][(m + 1) * B] out, may be NULL: the token ids of the kept
 *           blocks, then those of the partial block, ascending, -1 padded (the
 *           candidate list of misa_hier_rerank's form, for the fine stage)
 *   ws: misa_workspace_bytes(MISA_OP_BLOCK_FILTER, T, H, Lmax, B, 0, m)
 * Errors: as misa_route, and MISA_ERR_ARG for m outside [1, Lmax / B].
 */
MISA_API int32_t misa_block_filter(const void* q, const float* w, const float* kbar, const int32_t* heads,
                                   int32_t h, const int32_t* q_seq, const int32_t* q_len, int64_t T, int32_t H,
                                   int32_t d, int64_t nseq, int64_t Lmax, int32_t B, int32_t m, int32_t* blocks,
                                   int32_t* cand, void* ws, size_t ws_bytes, void* stream);

/*
 * Routed indexer restricted to the retained blocks: misa_route, then
 * misa_block_filter, then the routed scores of the candidate tokens and their
 * top-k (score descending, token id ascending; ids ascending, -1 padded). With
 * m = Lmax / B every visible token is a candidate and the result equals
 * misa_indexer's. Each query reads the keys of at most (m + 1) * B tokens.
 *   heads   int32 [T][h] out, may be NULL;  blocks  int32 [T][m] out, may be NULL
 *   idx / score as misa_score_topk (score: routed scores)
 *   ws: misa_workspace_bytes(MISA_OP_BLOCK_INDEXER, T, H, Lmax, B, topk, m)
 */
MISA_API int32_t misa_block_indexer(const void* q, const float* w, const void* k, const float* kbar,
                                    const int32_t* q_seq, const int32_t* q_len, int64_t T, int32_t H, int32_t d,
                                    int64_t nseq, int64_t Lmax, int32_t B, int32_t h, int32_t m, int32_t topk,
                                    int32_t* heads, int32_t* blocks, int32_t* idx, float* score, void* ws,
                                    size_t ws_bytes, void* stream);

/*
 * Proxy-query shared scan with per-query refinement (PIVOT-Refine;
 * thelatestinai.com paper cards, the PIVOT abstract). The queries are taken in
 * groups of G consecutive ones (the last group may be shorter), and every query
 * of a group must belong to the sequence of its first query (prefill: G
 * consecutive positions; decode: the positions of one multi-token step). Each
 * group is folded into a proxy query, the sum of its per-head queries rounded to
 * bf16 (nearest, ties to even) with the sum of their head weights (the page
 * leaves the fold open; the sum is the mean up to a positive factor, which
 * changes no ranking). The proxy scans its group's longest prefix once with the
 * dense indexer (all H heads) and keeps kc candidates (ties to the lower token
 * id); each query then re-ranks those candidates with its own dense indexer as
 * misa_hier_rerank does (ids at or beyond its own prefix are skipped).
 *   cand   int32 [T][kc] out, may be NULL: the candidates of each query's group
 *   idx / score as misa_hier_rerank (dense scores)
 *   ws: misa_workspace_bytes(MISA_OP_PIVOT_INDEXER, T, H, Lmax, G, topk, kc) (sized for d up to 256)
 * Errors: as misa_hier_rerank, and MISA_ERR_ARG for G < 1 or kc outside [topk, Lmax].
 */
MISA_API int32_t misa_pivot_indexer(const void* q, const float* w, const void* k, const int32_t* q_seq,
                                    const int32_t* q_len, int64_t T, int32_t H, int32_t d, int64_t nseq, int64_t Lmax,
                                    int32_t G, int32_t kc, int32_t topk, int32_t* cand, int32_t* idx, float* score,
                                    void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Key/value cache and attention
 *
 * A cache holds one row of d elements per token and kv head, keys and values
 * apart, in pages of `page` tokens. Token s of sequence n lies in row s % page
 * of page table[n][s / page]; without a table sequence n is page n (the layout
 * k [nseq][Lmax][d] of the indexer keys is such a cache, with one head and
 * page = Lmax). The element of (page p, row r, head g, i) is at
 *     p * page_stride + r * token_stride + g * head_stride + i
 * in elements, the same for k and v, so token-major and head-major pages both
 * fit; strides are positive multiples of 8 and the pointers 16-byte aligned.
 * The struct is read on the host during the call only; k, v and table are
 * device memory.
 *  - d: any multiple of 16 up to 1024 to append; 64, 128 or 256 to attend.
 *  - A sequence can address table_cols * page tokens (page without a table),
 *    less than 2^31 - 65536.
 *  - A table entry outside [0, npages) is no page: nothing is written there, and
 *    its tokens are not visible.
 *  - The table's rows follow each other (table_cols entries each).
 *  - Keys, and values, reach over less than 4 GiB, or over at most 2^32 - 2^16 times
 *    the largest power of two that divides page_stride and token_stride (2^35
 *    elements for odd multiples of 8, 2^39 for multiples of 128).
 */
#define MISA_BF16 1
#define MISA_FP16 2
typedef struct misa_kv_cache {
  void* k;
  void* v;                /* NULL: a cache of keys alone (append only) */
  int64_t npages;
  int64_t page;           /* tokens per page */
  int64_t page_stride;    /* in elements */
  int64_t token_stride;
  int64_t head_stride;
  int32_t heads;          /* kv heads */
  int32_t d;
  int32_t dtype;          /* MISA_BF16 or MISA_FP16 */
  const int32_t* table;   /* [nseq][table_cols] or NULL */
  int64_t table_cols;
  int64_t nseq;           /* rows of the table (without one: npages) */
} misa_kv_cache;

/*
 * Appends N tokens to the cache, rotating their keys (and, in the same launch,
 * their queries) by the angles of their positions.
 *   k, v   [N][heads][d]  the new keys and values, of the cache's type; v is NULL
 *          exactly when the cache has no values
 *   q      [N][Hq][d]     queries of the same tokens, rotated into q_out; both may
 *          be NULL (Hq = 0). q_out may be q itself (with the same strides).
 *   *_ts, *_hs            token and head strides of these arrays in elements,
 *          multiples of 8 (slices of one fused projection need no copy)
 *   q_seq, q_tok  int32 [N]  the token's sequence and its index there
 *   q_pos  int32 [N]      rotary position, or NULL: q_tok
 *   cos_sin fp32 [P][rot] cosines, then sines, of the rot / 2 angles of position p
 *   rot    rotated elements at the start of each row, a multiple of 16 up to d;
 *          0: none (cos_sin may be NULL)
 *   interleaved  pairs (2i, 2i + 1) instead of (i, i + rot / 2)
 * Pair i becomes (a cos - b sin, b cos + a sin), computed in fp32 and rounded
 * once. A token whose sequence, index, page or (rot > 0) position is out of
 * range is skipped: neither the cache nor its q_out rows are written. No two
 * tokens of a call may have the same (sequence, index) or share a page's row
 * (the row would hold parts of both). Rows of other tokens keep their values.
 * The pooled keys of an indexer cache follow with misa_pool_update.
 * Errors: MISA_ERR_ARG (sizes, null pointers; 2^24 workgroups and more, which no
 * N below 2^24 needs), MISA_ERR_ALIGN.
 */
MISA_API int32_t misa_cache_append(const misa_kv_cache* cache, const void* k, int64_t k_ts, int64_t k_hs, const void* v,
                                   int64_t v_ts, int64_t v_hs, const void* q, int64_t q_ts, int64_t q_hs, void* q_out,
                                   int64_t o_ts, int64_t o_hs, int32_t Hq, const int32_t* q_seq, const int32_t* q_tok,
                                   const int32_t* q_pos, const float* cos_sin, int64_t P, int32_t rot,
                                   int32_t interleaved, int64_t N, void* stream);

/*
 * Attention of T queries over their sequences' caches. For query t and head
 * j (kv head g = j / (Hq / heads)), over the visible tokens
 * q_start[t] <= s < q_len[t]:
 *     x_s = scale * q[t][j] . k_s
 *     x_s = cap * tanh(x_s / cap)                     if cap > 0
 *     x_s = x_s - slopes[j] * |q_pos[t] - s|          if slopes
 *     out[t][j] = sum_s exp(x_s - m) v_s / sum_s exp(x_s - m),   lse = log sum_s exp(x_s)
 * A causal query at position t has q_len = t + 1; a decode step has one query
 * per sequence; a document mask sets q_start to the document's first token, a
 * sliding window to t + 1 - window; a bidirectional prefix raises q_len to it.
 * Queries of one sequence next to each other share its keys; how many are taken
 * at a time goes by T / nseq, so the table should hold the batch's sequences, not
 * a whole pool's (T <= nseq is a decode step: every query reads its own keys).
 *   q        [T][Hq][d] of the cache's type, strides q_ts, q_hs in elements
 *            (multiples of 8); Hq a multiple of the cache's heads
 *   q_seq, q_len  int32 [T];  q_start  int32 [T] or NULL (0)
 *   q_pos    int32 [T] or NULL (q_len - 1), not negative; read with slopes only
 *   scale    in [1e-30, 1e4];  cap  0 (none) or in [1e-6, 1e30];  slopes  fp32 [Hq] or NULL
 *   out      [T][Hq][d] of the cache's type, apart from q;  lse  fp32 [T][Hq] or NULL
 * Scores are fp32: the largest x_s of a row is taken to be at most 5e7 in size
 * (where neighbouring values are 4 apart); beyond that its weights may overflow.
 * A query that sees nothing (empty interval, sequence out of range) gets zeros
 * and lse = -inf. q_len is clamped to what a sequence can address, q_start to
 * [0, q_len]. What a query does not see may hold anything, NaN included; a NaN
 * or an infinity reaches exactly the queries that see it.
 *   ws: misa_attend_workspace_bytes(MISA_OP_ATTEND, T, Hq, heads, d, nseq, 0)
 * Errors: MISA_ERR_ARG, MISA_ERR_ALIGN, MISA_ERR_WORKSPACE.
 */
MISA_API int32_t misa_attend(const misa_kv_cache* cache, const void* q, int64_t q_ts, int64_t q_hs,
                             const int32_t* q_seq, const int32_t* q_start, const int32_t* q_len, const int32_t* q_pos,
                             int64_t T, int32_t Hq, float scale, float cap, const float* slopes, void* out, float* lse,
                             void* ws, size_t ws_bytes, void* stream);

/*
 * Attention over selected tokens, the consumer of the indexers' output (MISA
 * abstract; "Probleemstelling": the selected set is shared by all heads): as
 * misa_attend, over the tokens idx[t][0 .. topk) of sequence q_seq[t]. Entries
 * outside [0, q_len[t]) (the -1 padding) are skipped, the others count once per
 * occurrence, in any order.
 *   idx  int32 [T][topk]
 *   ws: misa_attend_workspace_bytes(MISA_OP_ATTEND_SELECTED, T, Hq, heads, d, nseq, 0)
 */
MISA_API int32_t misa_attend_selected(const misa_kv_cache* cache, const void* q, int64_t q_ts, int64_t q_hs,
                                      const int32_t* idx, int32_t topk, const int32_t* q_seq, const int32_t* q_len,
                                      const int32_t* q_pos, int64_t T, int32_t Hq, float scale, float cap,
                                      const float* slopes, void* out, float* lse, void* ws, size_t ws_bytes,
                                      void* stream);

/*
 * Attention of a batch whose sequences share long prefixes: query t sees the
 * pre_len[pre[t]] tokens of prefix pre[t], at positions 0 .., and behind them
 * the q_len[t] tokens of its own sequence. The keys of a prefix are read once
 * for its queries that stand next to each other in the batch, instead of once
 * per sequence; the two parts are joined by their log-sums.
 *   pre        int32 [T]  prefix of each query; outside [0, npre): none
 *   pre_len    int32 [npre]
 *   pre_table  int32 [npre][pre_cols] pages of the prefixes in the same cache, or
 *              NULL: prefix i is page i
 *   q_pos      int32 [T] or NULL (pre_len + q_len - 1, below 2^31); read with slopes only
 *   the rest as misa_attend (q_seq, q_len: the own part)
 *   ws: misa_attend_workspace_bytes(MISA_OP_ATTEND_SHARED, T, Hq, heads, d, nseq, npre)
 */
MISA_API int32_t misa_attend_shared(const misa_kv_cache* cache, const void* q, int64_t q_ts, int64_t q_hs,
                                    const int32_t* q_seq, const int32_t* q_len, const int32_t* q_pos,
                                    const int32_t* pre, const int32_t* pre_len, const int32_t* pre_table,
                                    int64_t pre_cols, int64_t npre, int64_t T, int32_t Hq, float scale, float cap,
                                    const float* slopes, void* out, float* lse, void* ws, size_t ws_bytes,
                                    void* stream);

/* op codes of misa_attend_workspace_bytes */
#define MISA_OP_ATTEND 10
#define MISA_OP_ATTEND_SELECTED 11
#define MISA_OP_ATTEND_SHARED 12

/* Workspace bytes of one attention call (0: none needed, or sizes out of range). */
MISA_API size_t misa_attend_workspace_bytes(int32_t op, int64_t T, int32_t Hq, int32_t heads, int32_t d, int64_t nseq,
                                            int64_t npre);

/*
 * Accumulated attention weight, the measure that misa_cache_evict keeps tokens by:
 * how much weight the T queries of an attention call gave each cached token. With
 * x_s as in misa_attend (same scale, cap, slopes and intervals) and lse the log-sums
 * that the attention call returned,
 *     out[n][g][s] = in[n][g][s] + sum over the queries t of sequence n that see s, and
 *                    the heads j of kv head g, of  exp(x_s - lse[t][j])
 * for every token s that a sequence can address (L = table_cols * page, or page without
 * a table). Keys are read once for each part that their queries are split into (decode
 * steps: once), values not at all (cache->v may be NULL).
 *   lse     fp32 [T][Hq]; a row of -inf (a query that sees nothing) gives nothing. Of
 *           misa_attend over the same interval: the log-sums of misa_attend_selected count
 *           the selected tokens alone, and tokens that were not selected would still be given
 *           weight here
 *   lists   cache->heads: a sum per kv head; 1: one sum over all heads
 *   in      fp32 [nseq][lists][L] or NULL (zeros);  out  the same shape, every element
 *           written; may be in itself
 * The queries of a call may stand in any order; those of a sequence next to each other
 * are fastest. How many queries are taken at a time goes by T / nseq, so the table should
 * hold the batch's sequences, not a whole pool's. The last queries of a prompt, all of them,
 * or a decode step's make such a sum alike. It is the same from run to run: nothing depends on the order of workgroups.
 * What a query does not see may hold anything; tokens without a page get nothing.
 *   ws: misa_cache_workspace_bytes(MISA_OP_ATTEND_MASS, cache, T, Hq, lists, 0)
 * Errors: as misa_attend (d in {64, 128, 256}); MISA_ERR_ARG for lists neither 1 nor
 * cache->heads, T * Hq / heads of 2^31 - 64 and more, or nseq * heads * L too large for one launch.
 */
MISA_API int32_t misa_attend_mass(const misa_kv_cache* cache, const void* q, int64_t q_ts, int64_t q_hs,
                                  const float* lse, const int32_t* q_seq, const int32_t* q_start,
                                  const int32_t* q_len, const int32_t* q_pos, int64_t T, int32_t Hq, float scale,
                                  float cap, const float* slopes, int32_t lists, const float* in, float* out, void* ws,
                                  size_t ws_bytes, void* stream);

/*
 * Evicts tokens from the cache, in place. Of each sequence's lens[n] tokens at most
 * `budget` stay and become its first rows. The rank of a token:
 *   1. protected ones: pos < sinks, or among the `recent` latest positions
 *      (pos > newest - recent, newest the largest position of the list);
 *   2. then by mass, larger first (NaN above all numbers, -0 equal to 0);
 *   3. ties to the lower row.
 * With lists = cache->heads each kv head keeps its own tokens, with lists = 1 all heads
 * the same. new_len = min(lens, budget). A kept row below new_len stays where it is; the
 * rows of dropped tokens below new_len take, both in ascending order, the kept rows from
 * behind. So the kept rows are in no order of position afterwards (attention over
 * [0, new_len) needs none; `pos` says which is which), few rows move, and no row that is
 * read is written. Rows from new_len on keep their contents in the cache. (Attention's
 * intervals and distance bias go by row, so neither fits a cache whose rows have moved;
 * rotations stay with the keys.)
 *   mass     fp32 [nseq][lists][L]; L = table_cols * page, or page without a table
 *   pos      int32 [nseq][lists][L] positions, or NULL: a row's number is its position
 *   lens     int32 [nseq], clamped to [0, L]
 *   mass_out, pos_out  the same shapes, or NULL; may be mass and pos themselves. Rows
 *            follow their tokens; behind new_len: 0 and -1.
 *   src      int32 [nseq][lists][budget] out: the row that each of the first rows came
 *            from, -1 from new_len on
 *   new_len  int32 [nseq] out; may be lens itself
 * No two rows that a sequence addresses below lens[n] may be one place of memory, and no
 * two sequences may share such rows (a prefix they share is to be kept apart, as
 * misa_attend_shared does). A row whose page, or whose source's page, does not exist is
 * not moved. d: any multiple of 8 up to 1024; cache->v may be NULL.
 *   ws: misa_cache_workspace_bytes(MISA_OP_CACHE_EVICT, cache, 0, 0, lists, budget)
 * Errors: MISA_ERR_ARG (budget < 1, sinks or recent negative or together more than
 * budget, lists neither 1 nor cache->heads, sizes), MISA_ERR_ALIGN, MISA_ERR_WORKSPACE.
 */
MISA_API int32_t misa_cache_evict(const misa_kv_cache* cache, const float* mass, const int32_t* pos,
                                  const int32_t* lens, int32_t lists, int64_t budget, int64_t sinks, int64_t recent,
                                  float* mass_out, int32_t* pos_out, int32_t* src, int32_t* new_len, void* ws,
                                  size_t ws_bytes, void* stream);

/*
 * The same moves in another cache of the same sequences (the indexer's keys, another
 * layer's cache): row i of a list takes row src[n][list][i], for i < n_src. Entries
 * outside [0, L), and those equal to i, move nothing; rows without a page neither. A row
 * that is a source must not be moved onto by the same call (src of misa_cache_evict never
 * does that). Pooled keys of an indexer cache whose rows moved are to be pooled again.
 *   src  int32 [nseq][lists][n_src];  lists  1 (all heads) or cache->heads
 * Errors: MISA_ERR_ARG, MISA_ERR_ALIGN.
 */
MISA_API int32_t misa_cache_move(const misa_kv_cache* cache, const int32_t* src, int32_t lists, int64_t n_src,
                                 void* stream);

/* op codes of misa_cache_workspace_bytes */
#define MISA_OP_ATTEND_MASS 13
#define MISA_OP_CACHE_EVICT 14

/* Workspace bytes of one call (0: none needed, or sizes out of range); the cache's pointers are not used. */
MISA_API size_t misa_cache_workspace_bytes(int32_t op, const misa_kv_cache* cache, int64_t T, int32_t Hq,
                                           int32_t lists, int64_t budget);

/* ------------------------------------------------------------------------
 * The next token of each of T rows of logits, from given random numbers.
 * With temperature t > 0, w_i = exp((l_i - max l) / t); then, in this order,
 *   top_k   keeps the top_k largest logits (ties to the lower id); 0 or less, or V and
 *           more: all
 *   min_p   keeps those with w_i >= min_p (1 at most); 0 or less, or NaN: all
 *   top_p   keeps the shortest prefix, in descending order (ties to the lower id), whose
 *           weights sum to at least top_p of what the first two left, one token at
 *           least; 1 and more, or NaN: all
 * and the token is the first one, in ascending order of ids, whose running sum over the
 * kept ones exceeds u times their sum. t of 0 or less, or NaN: the first of the largest
 * logits. Logits of -inf and NaN are never drawn; those of +inf share all weight. A row
 * with nothing to draw gets token -1 and logprob -inf.
 *   logits   [T][V] of dtype MISA_BF16, MISA_FP16 or MISA_FP32, rows row_stride elements apart
 *   temperature, top_p, min_p  fp32 [T], top_k  int32 [T]: each may be NULL (1, 1, 0, 0)
 *   u        fp32 [T], in [0, 1) (clamped to it; NaN counts as 0)
 *   token    int32 [T] out;  logprob  fp32 [T] out, may be NULL: the logarithm of the
 *            token's share of the kept weights (0 where t picks the largest)
 * Weights are multiples of 2^-42 of the row's largest one (worked out in fp64; below
 * 2^-43 they are 0), and their sums exact, so the result depends on no order.
 * 1 <= V <= 2^20.
 *   ws: misa_sample_workspace_bytes(T, V)
 * Errors: MISA_ERR_ARG, MISA_ERR_ALIGN, MISA_ERR_WORKSPACE.
 */
#define MISA_FP32 3
MISA_API int32_t misa_sample(const void* logits, int32_t dtype, int64_t row_stride, int64_t T, int32_t V,
                             const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                             const float* u, int32_t* token, float* logprob, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes of one misa_sample call (0: none needed, or sizes out of range). */
MISA_API size_t misa_sample_workspace_bytes(int64_t T, int32_t V);

/*
 * Full score rows of the routed scoring step (a diagnostic of step 3 above):
 * scores fp32 [T][Lmax], row t filled for s < q_len[t], other entries untouched.
 * heads may be NULL (then h must equal H: dense scores).
 */
MISA_API int32_t misa_debug_scores(const void* q, const float* w, const void* k, const int32_t* heads, int32_t h,
                          const int32_t* q_seq, const int32_t* q_len, int64_t T, int32_t H, int32_t d,
                          int64_t nseq, int64_t Lmax, float* scores, void* stream);

/*
 * Event timing of one internal kernel class, for measurement tools:
 * kernel 1 = token scoring over prefixes (routed or dense), 2 = top-k,
 * 3 = router, 4 = pooling, 5 = token scoring over candidate lists (re-rank).
 * After misa_timing_begin(kernel, capacity, stream), each launch of that kernel
 * class on `stream` (up to `capacity` launches) is bracketed by events on that
 * stream; launches on other streams are not touched. misa_timing_end(stream,
 * ...) waits for the recorded events, returns the summed duration in ms and
 * the number of launches timed, and ends the timing of that stream. A second
 * begin on a stream replaces the first. While no stream is timed the launch
 * hooks cost one atomic load. Beginning or ending the timing of a stream while
 * another thread launches on that same stream is not supported.
 */
MISA_API int32_t misa_timing_begin(int32_t kernel, int32_t capacity, void* stream);
MISA_API int32_t misa_timing_end(void* stream, float* total_ms, int32_t* launches);

#ifdef __cplusplus
}
#endif

#endif /* MISA_H */
