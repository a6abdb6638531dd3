/*
 * spec_paged_kv.h -- a verification round on a paged key/value cache: the new tokens'
 * keys and values written into cache pages (as bf16, or quantised to e4m3), their
 * attention over the cache under the chain's or the tree's mask, pages read back, and
 * the accepted tree nodes' rows moved through the page table after the verify.  Same
 * library, status codes and conventions as spec_verify.h (caller-owned device arrays,
 * asynchronous on `stream`, argument errors returned before any launch, SV_ERR_CUDA for
 * launch failures).
 *
 * Defining passages (page title, section):
 *  - "Speculative Decoding and EAGLE", sections "개념" and "트리 어텐션 검증 (Tree
 *    Attention Verification)": the target checks every drafted token in one forward
 *    pass; in a tree each token attends to its ancestors only.
 *  - "[논문 리뷰] Fast Inference from Transformers via Speculative Decoding", section 2
 *    "제안 방법", Step 2: the K+1 positions are scored in parallel over the shared
 *    prefix; section 4 "한계점": the cache entries of rejected tokens are rolled back.
 * The pages give no cache layout; the paged layout and the quantised form are this
 * library's own.
 */
#ifndef SPEC_PAGED_KV_H
#define SPEC_PAGED_KV_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of cache pages (activations use sv_dtype). */
typedef enum {
    SV_CACHE_BF16 = 0,
    SV_CACHE_E4M3 = 1 /* 8-bit floats, 448 at most, with an fp32 scale per token and head */
} sv_cache_dtype;

/*
 * A paged cache.  Position pos of batch row b lives in page page_table[b][pos / page_size],
 * row pos % page_size of that page; the row of head h starts at
 *   k_pages + page * page_stride + h * head_stride + row * row_stride   (bytes)
 * and holds head_dim elements; v_pages alike.  A table entry outside [0, num_pages) is a
 * hole: nothing is stored there.
 *   k_scale, v_scale  device fp32 [num_pages][num_heads][page_size], dense; the value of a
 *                e4m3 element is its code times the scale of its position and head.  NULL
 *                for SV_CACHE_BF16.
 *   page_table   device int32 [B][max_pages], dense.
 * The struct is read during the call and is not retained.
 *   1 <= num_pages, 1 <= page_size <= 65536, 1 <= max_pages, max_pages * page_size <= 2^30,
 *   1 <= num_heads <= 1024, 1 <= head_dim <= 256; strides are multiples of the element
 *   size and row_stride covers a row.
 */
typedef struct {
    void *k_pages;
    void *v_pages;
    float *k_scale;
    float *v_scale;
    const int32_t *page_table;
    int64_t page_stride, head_stride, row_stride;
    int dtype; /* sv_cache_dtype */
    int num_pages, page_size, max_pages, num_heads, head_dim;
} sv_paged_cache;

/*
 * Rows of a call.  base[b] (device int32 [B]) is the number of positions of batch row b
 * before the call's first token, and new_len[b] (device int32 [B], or NULL: N for every
 * row) the number of its tokens that are real, 0 <= new_len[b] <= N; token i of row b has
 * position base[b] + i.  A batch row with a negative base, a new_len outside [0, N] or
 * base + new_len beyond max_pages * page_size is left untouched by every entry, as are
 * outputs and cache rows of tokens i >= new_len[b].
 */

/*
 * Writes the new tokens' keys and values into the cache.
 *   key, value   device [B][N][num_heads][head_dim], dtype src (SV_F32 or SV_BF16), with
 *                element strides src_stride[0..2] (batch, token, head; HOST int64 array of
 *                three) and contiguous elements.  0 <= N < 2^31 / num_heads.
 * SV_CACHE_BF16: elements are rounded to nearest even.  SV_CACHE_E4M3: with a the largest
 * finite |x| of the row of one token and head, scale = max(a / 448, 2^-126) and each
 * element becomes the e4m3 value nearest to x / scale (even on ties), at most 448 in
 * magnitude; infinities become +-448 * scale, NaN stays NaN.  scale and x / scale are fp32
 * quotients, rounded to nearest even (x / scale from within 2^-46 of itself).
 * Tokens whose table entry is a hole are not written.  Two tokens must not share a cache
 * row (rows may share pages that they only read).
 * Errors: SV_ERR_INVALID_ARG for a bad size, dtype, pointer or stride (B = 0 or N = 0
 * returns SV_OK and launches nothing).
 */
SV_API sv_status spec_kv_append(const void *key, const void *value, sv_dtype src, const int64_t *src_stride,
                                const sv_paged_cache *cache, const int32_t *base, const int32_t *new_len, int B,
                                int N, void *stream);

/*
 * Reads positions base[b] .. base[b] + new_len[b] - 1 back into dense arrays.
 *   out_key, out_value  device [B][N][num_heads][head_dim], dense, dtype dst (SV_F32 or
 *                SV_BF16): the element, or code times scale in fp32, rounded once.
 *                Positions in holes read as zero.
 * Other arguments and errors as spec_kv_append.
 */
SV_API sv_status spec_kv_read(const sv_paged_cache *cache, const int32_t *base, const int32_t *new_len, int B, int N,
                              void *out_key, void *out_value, sv_dtype dst, void *stream);

/*
 * Attention of a chunk of new tokens over the paged cache, which already holds the new
 * tokens' own keys and values (spec_kv_append): the attention of a target's verify pass.
 *   q            device bf16 [B][Q][num_q_heads][head_dim] with element strides
 *                q_stride[0..2] (batch, token, head; HOST int64 array of three) and
 *                contiguous elements.  num_q_heads is a multiple of cache->num_heads; query
 *                head h reads cache head h / (num_q_heads / num_heads).
 *   base, new_len  as above, with N = Q.  Query i of row b sees every position below
 *                base[b] that is no hole, and of the new positions base[b] + j, j < new_len[b]:
 *   tree_mask    NULL: those with j <= i (a chain, or a chunk of a prompt);
 *                device uint32 [B][Q-1][W], W = ceil((Q-1) / 32), as spec_tree_mask writes
 *                it for the N = Q - 1 nodes of draft trees: token 0 is the tree's root,
 *                token i + 1 node i (the rows of spec_verify_tree).  Every query sees the
 *                root, query i + 1 also node j where bit j of mask row i is set.
 *   scale        factor of the scores (1 / sqrt(head_dim) as a rule), finite.
 *   max_len      host bound on base[b] + new_len[b] over the rows, by which the work is
 *                split; 1 <= max_len.  Rows beyond it are still right, but slower.
 *   out          device bf16 [B][Q][num_q_heads][head_dim], dense: softmax(scale q k) v.
 *   out_lse      device fp32 [B][Q][num_q_heads] or NULL: natural logarithm of the sum of
 *                exponentials of the scaled scores.
 * A query that sees no position (or only scores of -inf) gets a zero output and lse -inf.  Keys and values at
 * positions that a query does not see never affect it, whatever they hold.  Scores,
 * softmax sums and outputs are accumulated in fp32; the probabilities enter the second
 * product rounded to bf16 (for e4m3, times the value's scale).  e4m3 calls of more than 16
 * query rows per cache head multiply as fp16 instead: a value's code
 * times its scale and a probability are rounded once each to 11 bits, and with V = 448 times the
 * largest value scale of the positions that a query sees, what a position adds below 2^-31 V,
 * and of a value what lies below 2^-25 V, may be lost.
 * Weights may stand at up to 2^8 times their value while they are summed: bf16 values beyond
 * 2^110 may overflow to infinity.
 * out must not overlap q or the cache.  Every wait inside the kernels is bounded; where one
 * runs out, the rows concerned are written as NaN, which a verify reports as invalid data.
 *   workspace    device scratch of ws_bytes, 16-byte aligned (spec_paged_attention_workspace_size;
 *                no initialisation, free for other uses once the call has run), or NULL, or
 *                less than that or not so aligned: contexts are then not split, which is slower
 *                for few rows and long contexts.
 * 1 <= Q <= 65536, Q * num_q_heads / num_heads < 2^30, head_dim a multiple of 8 (SV_ERR_UNSUPPORTED otherwise), pages, strides
 * and q aligned to 16 bytes (SV_ERR_UNSUPPORTED otherwise).  Errors: SV_ERR_INVALID_ARG for
 * a bad size, pointer or stride (B = 0 returns SV_OK).
 */
SV_API sv_status spec_paged_attention(const void *q, const int64_t *q_stride, int num_q_heads,
                                      const sv_paged_cache *cache, const int32_t *base, const int32_t *new_len,
                                      const uint32_t *tree_mask, float scale, int B, int Q, int max_len, void *out,
                                      float *out_lse, void *workspace, size_t ws_bytes, void *stream);

/* Bytes of workspace that spec_paged_attention can use for such a call (0: none), a
 * function of the sizes and of the current device. */
SV_API size_t spec_paged_attention_workspace_size(int B, int Q, int num_q_heads, int num_heads, int head_dim,
                                                  sv_cache_dtype dtype, int max_len);

/*
 * spec_kv_compact on a paged cache: row base[b] + d <- row base[b] + path[b][d] for
 * d = 0 .. count[b] - 2, every row through the page table, in every buffer.
 *   kv_buffers   HOST array of num_buffers device pointers, 1 <= num_buffers <= 256 (each
 *                layer's K and V pages; their scales in a call of their own, as rows of 4
 *                bytes); row r of page p and plane h (a KV head) of buffer k starts at
 *                kv_buffers[k] + p*page_stride + h*plane_stride + r*row_stride (bytes).
 *                Buffers must not overlap one another.
 *   page_table   device int32 [B][max_pages]; num_pages, page_size as in sv_paged_cache.
 *   path, count, base, row_bytes, B, max_depth  as spec_kv_compact.  base is the cache row
 *                of tree node 0 (one behind the root's).
 * A batch row that spec_kv_compact would leave untouched (count 0 or beyond max_depth + 1,
 * path[d] < d, a negative base, a row beyond the table) is left untouched, and so is one
 * with a hole among the rows it would move.  No page may be in the table twice where it
 * is written.  Errors as spec_kv_compact.
 */
SV_API sv_status spec_kv_compact_paged(void *const *kv_buffers, int num_buffers, int64_t page_stride,
                                       int64_t plane_stride, int num_planes, int64_t row_stride, int64_t row_bytes,
                                       const int32_t *page_table, int num_pages, int page_size, int max_pages,
                                       const int32_t *path, const int32_t *count, const int32_t *base, int B,
                                       int max_depth, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_PAGED_KV_H */
