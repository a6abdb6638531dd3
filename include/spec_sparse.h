/*
 * spec_sparse.h -- attention of the new tokens over some blocks of a long paged cache
 * (spec_paged_kv.h): summaries of the blocks' keys, the blocks that a cheap score against
 * them selects for each query, and attention over the selected blocks.  A block is a page.
 * Same library, status codes and conventions as spec_verify.h (caller-owned device arrays,
 * asynchronous on `stream`, argument errors returned before any launch, SV_ERR_CUDA for
 * launch failures).
 *
 * Defining passages (page title, section): "Speculative Decoding and EAGLE", sections
 * "개념" and "트리 어텐션 검증 (Tree Attention Verification)": the target checks every drafted
 * token in one forward pass over the shared prefix, in a tree each node under its ancestors.
 * The pages give no selection of that prefix; summaries, scores and lists are this library's.
 *
 * The context blocks of batch row b are its blocks 0 .. base[b] / page_size - 1, which the
 * positions before the chunk fill; the blocks from base[b] / page_size on hold the last of
 * those positions and the new tokens, and every query's attention takes them all, under the
 * chain's or the tree's mask.  What is selected is context blocks.
 */
#ifndef SPEC_SPARSE_H
#define SPEC_SPARSE_H

#include "spec_paged_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What is kept of a block's keys. */
typedef enum {
    SV_SUMMARY_MEAN = 0,  /* the mean of each element: head_dim numbers */
    SV_SUMMARY_BOUNDS = 1 /* the largest value of each element, then the smallest: 2 * head_dim */
} sv_summary;

/*
 * Summaries of the blocks that hold a position base[b] .. base[b] + new_len[b] - 1, over all
 * of the block's positions below base[b] + new_len[b], from the cache as it is: called after
 * the positions have been written or moved, it replaces what was there.
 *   cache        as spec_kv_append; values and their scales are not read (v_pages may equal
 *                k_pages).
 *   summary      device bf16 [num_pages][num_heads][head_dim or 2 * head_dim], dense: a page's
 *                summary lies at the page.  Sums and means are fp32, means are rounded to bf16
 *                once; bounds are rounded to nearest (bf16 pages: exact; e4m3 pages: off by up to
 *                half a step to either side).  NaN among an element's values makes it NaN.
 * Blocks in holes are passed over, and so are rows that spec_kv_append leaves untouched.  A
 * page that two rows hold must have the same positions in both.
 * 0 <= N <= 2^30.  Errors: SV_ERR_INVALID_ARG for a bad size, kind, pointer or stride
 * (B = 0 or N = 0 returns SV_OK and launches nothing).
 */
SV_API sv_status spec_block_summary(const sv_paged_cache *cache, const int32_t *base, const int32_t *new_len,
                                    sv_summary kind, int B, int N, void *summary, void *stream);

/*
 * Selects top_k context blocks for each query and cache head, or for all queries of a row
 * (shared not 0).
 *   q            device bf16 [B][Q][num_q_heads][head_dim], element strides q_stride[0..2],
 *                as spec_paged_attention.
 *   summary      as spec_block_summary writes it, of the given kind.
 *   page_table   device int32 [B][max_pages], dense, with base and new_len as
 *                spec_paged_attention.
 * A block's score for a query is the largest, over the heads that share the cache head (and
 * over the row's real queries where shared), of sum_d q_d m_d (mean m), or of
 * sum_d (q_d >= 0 ? q_d max_d : q_d min_d).  On bf16 pages no key of the block has a larger
 * product with q; on e4m3 pages, whose bounds are rounded, none has one that is larger by more
 * than 2^-8 sum_d |q_d| |m_d|, m_d the bound that the sum took.
 * Selected are the first `sink` context blocks, the last `recent` ones, and of the others
 * those with the largest scores, top_k in all (all of them where there are no more).  The
 * order is that of the scores summed in 64 bits; of equal ones the lower block comes first;
 * a score that is not a number is below all others, and a block in a hole below those.
 *   out_blocks   device int32 [B][Q or 1][num_heads][top_k]: the blocks in ascending order,
 *                -1 behind the last one.  Lists of queries that are not real, and of rows that
 *                spec_paged_attention leaves untouched, are all -1.
 *   workspace    device scratch of ws_bytes, 16-byte aligned, at least
 *                spec_block_select_workspace_size (no initialisation, free for other uses
 *                once the call has run).
 * 1 <= Q <= 65536, Q * num_q_heads / num_heads < 2^30, head_dim a multiple of 8 of at most
 * 256, q and summary aligned to 16 bytes and q_stride to 8 elements (SV_ERR_UNSUPPORTED
 * otherwise), B * num_heads <= 65535, max_pages <= 65536, 1 <= top_k <= 4096, 0 <= sink, 0 <= recent,
 * sink + recent <= top_k.  Errors: SV_ERR_INVALID_ARG for a bad size, kind or pointer, or a
 * workspace too small or not aligned (B = 0 returns SV_OK).
 */
SV_API sv_status spec_block_select(const void *q, const int64_t *q_stride, int num_q_heads, const void *summary,
                                   sv_summary kind, const int32_t *page_table, int num_pages, int page_size,
                                   int max_pages, int num_heads, int head_dim, const int32_t *base,
                                   const int32_t *new_len, int shared, int top_k, int sink, int recent, int B, int Q,
                                   int32_t *out_blocks, void *workspace, size_t ws_bytes, void *stream);

SV_API size_t spec_block_select_workspace_size(int B, int Q, int num_q_heads, int num_heads, int max_pages,
                                               int shared);

/*
 * spec_paged_attention over some blocks: each query sees, of what spec_paged_attention would
 * show it, the positions in the listed context blocks and in the blocks from
 * base[b] / page_size on.
 *   blocks       device int32 [B][Q][num_heads][num_blocks], or [B][1][num_heads][num_blocks]
 *                where shared is not 0 (the row's queries share a list).  An entry that is
 *                negative, no context block, or not greater than the last one taken of its list
 *                is passed over.
 *   workspace    device scratch of ws_bytes, 16-byte aligned, at least
 *                spec_sparse_attention_workspace_size (no initialisation, free for other uses
 *                once the call has run).
 * Other arguments, results, numerics, limits and errors as spec_paged_attention; and
 * 0 <= num_blocks <= 4096, page_size * (num_blocks + 2) + Q <= 2^30, B <= 65535 and, where not
 * shared, B * Q * num_heads < 2^31.  A workspace that is too small or not aligned is
 * SV_ERR_INVALID_ARG.
 */
SV_API sv_status spec_sparse_attention(const void *q, const int64_t *q_stride, int num_q_heads,
                                       const sv_paged_cache *cache, const int32_t *base, const int32_t *new_len,
                                       const uint32_t *tree_mask, const int32_t *blocks, int num_blocks, int shared,
                                       float scale, int B, int Q, void *out, float *out_lse, void *workspace,
                                       size_t ws_bytes, void *stream);

/* Bytes of workspace of such a call, a function of the sizes and of the current device; 0
 * for sizes that the call refuses. */
SV_API size_t spec_sparse_attention_workspace_size(int B, int Q, int num_q_heads, int num_heads, int head_dim,
                                                   sv_cache_dtype dtype, int page_size, int num_blocks, int shared);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_SPARSE_H */
