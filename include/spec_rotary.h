/*
 * spec_rotary.h -- rotary positions of the new tokens' queries and keys, for chains and for
 * draft trees, alone or with the keys and values written into a paged cache.  Same library,
 * status codes and conventions as spec_verify.h (caller-owned device arrays, asynchronous
 * on `stream`, argument errors returned before any launch, SV_ERR_CUDA for launch failures).
 *
 * Defining passage (page title, section): "Speculative Decoding and EAGLE", section "트리
 * 어텐션 검증 (Tree Attention Verification)": one forward pass checks every branch, so a
 * node's position follows from its depth and not from its place among the tokens.  The
 * pages give no formula of positions; this is the rotation of pairs of elements by an angle
 * that grows with the position.
 */
#ifndef SPEC_ROTARY_H
#define SPEC_ROTARY_H

#include "spec_paged_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * How elements are turned.  A pair (x, y) of a head's first 2 * num_freq elements becomes
 *   amplitude * (x cos t - y sin t, y cos t + x sin t),   t = position * freq[j],
 * with the pairs (j, j + num_freq), or (2 j, 2 j + 1) where interleaved is not 0; the other
 * way (-t) where inverse is not 0.  Elements from 2 * num_freq on are copied.
 *   freq         device double [num_freq]: radians per position, finite.
 *   tree_depth   NULL: token i of batch row b has position base[b] + i; device int32
 *                [B][N-1] as spec_tree_mask writes it for the N - 1 nodes of draft trees:
 *                token 0 (the root) has position base[b], token i + 1 base[b] + tree_depth[b][i].
 * Angles are within 2^-24 of a turn up to 2^24 positions, and within 2^-19 up to 2^30, for
 * frequencies of at most 1 radian.  Products are fp32, results are rounded once to their type.
 * The struct is read during the call and is not retained.
 *   0 <= num_freq <= 128, 2 * num_freq <= head_dim.
 */
typedef struct {
    const double *freq;
    const int32_t *tree_depth;
    float amplitude;
    int num_freq, interleaved, inverse;
} sv_rotary;

/*
 * Turns queries and keys.
 *   q, k         device [B][N][num_q_heads][head_dim] and [B][N][num_k_heads][head_dim], dtype
 *                dt (SV_F32 or SV_BF16), element strides q_stride[0..2], k_stride[0..2] (batch,
 *                token, head; HOST int64 arrays of three), contiguous elements.  k may be NULL
 *                with num_k_heads 0.
 *   base, new_len  device int32 [B]; new_len may be NULL (N for every row).  Rows with a
 *                base outside [0, 2^30] or a new_len outside [0, N], and tokens i >= new_len[b],
 *                are not written.
 *   out_q, out_k  device, same types, element strides out_q_stride, out_k_stride.  Each is
 *                its input itself, with its strides, or does not overlap it.
 * 1 <= head_dim <= 256, 1 <= num_q_heads <= 65536, 0 <= num_k_heads <= 65536,
 * 0 <= B <= 65535, 0 <= N <= 2^20, B * N < 2^31.  Errors: SV_ERR_INVALID_ARG for a bad size,
 * dtype, pointer, stride or number (B = 0 or N = 0 returns SV_OK and launches nothing).
 */
SV_API sv_status spec_rotary(const void *q, const int64_t *q_stride, int num_q_heads, const void *k,
                             const int64_t *k_stride, int num_k_heads, sv_dtype dt, const sv_rotary *rotary,
                             const int32_t *base, const int32_t *new_len, int B, int N, int head_dim, void *out_q,
                             const int64_t *out_q_stride, void *out_k, const int64_t *out_k_stride, void *stream);

/*
 * The same for queries, and keys and values written into a paged cache in one pass, as
 * spec_kv_append writes them: the keys turned (fp32 until the cache's rounding), the values
 * as they are.  A key's cache row is base[b] + i, whatever its position.
 *   q, out_q     as above (out_q_stride alike); q may be NULL with num_q_heads 0.
 *   key, value   device [B][N][cache->num_heads][cache->head_dim], element strides
 *                kv_stride[0..2], which both share.
 * Other arguments, rows that are left untouched, limits and errors as spec_rotary and
 * spec_kv_append (0 <= num_q_heads <= 65536).
 */
SV_API sv_status spec_rotary_append(const void *q, const int64_t *q_stride, int num_q_heads, const void *key,
                                    const void *value, const int64_t *kv_stride, sv_dtype dt, const sv_rotary *rotary,
                                    const sv_paged_cache *cache, const int32_t *base, const int32_t *new_len, int B,
                                    int N, void *out_q, const int64_t *out_q_stride, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_ROTARY_H */
