/*
 * spec_logits.h -- what a server does to the target's logits before it verifies drafts:
 * penalties for repeated tokens, biases and grammar masks, for every position of a chain
 * or a tree at once.  Same library, status codes and conventions as spec_verify.h.
 *
 * Defining passage (page title, section): "Speculative Decoding and EAGLE", section
 * "정확성 규칙 (The Exactness Rule)": the verify samples from the target's own
 * distribution, so whatever shapes that distribution is applied to the target's logits of
 * every drafted position before the rule.  The pages give no penalties; the usual
 * repetition, presence and frequency penalties are meant.
 */
#ifndef SPEC_LOGITS_H
#define SPEC_LOGITS_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * out[b][r][v] from logits[b][r][v], r = 0..R-1 the rows of a verify call (row 0 the last
 * emitted token's, row i + 1 the row after drafted token or tree node i).  Let c be the
 * number of times token v occurs in the row's output so far: in the history from
 * prompt_len[b] on, plus among the drafted tokens that row r follows (a chain: drafts
 * 0..r-1; a tree: node r-1 and its ancestors).  Let v be seen if c > 0 or v is in the
 * history before prompt_len[b].  Then
 *   x = logits[b][r][v]
 *   x = x / repetition[b] if x > 0, else x * repetition[b]        where v is seen
 *   x = x - c * frequency[b] - presence[b] * (c > 0)
 *   x = x + bias of v
 *   x = -inf                                                       where v is not allowed
 * in fp32, rounded once to the logits' type.  A row that allows nothing becomes all -inf,
 * which the verify reports as invalid data.  NaN survives unless its token is not allowed.
 *   logits       device [B][R][V], dtype dt (SV_F32 or SV_BF16).
 *   out          device [B][R][V], same dtype: another array, or logits itself (in place;
 *                then only the entries that change are touched).  Partial overlap is not
 *                allowed.
 *   history      device int32 [B][H], history_len, prompt_len device int32 [B]: tokens
 *                0 .. history_len[b]-1 count (clamped to [0, H]), those before
 *                prompt_len[b] as the prompt.  history may be NULL (H = 0); prompt_len
 *                NULL: no prompt.  Tokens outside [0, V) are ignored, everywhere.
 *   draft_tokens device int32 [B][R-1], or NULL: no drafted token counts.
 *   tree_mask    NULL (a chain), or device uint32 [B][R-1][W], W = ceil((R-1) / 32), as
 *                spec_tree_mask writes it.
 *   repetition, presence, frequency  device fp32 [B], each or NULL (no such penalty);
 *                repetition > 0.
 *   bias_tokens  device int32 [B][M], bias_values device fp32 [B][M], or NULL (M = 0).
 *                Where a token is listed twice the later entry holds; a negative token is
 *                an empty entry.
 *   allowed      device uint32 [B][R][ceil(V / 32)] or NULL: bit v % 32 of word v / 32 is
 *                set iff v is allowed in that row.
 *   0 <= B <= 65535, 1 <= R <= 1025, 1 <= V <= 1<<24, 0 <= H < 2^31 - 1, 0 <= M <= 65535.
 * Errors: SV_ERR_INVALID_ARG for a bad size, dtype or pointer (B = 0 returns SV_OK).
 */
SV_API sv_status spec_adjust_logits(const void *logits, sv_dtype dt, const int32_t *history,
                                    const int32_t *history_len, const int32_t *prompt_len, int H,
                                    const int32_t *draft_tokens, const uint32_t *tree_mask, const float *repetition,
                                    const float *presence, const float *frequency, const int32_t *bias_tokens,
                                    const float *bias_values, int M, const uint32_t *allowed, int B, int R, int V,
                                    void *out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_LOGITS_H */
