/*
 * spec_pages.h -- page tables of a paged key/value cache (spec_paged_kv.h) kept on the
 * device: rows grow and shrink to lengths that are device data, pages come from and go
 * back to a stack of free ones, and new tokens get their slots.  Same library, status
 * codes and conventions as spec_verify.h (caller-owned device arrays, asynchronous on
 * `stream`, argument errors returned before any launch, SV_ERR_CUDA for launch failures).
 *
 * Defining passage (page title, section): "[논문 리뷰] Fast Inference from Transformers
 * via Speculative Decoding", section 4 "한계점": the cache entries of rejected tokens are
 * rolled back, by a number of tokens that the verify leaves on the device.  The pages give
 * no cache layout; the page table and the stack of free pages are this library's own.
 */
#ifndef SPEC_PAGES_H
#define SPEC_PAGES_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Brings every batch row to the pages that its length needs, ceil(length[b] / page_size).
 *   page_table   device int32 [B][max_pages], in place; the row's pages are the entries
 *                below pages[b].
 *   pages        device int32 [B], in place: pages that the row holds.
 *   length       device int32 [B]: positions that the row is to hold.
 *   free_pages   device int32 [num_pages], in place: a stack of free pages, the lowest
 *                free_count[0] entries (device int32 [1], in place; read as if within
 *                [0, num_pages]).
 * Rows that hold more pages than they need push the others, row by row and within a row
 * by index, and their entries become -1; an entry that is no page (outside
 * [0, num_pages): a hole) is not pushed.  Then the rows that lack pages take them from the
 * top of the stack, row by row and within a row by index.  The first row that finds too
 * few, and every later row that lacks pages, stays as it is.  Entries that are not pushed
 * or taken, and the stack above the new free_count, are not written.  A page must stand in
 * the table at most once among the rows' pages, and not on the stack as well: rows that
 * share pages must not be shrunk into them.  Pushes beyond num_pages entries are dropped.
 *   out_ok       device int32 [B]: 1 where the row now holds its length; 0 where there were
 *                too few pages, or where length[b] is outside [0, max_pages * page_size] or
 *                pages[b] outside [0, max_pages] (the row is left untouched).
 *   base, out_slots  both or neither: device int32 [B], int64 [B][N]: the place of
 *                position base[b] + i, i < N: page * page_size + position % page_size;
 *                -1 for a position that is negative, not below length[b], in a hole, or of a
 *                row whose out_ok is 0.
 * No array may overlap another.
 * 0 <= B <= 16384, 0 <= num_pages <= 2^30, 1 <= page_size <= 65536, 1 <= max_pages,
 * max_pages * page_size <= 2^30, 0 <= N <= 2^30, B * N < 2^40.  Errors:
 * SV_ERR_INVALID_ARG for a bad size or pointer (B = 0 returns SV_OK and launches nothing).
 */
SV_API sv_status spec_page_resize(int32_t *page_table, int32_t *pages, const int32_t *length, int32_t *free_pages,
                                  int32_t *free_count, int num_pages, int page_size, int max_pages,
                                  const int32_t *base, int64_t *out_slots, int32_t *out_ok, int B, int N,
                                  void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_PAGES_H */
