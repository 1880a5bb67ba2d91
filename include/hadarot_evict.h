/*
 * hadarot_evict -- fewer positions in the paged 4-bit cache of hadarot_cache.h:
 * the attention weight that every cached position gets, added up over the new
 * tokens of a step, and the eviction of the positions that got least.
 *
 * Conventions, page records, page tables and sequences are those of
 * hadarot_cache.h: every argument is checked before anything is enqueued,
 * launches are asynchronous on `stream`, buffers are the caller's, no device
 * memory is allocated and only kernels are launched, so a call may be captured
 * in a HIP graph (after one call of the same kernel outside the capture).
 *
 * The weights.  float32 [rows, kv_heads, width] (where several layers share one
 * page table, `layers` of them one after the other), width at least max_pages *
 * page_size: one number for every position of every kv head.
 */
#ifndef HADAROT_EVICT_H
#define HADAROT_EVICT_H

#include "hadarot_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Adds the attention weights of a step's new tokens, after hr_cache_attention
 * of the same q, pool, seqs, scale, causal, window and rotate has given `lse`:
 *   weights(b, h, j) = (j < lens[b] - n(b) ? decay weights(b, h, j) : 0)
 *                      + sum over tokens t of row b and query heads i of kv head
 *                        h that see j of exp(scale q'(t, i) . k_j - lse(t, i))
 * for j < lens[b], with n(b) the row's new tokens: a position that is new starts
 * at 0 whatever was there.  Positions past lens, and all of a row without new
 * tokens, are left as they are.  A token whose lse is -inf adds nothing, whatever
 * its query is (a padded one's may be NaN).
 *   q        as in hr_cache_attention; queries carry 22 bits here for both
 *            types, so that the weights have float32's precision.
 *   lse      device float32 [tokens, q_heads].
 *   decay    finite, not negative; 1 keeps the sum over all steps.
 *   weights  device float32, read and written.
 *   max_q    an upper bound of one row's new tokens, or 0 if not known.
 *   work     device scratch of hr_cache_weights_work bytes, 16-byte aligned.
 * max_pages * page_size: at most 2^31 - 2^16 (else HR_EUNSUPPORTED).
 * Sums are taken in a fixed order: the result does not depend on scheduling.
 */
int hr_cache_weights(const void* q, int64_t q_stride_token, int64_t q_stride_head,
                     int dtype, int64_t tokens, int32_t q_heads,
                     const void* pool, int64_t n_pages, const hr_cache_spec* spec, const hr_cache_seqs* seqs,
                     const float* lse, float scale, int causal, int64_t window, int rotate,
                     float decay, float* weights, int64_t width, int64_t max_q,
                     void* work, int64_t work_bytes, void* stream);
int hr_cache_weights_work(int dtype, int64_t tokens, int32_t q_heads, const hr_cache_spec* spec,
                          int64_t rows, int64_t max_q, int64_t* bytes);

/*
 * Evicts: every row with more than `budget` positions keeps `budget` of them,
 * in every layer and kv head a choice of its own,
 *   - the first `sinks` and the last `recent` positions,
 *   - of the others those with the largest weights (of equal ones the first; a
 *     NaN counts as larger than every number),
 * moved to positions 0 ... budget - 1 in their order: keys, values, scales, zero
 * points and weights.  Its length becomes budget.  Positions and weights past
 * the new length are left as they are; so is every row of at most budget
 * positions, and one with an absent page below its length.
 * A page that several entries of the table hold is not written: the row gets a
 * free page in its place, one that no entry holds, handed out in ascending order
 * row by row.  Where the free pages run out, that row and the later ones that
 * need any are left as they are.  Pages past a row's new length are given up.
 *   pool       device, [layers, n_pages, page_bytes], written in place.
 *   table      device, int32 [rows, max_pages]; lens device, int32 [rows].
 *   weights    device, float32 [layers, rows, kv_heads, width].
 *   budget     positive; sinks, recent not negative, together at most budget.
 *   new_table  device, int32 [rows, max_pages], -1 past each length;
 *   new_lens   device, int32 [rows];
 *   refs       device, int32 [n_pages]: entries of the new table that hold each
 *              page;
 *   status     device, int32 [4]: pages in use, pages that were lacking, rows
 *              evicted, pages left free.
 *   work       device scratch of hr_cache_evict_work bytes, 16-byte aligned.
 * The old table and lens are only read and may not overlap the new ones; each
 * table has fewer than 2^31 entries.
 */
int hr_cache_evict(void* pool, int64_t layers, int64_t n_pages, const hr_cache_spec* spec,
                   const int32_t* table, const int32_t* lens, int64_t rows, int64_t max_pages,
                   float* weights, int64_t width, int64_t budget, int64_t sinks, int64_t recent,
                   int32_t* new_table, int32_t* new_lens, int32_t* refs, int32_t* status,
                   void* work, int64_t work_bytes, void* stream);
int hr_cache_evict_work(int64_t n_pages, int64_t rows, int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* HADAROT_EVICT_H */
