/*
 * hadarot_cache -- a paged key/value cache held in 4 bits: writing rotated
 * keys and values into pages, attention over them, and the moves of pages
 * when sequences are forked, grown, cut, freed or compacted.
 *
 * The conventions of hadarot.h hold here too: plain pointers and sizes, an
 * hr_status per call, every argument checked before anything is enqueued,
 * asynchronous launches on `stream`, buffers owned by the caller, no device
 * memory allocated and kernel launches only, so a call may be captured in a
 * HIP graph (after one call of the same kernel outside the capture).
 *
 * The page record.  A pool is n_pages records of page_bytes bytes each (and,
 * where several layers share one page table, `layers` such pools one after
 * the other).  A page holds page_size consecutive positions of one sequence,
 * one head after the other; a head's part holds, each section 16-byte and
 * each head 128-byte aligned,
 *     codes of K, codes of V    page_size * head_dim / 2 bytes each
 *     scales of K, scales of V  page_size * head_dim / group_size values each
 *     zeros of K, zeros of V    half a byte for each scale (asymmetric only)
 * Every section is what rotate_quantize_act writes for [page_size, head_dim]
 * rows, so dequant_check reads it.  hr_cache_page_layout gives the offsets.
 * A head's keys, values and scales of page_size positions are therefore one
 * run of memory, and a page of all heads is one record to copy.
 *
 * The page table.  int32 [rows, max_pages], row-major: entry j of a row is
 * the page of positions j * page_size ... of that sequence.  An entry outside
 * [0, n_pages) (-1 by convention) is an absent page: its positions hold no
 * keys for attention, and appends to them are dropped.  lens[row] is the
 * number of positions of the sequence, new ones included, clamped to
 * [0, max_pages * page_size].  One page may stand in several rows; nothing
 * counts its holders between calls.
 *
 * New tokens.  The tokens of a call are packed row after row: row b owns
 * tokens cu_q[b] ... cu_q[b + 1] - 1 of the call (int32 [rows + 1],
 * cu_q[0] = 0, not decreasing, cu_q[rows] = tokens), the last of them at position
 * lens[b] - 1.  cu_q NULL: every row has tokens / rows of them.  Values that
 * break these rules are clamped so that no access leaves a buffer; the result
 * is then unspecified.
 */
#ifndef HADAROT_CACHE_H
#define HADAROT_CACHE_H

#include "hadarot.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What a cache holds.  head_dim 64, 128 or 256; page_size 16, 32, 64, 128 or
 * 256; q: format HR_Q_INT, 4 bits, symmetric or asymmetric, group_size a
 * power of two from 32 to head_dim, scales HR_F32 or HR_BF16.  MXFP4 and
 * NVFP4 pages are not implemented (HR_EUNSUPPORTED). */
typedef struct hr_cache_spec {
    int32_t kv_heads;
    int32_t head_dim;
    int32_t page_size;
    hr_qspec q;
} hr_cache_spec;

/* Byte offsets inside a page: head h starts at h * head_bytes, and its
 * sections at these offsets from there (zeros: 0 if symmetric). */
typedef struct hr_cache_page {
    int64_t page_bytes, head_bytes;
    int64_t k_codes, v_codes, k_scales, v_scales, k_zeros, v_zeros;
} hr_cache_page;

/* The sequences of a call (see "The page table" and "New tokens"). */
typedef struct hr_cache_seqs {
    const int32_t* table;   /* device, [rows, max_pages] */
    const int32_t* lens;    /* device, [rows] */
    const int32_t* cu_q;    /* device, [rows + 1], or NULL */
    int64_t rows;
    int64_t max_pages;
} hr_cache_seqs;

/* Host-only: the layout of a page. */
int hr_cache_page_layout(const hr_cache_spec* spec, hr_cache_page* out);

/*
 * Writes the new tokens' keys and values into their pages: each key vector
 * is rotated by H / sqrt(head_dim) if `rotate` is not 0 (R3; the value
 * vectors never are), and both are quantized with spec->q as in
 * rotate_quantize_act, from the float32 values.  A group with a NaN gets a NaN
 * scale (its codes do not matter then), so attention gives NaN to the tokens
 * that see it.
 *   pool    device, [n_pages, page_bytes], 16-byte aligned.
 *   k, v    device, element (t, h, i) at t * stride_token + h * stride_head
 *           + i (strides in elements, so a slice of a fused projection's
 *           output can be passed); rows 16-byte aligned, `dtype` HR_F32 or
 *           HR_BF16.
 * A page that several rows hold must not be written: hr_cache_update gives a
 * row that grows a page of its own.  A byte of zero points that holds a
 * neighbouring position's too keeps that half.
 */
int hr_cache_append(void* pool, int64_t n_pages, const hr_cache_spec* spec, const hr_cache_seqs* seqs,
                    const void* k, int64_t k_stride_token, int64_t k_stride_head,
                    const void* v, int64_t v_stride_token, int64_t v_stride_head,
                    int dtype, int64_t tokens, int rotate, void* stream);

/*
 * Attention of the new tokens over the cache:
 *   out(t, h) = sum_j softmax_j(scale q'(t, h) . k_j) v_j
 * over the positions j of the token's own sequence that it sees, with k_j and
 * v_j the dequantized vectors of kv head h / (q_heads / kv_heads) and q' the
 * query, rotated by H / sqrt(head_dim) if `rotate` is not 0.  The new tokens'
 * own keys and values are read from the cache: append them first.
 *   causal  0: every position below lens.  1: positions up to the token's own.
 *   window  0: no limit; w > 0 (causal only): the last w of those positions.
 * Positions of absent pages are not seen.  What a token does not see has no
 * influence, whatever its bytes are.  A token that sees nothing gets zeros
 * (and a log-sum-exp of -inf).  Keys whose scales are far from their
 * neighbours', by 2^10 and more, may be taken one at a time, which is slower.
 *   q, out  device, element (t, h, i) at t * stride_token + h * stride_head
 *           + i; 16-byte aligned rows; `dtype` HR_F32 or HR_BF16.  out may be
 *           q with the same strides.
 *   scale   positive and finite; 0 means 1 / sqrt(head_dim).
 *   lse     device float32 [tokens, q_heads] or NULL: the natural logarithm of
 *           the softmax's sum of exponentials.
 *   max_q   an upper bound of one row's new tokens, or 0 if not known (the
 *           mean is taken).  It only chooses the kernel: a larger row is
 *           still computed in full.
 *   work    device scratch of at least the bytes that
 *           hr_cache_attention_work gives for the same arguments, 16-byte
 *           aligned.  Contents do not matter.
 * Products use float16 operands with float32 sums for HR_BF16: the queries and
 * probabilities carry 11 bits, and so do scale (c - z) of values in several
 * groups and, where a call has many new tokens, of all keys and values (which
 * is exact with bfloat16 scales but for |c - z| of 9, 11, 13 and 15); the codes
 * are exact otherwise.  The log-sum-exp of such a call errs by up to 2^-12 by
 * the rounding of its probabilities.  HR_F32 takes pairs of float16 (22 bits).
 * The result does not depend on scheduling:
 * partial sums over a long sequence are joined in a fixed order.
 */
int hr_cache_attention(const void* q, int64_t q_stride_token, int64_t q_stride_head,
                       int dtype, int64_t tokens, int32_t q_heads,
                       const void* pool, int64_t n_pages, const hr_cache_spec* spec, const hr_cache_seqs* seqs,
                       float scale, int causal, int64_t window, int rotate,
                       void* out, int64_t out_stride_token, int64_t out_stride_head, float* lse,
                       int64_t max_q, void* work, int64_t work_bytes, void* stream);

/* Bytes of scratch for the call with these arguments on the current device. */
int hr_cache_attention_work(int dtype, int64_t tokens, int32_t q_heads, const hr_cache_spec* spec,
                            int64_t rows, int64_t max_q, int64_t* bytes);

/*
 * One scheduling step over the page table: forking, growing, cutting back and
 * freeing sequences.  Row i of the new table continues row parents[i] of the
 * old one (an index outside [0, rows): a new, empty sequence) with
 * len = clamp(lens[parents[i]] + grow[i], 0, max_pages * page_size) positions.
 *   - Pages of the common prefix are shared; rows of the old table that are
 *     nobody's parent give theirs up.
 *   - A row that grows into a partly filled page must own it.  If other new
 *     rows hold that page too, the lowest-numbered growing row keeps it,
 *     provided that every holder grows into it; the others get a copy (of
 *     all layers).
 *   - Further pages are fresh.  Pages that no new row inherits are free, and
 *     are handed out in ascending order: row by row, a row's copy first.
 *     When none is left the entry is -1.
 *   pool       device, [layers, n_pages, page_bytes]: the copies are made here.
 *   new_table  device, int32 [new_rows, max_pages], -1 past each length;
 *   new_lens   device, int32 [new_rows];
 *   refs       device, int32 [n_pages]: how many entries of the new table
 *              hold each page;
 *   status     device, int32 [4]: pages in use, pages that were lacking,
 *              pages copied, pages left free.
 *   work       device scratch of hr_cache_update_work bytes, 16-byte aligned.
 * The old table and lens are only read and may not overlap the new ones; each
 * has fewer than 2^31 entries.
 */
int hr_cache_update(void* pool, int64_t layers, int64_t n_pages, const hr_cache_spec* spec,
                    const int32_t* table, const int32_t* lens, int64_t rows, int64_t max_pages,
                    const int32_t* parents, const int32_t* grow, int64_t new_rows,
                    int32_t* new_table, int32_t* new_lens, int32_t* refs, int32_t* status,
                    void* work, int64_t work_bytes, void* stream);
int hr_cache_update_work(int64_t n_pages, int64_t new_rows, int64_t* bytes);

/*
 * Moves the pages that the table holds together.
 *   into NULL: within the pool.  With n live pages, those at n and above move
 *     to the free places below n, both in ascending order; the others stay.
 *   into given: every live page is copied to the pool `into`, [layers,
 *     into_pages, page_bytes], in ascending order from page 0; pages past
 *     into_pages are not, and their entries become -1.
 *   new_table  device, int32 [rows, max_pages]: the table in the new places,
 *              -1 past each length;
 *   refs       device, int32 [n_pages], or [into_pages] with into: entries
 *              that hold each page;
 *   status     device, int32 [4]: live pages, pages that found no place,
 *              pages moved, places left free.
 *   work       device scratch of hr_cache_compact_work bytes, 16-byte aligned.
 * Lengths do not change.  The old table is only read and may not overlap the
 * new one; each has fewer than 2^31 entries; `into` may not overlap the pool.
 */
int hr_cache_compact(void* pool, int64_t layers, int64_t n_pages, const hr_cache_spec* spec,
                     const int32_t* table, const int32_t* lens, int64_t rows, int64_t max_pages,
                     void* into, int64_t into_pages,
                     int32_t* new_table, int32_t* refs, int32_t* status,
                     void* work, int64_t work_bytes, void* stream);
int hr_cache_compact_work(int64_t n_pages, int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* HADAROT_CACHE_H */
