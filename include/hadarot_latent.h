/*
 * hadarot_latent -- latent attention over a paged 4-bit cache: instead of keys and
 * values of every head a position holds one vector, the latent, that all heads'
 * keys and values are linear maps of, and one rotary key that all heads share.
 *
 * Conventions, page tables, sequences and new tokens are those of
 * hadarot_cache.h: every argument is checked before anything is enqueued,
 * launches are asynchronous on `stream`, buffers are the caller's, no device
 * memory is allocated and only kernels are launched, so a call may be captured
 * in a HIP graph (after one call of the same kernel outside the capture).
 *
 * The page record.  A page holds page_size consecutive positions of one sequence,
 * each section 16-byte and the record 128-byte aligned:
 *     codes        page_size * latent_dim / 2 bytes
 *     scales       page_size * latent_dim / group_size values
 *     zeros        half a byte for each scale (asymmetric only)
 *     rotary keys  page_size * rope_dim bfloat16
 * The first three are what rotate_quantize_act writes for [page_size, latent_dim]
 * rows, so dequant_check reads them.
 *
 * hr_cache_update and hr_cache_compact move such pages by hr_latent_update and
 * hr_latent_compact, whose arguments are the same but for the spec.
 */
#ifndef HADAROT_LATENT_H
#define HADAROT_LATENT_H

#include "hadarot_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What a cache of latents holds.  latent_dim 256 or 512; rope_dim 64; page_size 16,
 * 32, 64, 128 or 256; q: format HR_Q_INT, 4 bits, symmetric or asymmetric,
 * group_size a power of two from 128 to latent_dim, scales HR_F32 or HR_BF16. */
typedef struct hr_latent_spec {
    int32_t latent_dim;
    int32_t rope_dim;
    int32_t page_size;
    hr_qspec q;
} hr_latent_spec;

/* Bytes of a page, and offsets of its sections (zeros: 0 if symmetric). */
typedef struct hr_latent_page {
    int64_t page_bytes;
    int64_t codes, scales, zeros, rope;
} hr_latent_page;

/* Host-only: the layout of a page. */
int hr_latent_page_layout(const hr_latent_spec* spec, hr_latent_page* out);

/*
 * Writes the new tokens' latents and rotary keys into their pages: a latent is
 * rotated by H / sqrt(latent_dim) if `rotate` is not 0 and quantized with spec->q
 * as in rotate_quantize_act, from the float32 values (a group with a NaN gets a
 * NaN scale); a rotary key is rounded to bfloat16.
 *   c, rope  device, element (t, i) at t * stride + i, rows 16-byte aligned,
 *            `dtype` HR_F32 or HR_BF16.
 * Otherwise as hr_cache_append.
 */
int hr_latent_append(void* pool, int64_t n_pages, const hr_latent_spec* spec, const hr_cache_seqs* seqs,
                     const void* c, int64_t c_stride, const void* rope, int64_t rope_stride,
                     int dtype, int64_t tokens, int rotate, void* stream);

/*
 * Takes latents and rotary keys out of the pages: output row cu_q[b] + j is
 * position j of sequence b, for as many positions as cu_q gives the sequence
 * (seqs->cu_q NULL: positions / rows of each).  Latents are dequantized and, if
 * `rotate` is not 0, rotated back.  Positions past lens[b] and those of absent
 * pages give zeros.
 *   c, rope  device, element (p, i) at p * stride + i, rows 16-byte aligned,
 *            `dtype` HR_F32 or HR_BF16.
 */
int hr_latent_read(const void* pool, int64_t n_pages, const hr_latent_spec* spec, const hr_cache_seqs* seqs,
                   void* c, int64_t c_stride, void* rope, int64_t rope_stride,
                   int dtype, int64_t positions, int rotate, void* stream);

/*
 * Attention of the new tokens over the cached latents (the absorbed form: queries
 * have been multiplied by the map from latents to keys, and the map to values is
 * applied to the result):
 *   w_j(t, h) = scale (q'(t, h) . c_j + q_rope(t, h) . r_j)
 *   out(t, h) = (sum_j softmax_j(w(t, h)) c_j) H / sqrt(latent_dim)
 * over the positions j of the token's own sequence that it sees, with c_j the
 * dequantized latent, r_j the rotary key, and q' = q H / sqrt(latent_dim).  With
 * `rotate` 0 neither q nor the result is rotated: for maps that H has been fused
 * into (rotate_fuse_weight).  The new tokens' own latents are read from the cache:
 * append them first.
 *   causal   0: every position below lens.  1: positions up to the token's own.
 *   q, out   device, element (t, h, i) at t * stride_token + h * stride_head + i,
 *            latent_dim elements a row; q_rope the same with rope_dim; rows
 *            16-byte aligned, `dtype` HR_F32 or HR_BF16.
 *   scale    positive and finite.
 *   lse, max_q, work  as in hr_cache_attention; max_pages * page_size at most 2^31 -
 *            2^16 (else HR_EUNSUPPORTED).
 * Positions of absent pages are not seen; what a token does not see has no
 * influence, whatever its bytes are.  A token that sees nothing gets zeros (and a
 * log-sum-exp of -inf).  Scales are the append's: positive, or NaN; an infinite one,
 * of an infinite latent, counts as NaN, which the tokens that see it get.
 * Products use float16 operands with float32 sums for HR_BF16: codes are exact,
 * queries and probabilities carry 11 bits (a pair of float16, 22 bits, for
 * HR_F32), and the products with rotary keys are exact.  An element of a query has
 * 11 of them down to 2^-27 of the row's largest, or to 2^-114 of its rotary query's
 * largest, and a probability times its latent's scale down to 2^-22 of the row's
 * largest; 22 down to 2^-15, 2^-102 and 2^-10.  Scales below 2^-92 or above 2^100 cost
 * more.  The result does not depend on scheduling: partial sums over a long sequence
 * are joined in a fixed order.
 */
int hr_latent_attention(const void* q, int64_t q_stride_token, int64_t q_stride_head,
                        const void* q_rope, int64_t q_rope_stride_token, int64_t q_rope_stride_head,
                        int dtype, int64_t tokens, int32_t heads,
                        const void* pool, int64_t n_pages, const hr_latent_spec* spec, const hr_cache_seqs* seqs,
                        float scale, int causal, int rotate,
                        void* out, int64_t out_stride_token, int64_t out_stride_head, float* lse,
                        int64_t max_q, void* work, int64_t work_bytes, void* stream);

/* Bytes of scratch for the call with these arguments on the current device. */
int hr_latent_attention_work(int dtype, int64_t tokens, int32_t heads, const hr_latent_spec* spec,
                             int64_t rows, int64_t max_q, int64_t* bytes);

/*
 * Attention of prompts over keys and values made from latents (the expanded form):
 *   w_j(t, h) = scale (q(t, h)[0, nope) . k(j, h) + q(t, h)[nope, nope + rope) . r_j)
 *   out(t, h) = sum_j softmax_j(w(t, h)) v(j, h)
 * Sequence b has the tokens cu_q[b] ... cu_q[b + 1] - 1 and the positions cu_k[b]
 * ... cu_k[b + 1] - 1 (int32 [rows + 1] both, from 0, not decreasing, the last
 * entry tokens or positions); its last token is at its last position.
 *   causal   0: every position of the sequence.  1: positions up to the token's own.
 *   nope     elements of a key, and of a value, of one head: 64 or 128.  The rotary
 *            keys have 64, queries nope + 64.
 *   q, out, k, v  device, element (t or j, h, i) at stride_token and stride_head
 *            as above; rope (j, i) at j * rope_stride + i; rows 16-byte aligned.
 *   dtype    HR_BF16 (float32 is not implemented: HR_EUNSUPPORTED).
 *   scale    positive and finite; 0 means 1 / sqrt(nope + 64).
 *   lse      device float32 [tokens, heads] or NULL.
 * A token that sees nothing gets zeros (and -inf); positions that it does not see
 * have no influence.  Queries, keys and values are exact, probabilities are rounded
 * to bfloat16, sums are float32.
 */
int hr_latent_prompt_attention(const void* q, int64_t q_stride_token, int64_t q_stride_head,
                               const void* k, int64_t k_stride_token, int64_t k_stride_head,
                               const void* v, int64_t v_stride_token, int64_t v_stride_head,
                               const void* rope, int64_t rope_stride,
                               int dtype, int64_t tokens, int64_t positions, int32_t heads, int32_t nope,
                               const int32_t* cu_q, const int32_t* cu_k, int64_t rows,
                               float scale, int causal,
                               void* out, int64_t out_stride_token, int64_t out_stride_head, float* lse, void* stream);

/* hr_cache_update and hr_cache_compact of a pool of latent pages. */
int hr_latent_update(void* pool, int64_t layers, int64_t n_pages, const hr_latent_spec* spec,
                     const int32_t* table, const int32_t* lens, int64_t rows, int64_t max_pages,
                     const int32_t* parents, const int32_t* grow, int64_t new_rows,
                     int32_t* new_table, int32_t* new_lens, int32_t* refs, int32_t* status,
                     void* work, int64_t work_bytes, void* stream);
int hr_latent_compact(void* pool, int64_t layers, int64_t n_pages, const hr_latent_spec* spec,
                      const int32_t* table, const int32_t* lens, int64_t rows, int64_t max_pages,
                      void* into, int64_t into_pages,
                      int32_t* new_table, int32_t* refs, int32_t* status,
                      void* work, int64_t work_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HADAROT_LATENT_H */
