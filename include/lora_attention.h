/*
 * lora_attention.h - C ABI of the operators that stand around the low-rank
 * projections in an attention layer: the norm in front of a projection, the
 * position rotation and cache write behind it, and attention over the cache.
 * They live in the same library and keep its conventions (lora_mi355x.h):
 *   - bf16 tensors are raw uint16 bit patterns; every pointer is a DEVICE
 *     pointer; nothing is allocated, synchronised or kept between calls.
 *   - Arguments are validated on the host before anything is enqueued.  Launch
 *     grids depend on the size arguments only, so calls can be captured into a
 *     HIP graph and replayed on other lengths, places and page tables.
 *   - Bad device data (a place, page or position out of range) cannot raise an
 *     error without a synchronisation; each call states what it does instead.
 *     No such value makes a kernel read or write outside its buffers.
 *   - Inputs are never written; outputs are written only where stated.
 *   - num_tokens is at most 2^22.
 *   - A call over zero tokens (or sequences) returns LORA_OK and enqueues
 *     nothing; its tensors may then be NULL.
 *
 * The 4-bit cache: uint8 [num_pages][2][kv_heads][page_bytes], 16-byte aligned,
 * part 0 the keys and part 1 the values.  The page_bytes = page_size *
 * (head_dim / 2 + head_dim / 32) bytes of one page of one head hold
 *   codes   [page_size][head_dim / 2]   two 4-bit codes a byte, the even element
 *                                       in the low half: sign, two exponent bits,
 *                                       one mantissa bit, the magnitudes
 *                                       0, 0.5, 1, 1.5, 2, 3, 4, 6;
 *   scales  [head_dim / 32][page_size]  one byte b for each 32 elements of one
 *                                       token's head: 2^(b - 127) for b in
 *                                       [2, 252], NaN for b = 255; lora_kv_append
 *                                       writes no others.
 * An element is its code's value times its block's scale, a bf16 number exactly.
 * A place (slot) is page * page_size + offset in the page.
 */
#ifndef LORA_ATTENTION_H
#define LORA_ATTENTION_H

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "lora_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * lora_rms_norm - the residual's addition and the root-mean-square norm of each
 * token's row, with the normalised row in bf16, in 8 bits with scales, or both:
 *   h  = bf16(x + residual)                    (h = x without a residual)
 *   v  = h * weight / sqrt(mean(h^2) + eps)    (64 bits)
 *   y  = bf16(v)
 *   s  = max(fp32(max|v| / 448), 2^-126)       (over the row, or a group of it)
 *   y8 = e4m3(v / s)                           (nearest, ties to even)
 * The row that is normalised is the rounded h, the one the next layer reads.
 * y feeds lora_shrink's x; y8 with its scales feeds a base product in 8 bits.
 * A NaN in h makes the whole row's v NaN; an infinity makes its own v NaN and
 * the others zero.  A scale over a NaN is NaN, and so is all of y8 under it.
 *
 *   x, residual  bf16 [num_tokens][ldx], [ldr]; residual may be NULL.
 *   weight       bf16 [hidden].
 *   eps          >= 0, finite.
 *   hidden       multiple of 8, 8 <= hidden <= 65536; above 32768, num_tokens is
 *                less than 2^22 (LORA_ERR_UNSUPPORTED otherwise).
 *   residual_out bf16 [num_tokens][ldo]: h; may be NULL; needs a residual.  May be
 *                x or residual itself (same address and stride).
 *   y            bf16 [num_tokens][ldy]; may be NULL; may be x itself.
 *   y8           e4m3 [num_tokens][ldy8]; may be NULL, scales is NULL then too.
 *   scales       fp32 [num_tokens][hidden / group], contiguous.
 *   group        elements that share a scale: hidden, or 32, 64, 128 or 256
 *                where that divides hidden (LORA_ERR_UNSUPPORTED otherwise).
 * One of residual_out, y and y8 at least is given.  bf16 buffers are 16-byte
 * aligned with row strides that are multiples of 8 elements and at least hidden;
 * y8 is 8-byte aligned, its stride a multiple of 8.
 */
lora_status_t lora_rms_norm(const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr,
                            const uint16_t *weight, double eps, int32_t num_tokens, int32_t hidden,
                            uint16_t *residual_out, int64_t ldo, uint16_t *y, int64_t ldy,
                            uint8_t *y8, int64_t ldy8, float *scales, int32_t group,
                            hipStream_t stream);

/*
 * lora_kv_append - turn a projection's q and k by their positions, write q in
 * bf16 and k and v into the 4-bit cache.
 *   a', b' = a cos - b sin, b cos + a sin      (64 bits, rounded to fp32)
 * for the pairs (a, b) of the first rot_dim elements of a head; the others and
 * v are kept.  A block of 32 elements of k' or v takes the smallest e in
 * [-125, 125] with max| | <= 7 * 2^e (125 if there is none) and holds the
 * nearest code of element / 2^e, ties to even, at most 6 in magnitude; the
 * scale byte is e + 127.  A block with an infinity or a NaN gets scale byte 255.
 *
 *   qkv          bf16 [num_tokens][ldqkv]: q_heads, kv_heads, kv_heads heads of
 *                head_dim (the y of lora_expand over the slices q, k, v).
 *   positions    int32 [num_tokens], rows of rope.  A token whose position is
 *                outside [0, rope_rows) is padding: nothing is written for it.
 *   slots        int64 [num_tokens], places in the cache.  A token whose place
 *                is outside [0, num_pages * page_size) gets q only.  No two
 *                tokens of one call share a place.
 *   rope         fp32 [rope_rows][rot_dim]: the cosines of the rot_dim / 2 angles,
 *                then their sines.
 *   rot_dim      multiple of 16, 0 <= rot_dim <= head_dim.  With 0, positions and
 *                rope are not read and may be NULL.
 *   interleaved  0: pairs (i, i + rot_dim / 2); 1: pairs (2i, 2i + 1).
 *   q_heads      1..1024; kv_heads 1..1024; head_dim 64 or 128
 *                (LORA_ERR_UNSUPPORTED otherwise).
 *   q_out        bf16 [num_tokens][ldq]; must not overlap qkv.
 *   cache        see above; page_size 16, 32, 64, 128 or 256
 *                (LORA_ERR_UNSUPPORTED otherwise).
 * qkv, rope, q_out and cache are 16-byte aligned, ldqkv and ldq multiples of 8.
 */
lora_status_t lora_kv_append(const uint16_t *qkv, int64_t ldqkv, const int32_t *positions,
                             const int64_t *slots, const float *rope, int32_t rope_rows,
                             int32_t rot_dim, int32_t interleaved, int32_t num_tokens,
                             int32_t q_heads, int32_t kv_heads, int32_t head_dim, uint16_t *q_out,
                             int64_t ldq, uint8_t *cache, int32_t num_pages, int32_t page_size,
                             hipStream_t stream);

/*
 * lora_kv_read - what the cache holds at given places, as bf16 (exact).
 *
 *   slots         int64 [num_tokens]; a place outside the cache reads as zeros.
 *                 Places may repeat.
 *   k_out, v_out  bf16 [num_tokens][ldk], [ldv]: kv_heads heads of head_dim; one
 *                 of them may be NULL.  16-byte aligned, strides multiples of 8.
 * Other arguments as in lora_kv_append.
 */
lora_status_t lora_kv_read(const int64_t *slots, int32_t num_tokens, int32_t kv_heads,
                           int32_t head_dim, const uint8_t *cache, int32_t num_pages,
                           int32_t page_size, uint16_t *k_out, int64_t ldk, uint16_t *v_out,
                           int64_t ldv, hipStream_t stream);

/*
 * lora_kv_attention - attention of each sequence's queries over its cached keys
 * and values, from one query a sequence to pieces of prompts:
 *   out = sum_t p_t v_t,  p = softmax over t of (scale * q . k_t),
 * over the t that query i of a sequence with `length` cached tokens and
 * `queries` queries sees: t <= place = length - queries + i, t < length, and
 * t > place - window where a window is given.  (The queries are the sequence's
 * last tokens, already appended.)  A query that sees nothing gets zeros.
 * Query head h reads key head h / (q_heads / kv_heads).
 * Scores, their maxima and all sums are fp32; the weights exp(score - maximum) are
 * rounded to bf16 and divided by the sum of the rounded ones, so that a result is
 * off by about 2^-8 of the mean of |v_t - out| at most besides its own rounding.  Scores
 * have to stay inside fp32's range: a row that has some above it is NaN, and one
 * whose scores are all below it counts as one that sees nothing.
 *
 *   q            bf16 [num_tokens][ldq]: q_heads heads of head_dim.
 *   query_start  int32 [num_seqs + 1]: sequence s has the rows [query_start[s],
 *                query_start[s + 1]) of q, at most max_query_len of them.  Rows
 *                from num_tokens on and past max_query_len are ignored, and so
 *                is a sequence that starts below 0; out rows of no sequence are
 *                not written.
 *   seq_lens     int32 [num_seqs]: cached tokens; taken as at most max_seq_len.
 *   page_table   int32 [num_seqs][ld_table]: entry i of a sequence is the page of
 *                its tokens [i * page_size, (i + 1) * page_size); entries past
 *                its length may be anything.  The tokens of a page outside
 *                [0, num_pages) are skipped.
 *   max_seq_len  1 <= max_seq_len <= ld_table * page_size.
 *   num_seqs     0 <= num_seqs <= 65535.
 *   q_heads      multiple of kv_heads, at most 1024.  max_query_len * (q_heads /
 *                kv_heads) <= 2^22 (LORA_ERR_UNSUPPORTED otherwise).
 *   scale        finite.
 *   window       0 (none) or the number of keys, the query's own among them,
 *                that a query may see.
 *   out          bf16 [num_tokens][ldo].
 *   workspace    device memory of at least lora_kv_attention_workspace_bytes(...)
 *                bytes, 256-byte aligned; every call writes what it reads of it.
 *                Calls that overlap in time must not share it.  May be NULL if
 *                the size is 0.
 * Enqueues one kernel, or two where a workspace is needed (the second joins the
 * parts that long sequences are cut into).
 * q and out are 16-byte aligned, ldq and ldo multiples of 8 and at least
 * q_heads * head_dim.  The same call on the same data gives the same bits.
 */
int64_t lora_kv_attention_workspace_bytes(int32_t num_seqs, int32_t max_query_len,
                                          int32_t max_seq_len, int32_t q_heads, int32_t kv_heads,
                                          int32_t head_dim);

lora_status_t lora_kv_attention(const uint16_t *q, int64_t ldq, const int32_t *query_start,
                                const int32_t *seq_lens, const int32_t *page_table,
                                int64_t ld_table, const uint8_t *cache, int32_t num_pages,
                                int32_t page_size, int32_t num_tokens, int32_t num_seqs,
                                int32_t max_query_len, int32_t max_seq_len, int32_t q_heads,
                                int32_t kv_heads, int32_t head_dim, float scale, int32_t window,
                                uint16_t *out, int64_t ldo, void *workspace,
                                int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_ATTENTION_H */
