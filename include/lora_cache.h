/*
 * lora_cache.h - C ABI of drafted tokens and of caches of bounded length: trees of
 * drafted tokens and attention for them over the 4-bit paged cache, the weight that
 * each cached token draws, the choice of the tokens that a cache keeps, and their
 * move to the places in front.  They live in the same library as the operators of
 * lora_attention.h, keep its conventions and share its cache.
 *
 * A step with drafts: lora_draft_masks, lora_kv_append at its positions, attention by
 * lora_kv_tree_attention, and once the accepted ones are known lora_kv_compact, which
 * moves them to the places right behind the text.  From there on the sequence's length is
 * that of the text and the accepted drafts: seq_lens still counts all drafts until the
 * caller has set it.
 * A cache of bounded length: lora_kv_tree_attention with sums (and no masks, where
 * there are no drafts), lora_kv_attention_mass after it; when a sequence has grown
 * past its bound, lora_kv_select and lora_kv_compact.  With drafts, the mass is drawn
 * between the choice of the accepted ones and their move, with lse set to -infinity in
 * the rows of the others: these would count in the text's mass for good.
 *
 * The mass: fp32 [num_pages][kv_heads][page_size] beside the cache, 16-byte aligned;
 * an element is the attention that the token of its place has drawn from the rows of
 * its key head.
 */
#ifndef LORA_CACHE_H
#define LORA_CACHE_H

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "lora_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_MAX_MASK_WORDS 8 /* words of 64 bits of a drafted token's mask */

/*
 * lora_draft_masks - which drafted tokens of its sequence each one sees, and its
 * position, from the trees' parents:
 *   mask_i = bit i, and the mask of i's parent   (bit j of word w is draft 64 w + j)
 *   position_i = first + depth of i              (a root's depth is 0)
 * for the drafted tokens [query_start[s], query_start[s + 1]) of each sequence s,
 * counted from 0.
 *
 *   parents      int32 [num_tokens]: the parent's number in the sequence, or -1 for a
 *                root.  A token whose parent does not lie before it is a root.
 *   query_start  int32 [num_seqs + 1].  Rows from num_tokens on are ignored, and so is
 *                a sequence that starts below 0, and a sequence's tokens from 64 *
 *                mask_words on; what belongs to them is not written.
 *   masks        int64 [num_tokens][mask_words], contiguous; may be NULL.
 *   mask_words   1..LORA_MAX_MASK_WORDS (LORA_ERR_UNSUPPORTED above).
 *   first        int32 [num_seqs]: the position of each sequence's roots; NULL: 0.
 *   positions    int32 [num_tokens]; may be NULL.
 * One of masks and positions at least is given.
 */
lora_status_t lora_draft_masks(const int32_t *parents, const int32_t *query_start, int32_t num_tokens,
                               int32_t num_seqs, int64_t *masks, int32_t mask_words,
                               const int32_t *first, int32_t *positions, hipStream_t stream);

/*
 * lora_kv_tree_attention - lora_kv_attention for drafted tokens, or with sums:
 *   out = sum_t p_t v_t,  p = softmax over t of (scale * q . k_t),
 *   lse = ln sum_t exp(scale * q . k_t)
 * over the t that query i of a sequence with `length` cached tokens and `queries`
 * queries, its last ones, sees.  With masks those are, in this order, the tokens
 * t < length - queries and the drafts t = length - queries + j >= 0 whose bit j is set
 * in row i of masks (bits from `queries` on do not count; a token does not see itself
 * unless its own bit is set); with a window, the last `window` of those.  Without masks
 * they are lora_kv_attention's.  (Queries past max_query_len have no rows here, but are
 * drafts that others may see.)  A query that sees nothing gets zeros and -infinity.
 * out is computed as by lora_kv_attention; lse from the unrounded weights, in fp32.
 *
 *   masks        int64 [num_tokens][mask_words], contiguous; may be NULL.
 *   mask_words   1..LORA_MAX_MASK_WORDS (LORA_ERR_UNSUPPORTED above), and with masks
 *                max_query_len <= 64 * mask_words; not looked at without.
 *   lse          fp32 [num_tokens][ldl], 4-byte aligned, ldl >= q_heads; may be NULL.
 *                Rows of no sequence are not written.
 *   workspace    of lora_kv_tree_attention_workspace_bytes(...), as for
 *                lora_kv_attention.
 * Other arguments, and what is enqueued, as for lora_kv_attention.  The same call on
 * the same data gives the same bits.
 */
int64_t lora_kv_tree_attention_workspace_bytes(int32_t num_seqs, int32_t max_query_len,
                                               int32_t max_seq_len, int32_t q_heads,
                                               int32_t kv_heads, int32_t head_dim);

lora_status_t lora_kv_tree_attention(const uint16_t *q, int64_t ldq, const int32_t *query_start,
                                     const int32_t *seq_lens, const int32_t *page_table,
                                     int64_t ld_table, const uint8_t *cache, int32_t num_pages,
                                     int32_t page_size, int32_t num_tokens, int32_t num_seqs,
                                     int32_t max_query_len, int32_t max_seq_len, int32_t q_heads,
                                     int32_t kv_heads, int32_t head_dim, float scale,
                                     int32_t window, const int64_t *masks, int32_t mask_words,
                                     uint16_t *out, int64_t ldo, float *lse, int64_t ldl,
                                     void *workspace, int64_t workspace_bytes,
                                     hipStream_t stream);

/*
 * lora_kv_attention_mass - the attention that each cached token draws in a step:
 *   drawn[t] = sum over the rows (query, head) of its key head that see t of
 *              exp(scale * q . k_t - lse)
 *   mass[t]  = mass[t] + drawn[t]   for a sequence's tokens t < length - queries,
 *   mass[t]  = drawn[t]             for its last `queries`, this step's own, whatever
 *                                   their places held.
 * What a row sees is as for lora_kv_tree_attention on the same arguments; lse is what
 * that call wrote, or -infinity: such a row counts for nothing, whatever its q and the
 * keys that it sees hold.  Where it is NaN, as where a key that the row sees holds one,
 * so is the mass of what the row sees.  Scores and sums are fp32.
 * Sequences without rows in this call, places past a sequence's length and tokens of
 * pages outside [0, num_pages) are left as they are.  No page may stand twice among
 * those that hold the tokens of this call's sequences.
 * Enqueues one kernel.  The same call on the same data gives the same bits.
 */
lora_status_t lora_kv_attention_mass(const uint16_t *q, int64_t ldq, const float *lse, int64_t ldl,
                                     const int32_t *query_start, const int32_t *seq_lens,
                                     const int32_t *page_table, int64_t ld_table,
                                     const uint8_t *cache, int32_t num_pages, int32_t page_size,
                                     int32_t num_tokens, int32_t num_seqs, int32_t max_query_len,
                                     int32_t max_seq_len, int32_t q_heads, int32_t kv_heads,
                                     int32_t head_dim, float scale, int32_t window,
                                     const int64_t *masks, int32_t mask_words, float *mass,
                                     hipStream_t stream);

/*
 * lora_kv_select - the tokens that each key head of a sequence keeps: all of them if
 * there are at most `budget`; else the first `sinks`, the last `recent`, and the
 * heaviest of those between, of equal ones the first, `budget` in all.  A NaN weighs
 * -infinity, and so does a token of a page outside [0, num_pages).
 *
 *   seq_lens     int32 [num_seqs]: cached tokens; taken as at most max_seq_len.
 *   page_table   int32 [num_seqs][ld_table], as for lora_kv_attention.
 *   sinks, recent  >= 0, sinks + recent <= budget.
 *   budget       1..2^30.
 *   kept         int32 [num_seqs][kv_heads][budget], contiguous: the tokens' numbers,
 *                ascending; -1 past the last.
 *   new_lens     int32 [num_seqs]: how many each key head keeps; no part of it is seq_lens'.
 *   workspace    of lora_kv_select_workspace_bytes(...), 256-byte aligned, free for
 *                reuse when the call's kernels have finished; may be NULL where that is 0.
 * Enqueues one kernel, or four for long sequences.
 */
int64_t lora_kv_select_workspace_bytes(int32_t num_seqs, int32_t kv_heads, int32_t max_seq_len);

lora_status_t lora_kv_select(const float *mass, int32_t num_pages, int32_t page_size,
                             const int32_t *seq_lens, const int32_t *page_table, int64_t ld_table,
                             int32_t num_seqs, int32_t kv_heads, int32_t max_seq_len,
                             int32_t sinks, int32_t recent, int32_t *kept, int32_t budget,
                             int32_t *new_lens, void *workspace, int64_t workspace_bytes,
                             hipStream_t stream);

/*
 * lora_kv_compact - moves cached tokens (keys, values, and their mass) to the places
 * in front:
 *   place first + j  <-  what place first + kept[j] held before the call
 * for j < count of each sequence and key head, in place or into other pages.
 *
 *   kept         int32 [num_seqs][num_lists][max_kept], contiguous; num_lists is
 *                kv_heads, or 1: one list for all key heads.
 *   counts       int32 [num_seqs]; taken as at most max_kept.
 *   first        int32 [num_seqs], or NULL: 0.
 *   page_table   int32 [num_seqs][ld_table], of which table_pages entries a sequence
 *                may be read (those of the places named above are).
 *   dst_table    int32 [num_seqs][ld_dst], dst_pages entries a sequence: the pages
 *                that take place first + j; NULL: in place, and not page_table itself.
 *                None of these may be one that the call reads from, and none may take
 *                the tokens of two places.
 *   mass         may be NULL.
 * Entries below 0, and those whose source or destination lies outside its table or on
 * a page outside [0, num_pages), are skipped: their destinations stay as they are.
 * In place the entries ascend, each above the one before, those below 0 behind all others
 * (what the places named hold afterwards is open otherwise); kept[j] = j leaves the token
 * where it is.  No page may then stand twice among those that hold the places named.
 * Enqueues one kernel, or two for long lists of few key heads in place.
 */
lora_status_t lora_kv_compact(const int32_t *kept, int32_t num_lists, int32_t max_kept,
                              const int32_t *counts, const int32_t *first,
                              const int32_t *page_table, int64_t ld_table, int32_t table_pages,
                              const int32_t *dst_table, int64_t ld_dst, int32_t dst_pages,
                              uint8_t *cache, int32_t num_pages, int32_t page_size,
                              int32_t num_seqs, int32_t kv_heads, int32_t head_dim, float *mass,
                              hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_CACHE_H */
