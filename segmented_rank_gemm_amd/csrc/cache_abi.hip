// C ABI of drafted tokens and caches of bounded length (lora_cache.h): host-side
// argument checks, then the launch on the caller's stream.  No call allocates,
// synchronises or keeps state.

#include "cache_checks.hpp"
#include "lora_cache.h"

namespace lora {
hipError_t launch_draft_masks(const int32_t* parents, const int32_t* query_start, int num_tokens,
                              int num_seqs, int64_t* masks, int words, const int32_t* first_positions,
                              int32_t* positions, hipStream_t stream);
int64_t kv_tree_attention_workspace_bytes(int num_seqs, int max_query_len, int max_seq_len, int q_heads,
                                          int kv_heads, int head_dim);
hipError_t launch_kv_attention_mass(const uint16_t* q, int64_t ldq, const float* lse, int64_t ldl,
                                    const int32_t* query_start, const int32_t* seq_lens,
                                    const int32_t* page_table, int64_t ld_table, const uint8_t* cache,
                                    int num_pages, int page_shift, int num_tokens, int num_seqs,
                                    int max_query_len, int max_seq_len, int q_heads, int kv_heads,
                                    int head_dim, float scale, int window, const int64_t* masks,
                                    int64_t words, float* mass, hipStream_t stream);
hipError_t launch_kv_select(const float* mass, int num_pages, int page_shift, const int32_t* seq_lens,
                            const int32_t* page_table, int64_t ld_table, int num_seqs, int kv_heads,
                            int max_seq_len, int sinks, int recent, int32_t* kept, int budget,
                            int32_t* new_lens, void* workspace, hipStream_t stream);
int64_t kv_select_workspace_bytes(int num_seqs, int kv_heads, int max_seq_len);
hipError_t launch_kv_compact(const int32_t* kept, int lists, int max_kept, const int32_t* counts,
                             const int32_t* first, const int32_t* page_table, int64_t ld_table, int pages,
                             const int32_t* dst_table, int64_t ld_dst, int dst_pages, uint8_t* cache,
                             int num_pages, int page_shift, int num_seqs, int kv_heads, int head_dim,
                             float* mass, hipStream_t stream);
}  // namespace lora

using namespace lora;

namespace {

constexpr int32_t kMaxBudget = 1 << 30;

// The arguments that tree attention and the mass share, the cache's own checks among
// them; *used: there is something to do, so that the tensors were looked at.
lora_status_t step_ok(const void* q, int64_t ldq, const void* lse, int64_t ldl, const int32_t* query_start,
                      const int32_t* seq_lens, const int32_t* page_table, int64_t ld_table,
                      const uint8_t* cache, int32_t num_pages, int32_t page_size, int32_t num_tokens,
                      int32_t num_seqs, int32_t max_query_len, int32_t max_seq_len, int32_t q_heads,
                      int32_t kv_heads, int32_t head_dim, float scale, int32_t window, const int64_t* masks,
                      int32_t mask_words, bool* used) {
  if (num_tokens < 0 || num_tokens > kMaxTokens ||
      !attention_sizes_ok(num_seqs, max_query_len, max_seq_len, q_heads, kv_heads) ||
      !isfinite(scale) || window < 0)
    return LORA_ERR_INVALID_ARGUMENT;
  *used = num_tokens > 0 && num_seqs > 0;
  const lora_status_t st = cache_ok(*used, cache, num_pages, page_size, kv_heads, head_dim);
  if (st == LORA_ERR_INVALID_ARGUMENT) return st;
  if (masks && (mask_words < 1 || !aligned(masks, 8))) return LORA_ERR_INVALID_ARGUMENT;
  if (masks && mask_words <= LORA_MAX_MASK_WORDS && max_query_len > 64 * mask_words)
    return LORA_ERR_INVALID_ARGUMENT;
  if (*used) {
    if (!query_start || !seq_lens || !page_table ||
        ld_table < (static_cast<int64_t>(max_seq_len) + page_size - 1) / page_size)
      return LORA_ERR_INVALID_ARGUMENT;
    if (!rows_ok(q, ldq, static_cast<int64_t>(q_heads) * head_dim)) return LORA_ERR_INVALID_ARGUMENT;
    if (lse && (!aligned(lse, 4) || ldl < q_heads)) return LORA_ERR_INVALID_ARGUMENT;
  }
  if (st != LORA_OK) return st;
  if (masks && mask_words > LORA_MAX_MASK_WORDS) return LORA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(max_query_len) * (q_heads / kv_heads) > kMaxRows) return LORA_ERR_UNSUPPORTED;
  return LORA_OK;
}

// Arrays of n numbers that have some in common.
bool share_elements(const int32_t* a, const int32_t* b, int64_t n) {
  const auto x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return (x < y ? y - x : x - y) < static_cast<uintptr_t>(n) * sizeof(int32_t);
}

}  // namespace

extern "C" {

lora_status_t lora_draft_masks(const int32_t* parents, const int32_t* query_start, int32_t num_tokens,
                               int32_t num_seqs, int64_t* masks, int32_t mask_words, const int32_t* first,
                               int32_t* positions, hipStream_t stream) {
  if (num_tokens < 0 || num_tokens > kMaxTokens || num_seqs < 0 || num_seqs > kMaxSeqs || mask_words < 1)
    return LORA_ERR_INVALID_ARGUMENT;
  const bool used = num_tokens > 0 && num_seqs > 0;
  if (used && (!parents || !query_start || (!masks && !positions) || !aligned(masks, 8)))
    return LORA_ERR_INVALID_ARGUMENT;
  if (mask_words > LORA_MAX_MASK_WORDS) return LORA_ERR_UNSUPPORTED;
  if (!used) return LORA_OK;
  return launch_status(lora::launch_draft_masks(parents, query_start, num_tokens, num_seqs, masks, mask_words,
                                                first, positions, stream));
}

int64_t lora_kv_tree_attention_workspace_bytes(int32_t num_seqs, int32_t max_query_len, int32_t max_seq_len,
                                               int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
  if (!attention_sizes_ok(num_seqs, max_query_len, max_seq_len, q_heads, kv_heads) ||
      (head_dim != 64 && head_dim != 128) ||
      static_cast<int64_t>(max_query_len) * (q_heads / kv_heads) > kMaxRows)
    return 0;
  return lora::kv_tree_attention_workspace_bytes(num_seqs, max_query_len, max_seq_len, q_heads, kv_heads,
                                                 head_dim);
}

lora_status_t lora_kv_tree_attention(const uint16_t* q, int64_t ldq, const int32_t* query_start,
                                     const int32_t* seq_lens, const int32_t* page_table, int64_t ld_table,
                                     const uint8_t* cache, int32_t num_pages, int32_t page_size,
                                     int32_t num_tokens, int32_t num_seqs, int32_t max_query_len,
                                     int32_t max_seq_len, int32_t q_heads, int32_t kv_heads,
                                     int32_t head_dim, float scale, int32_t window, const int64_t* masks,
                                     int32_t mask_words, uint16_t* out, int64_t ldo, float* lse,
                                     int64_t ldl, void* workspace, int64_t workspace_bytes,
                                     hipStream_t stream) {
  bool used = false;
  const lora_status_t st = step_ok(q, ldq, lse, ldl, query_start, seq_lens, page_table, ld_table, cache,
                                   num_pages, page_size, num_tokens, num_seqs, max_query_len, max_seq_len,
                                   q_heads, kv_heads, head_dim, scale, window, masks, mask_words, &used);
  if (st == LORA_ERR_INVALID_ARGUMENT) return st;
  if (used && !rows_ok(out, ldo, static_cast<int64_t>(q_heads) * head_dim)) return LORA_ERR_INVALID_ARGUMENT;
  if (st != LORA_OK || !used) return st;
  const int64_t need = lora_kv_tree_attention_workspace_bytes(num_seqs, max_query_len, max_seq_len, q_heads,
                                                              kv_heads, head_dim);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
    return LORA_ERR_INVALID_ARGUMENT;
  return launch_status(lora::launch_kv_attention(
      q, ldq, query_start, seq_lens, page_table, ld_table, cache, num_pages, page_shift(page_size),
      num_tokens, num_seqs, max_query_len, max_seq_len, q_heads, kv_heads, head_dim, scale, window, masks,
      mask_words, true, out, ldo, lse, ldl, workspace, stream));
}

lora_status_t lora_kv_attention_mass(const uint16_t* q, int64_t ldq, const float* lse, int64_t ldl,
                                     const int32_t* query_start, const int32_t* seq_lens,
                                     const int32_t* page_table, int64_t ld_table, const uint8_t* cache,
                                     int32_t num_pages, int32_t page_size, int32_t num_tokens,
                                     int32_t num_seqs, int32_t max_query_len, int32_t max_seq_len,
                                     int32_t q_heads, int32_t kv_heads, int32_t head_dim, float scale,
                                     int32_t window, const int64_t* masks, int32_t mask_words, float* mass,
                                     hipStream_t stream) {
  bool used = false;
  const lora_status_t st = step_ok(q, ldq, lse, ldl, query_start, seq_lens, page_table, ld_table, cache,
                                   num_pages, page_size, num_tokens, num_seqs, max_query_len, max_seq_len,
                                   q_heads, kv_heads, head_dim, scale, window, masks, mask_words, &used);
  if (st == LORA_ERR_INVALID_ARGUMENT) return st;
  if (used && (!lse || !mass || !aligned(mass, 16))) return LORA_ERR_INVALID_ARGUMENT;
  if (st != LORA_OK || !used) return st;
  return launch_status(lora::launch_kv_attention_mass(
      q, ldq, lse, ldl, query_start, seq_lens, page_table, ld_table, cache, num_pages, page_shift(page_size),
      num_tokens, num_seqs, max_query_len, max_seq_len, q_heads, kv_heads, head_dim, scale, window, masks,
      mask_words, mass, stream));
}

int64_t lora_kv_select_workspace_bytes(int32_t num_seqs, int32_t kv_heads, int32_t max_seq_len) {
  if (num_seqs < 0 || num_seqs > kMaxSeqs || kv_heads < 1 || kv_heads > kMaxHeads || max_seq_len < 1 ||
      max_seq_len > kMaxSeqLen)
    return 0;
  return lora::kv_select_workspace_bytes(num_seqs, kv_heads, max_seq_len);
}

lora_status_t lora_kv_select(const float* mass, int32_t num_pages, int32_t page_size, const int32_t* seq_lens,
                             const int32_t* page_table, int64_t ld_table, int32_t num_seqs, int32_t kv_heads,
                             int32_t max_seq_len, int32_t sinks, int32_t recent, int32_t* kept,
                             int32_t budget, int32_t* new_lens, void* workspace, int64_t workspace_bytes,
                             hipStream_t stream) {
  if (num_seqs < 0 || num_seqs > kMaxSeqs || kv_heads < 1 || kv_heads > kMaxHeads || max_seq_len < 1 ||
      max_seq_len > kMaxSeqLen || sinks < 0 || recent < 0 || budget < 1 || budget > kMaxBudget ||
      static_cast<int64_t>(sinks) + recent > budget || num_pages < 0 || page_size < 1)
    return LORA_ERR_INVALID_ARGUMENT;
  if (num_seqs > 0 && (!mass || !aligned(mass, 16) || num_pages < 1 || !seq_lens || !page_table || !kept ||
                       !new_lens || share_elements(new_lens, seq_lens, num_seqs) ||
                       ld_table < (static_cast<int64_t>(max_seq_len) + page_size - 1) / page_size))
    return LORA_ERR_INVALID_ARGUMENT;
  if (page_shift(page_size) < 0) return LORA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return LORA_OK;
  const int64_t need = lora_kv_select_workspace_bytes(num_seqs, kv_heads, max_seq_len);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
    return LORA_ERR_INVALID_ARGUMENT;
  return launch_status(lora::launch_kv_select(mass, num_pages, page_shift(page_size), seq_lens, page_table,
                                              ld_table, num_seqs, kv_heads, max_seq_len, sinks, recent, kept,
                                              budget, new_lens, workspace, stream));
}

lora_status_t lora_kv_compact(const int32_t* kept, int32_t num_lists, int32_t max_kept, const int32_t* counts,
                              const int32_t* first, const int32_t* page_table, int64_t ld_table,
                              int32_t table_pages, const int32_t* dst_table, int64_t ld_dst,
                              int32_t dst_pages, uint8_t* cache, int32_t num_pages, int32_t page_size,
                              int32_t num_seqs, int32_t kv_heads, int32_t head_dim, float* mass,
                              hipStream_t stream) {
  if (num_seqs < 0 || num_seqs > kMaxSeqs || max_kept < 0 || max_kept > kMaxBudget)
    return LORA_ERR_INVALID_ARGUMENT;
  const bool used = num_seqs > 0 && max_kept > 0;
  const lora_status_t st = cache_ok(used, cache, num_pages, page_size, kv_heads, head_dim);
  if (st == LORA_ERR_INVALID_ARGUMENT) return st;
  if (num_lists != 1 && num_lists != kv_heads) return LORA_ERR_INVALID_ARGUMENT;
  if (used && (!kept || !counts || !page_table || table_pages < 1 || ld_table < table_pages ||
               (dst_table && (dst_pages < 1 || ld_dst < dst_pages)) || !aligned(mass, 16)))
    return LORA_ERR_INVALID_ARGUMENT;
  if (st != LORA_OK) return st;
  if (!used) return LORA_OK;
  // in place by the other table: the list would be shared out over places that it still reads
  if (dst_table == page_table) return LORA_ERR_INVALID_ARGUMENT;
  return launch_status(lora::launch_kv_compact(kept, num_lists, max_kept, counts, first, page_table, ld_table,
                                               table_pages, dst_table, ld_dst, dst_pages, cache, num_pages,
                                               page_shift(page_size), num_seqs, kv_heads, head_dim, mass,
                                               stream));
}

}  // extern "C"
