// Host-side checks that the entry points over the paged cache share, and the launch of
// attention, which two of them make.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "lora_attention.h"

namespace lora {

hipError_t launch_kv_attention(const uint16_t* q, int64_t ldq, const int32_t* query_start,
                               const int32_t* seq_lens, const int32_t* page_table,
                               int64_t ld_table, const uint8_t* cache, int num_pages,
                               int page_shift, int num_tokens, int num_seqs, int max_query_len,
                               int max_seq_len, int q_heads, int kv_heads, int head_dim,
                               float scale, int window, const int64_t* masks, int64_t words,
                               bool sums, uint16_t* out, int64_t ldo, float* lse, int64_t ldl,
                               void* workspace, hipStream_t stream);

constexpr int32_t kMaxTokens = 1 << 22;  // times up to 512 threads: a grid dimension
constexpr int32_t kMaxHeads = 1024;
constexpr int32_t kMaxSeqs = 65535;     // a grid dimension
constexpr int64_t kMaxRows = 1 << 22;   // queries times heads a key head, of one sequence
constexpr int32_t kMaxSeqLen = 1 << 30;

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// A bf16 matrix of rows of `width` elements.
inline bool rows_ok(const void* p, int64_t ld, int64_t width) {
  return p && aligned(p, 16) && ld >= width && ld % 8 == 0;
}

// log2 of a page size, or -1 where the library does not have it.
inline int32_t page_shift(int32_t page_size) {
  for (int32_t s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

// used: the call reads or writes the cache; its address is not looked at otherwise.
inline lora_status_t cache_ok(bool used, const uint8_t* cache, int32_t num_pages, int32_t page_size,
                              int32_t kv_heads, int32_t head_dim) {
  if (num_pages < 0 || page_size < 1 || kv_heads < 1 || kv_heads > kMaxHeads || head_dim < 1)
    return LORA_ERR_INVALID_ARGUMENT;
  if (used && (!cache || !aligned(cache, 16) || num_pages < 1)) return LORA_ERR_INVALID_ARGUMENT;
  if (page_shift(page_size) < 0 || (head_dim != 64 && head_dim != 128)) return LORA_ERR_UNSUPPORTED;
  return LORA_OK;
}

inline lora_status_t launch_status(hipError_t e) { return e == hipSuccess ? LORA_OK : LORA_ERR_LAUNCH; }

inline bool attention_sizes_ok(int32_t num_seqs, int32_t max_query_len, int32_t max_seq_len,
                               int32_t q_heads, int32_t kv_heads) {
  return num_seqs >= 0 && num_seqs <= kMaxSeqs && max_query_len >= 1 &&
         max_query_len <= kMaxTokens && max_seq_len >= 1 && max_seq_len <= kMaxSeqLen &&
         kv_heads >= 1 && q_heads >= kv_heads && q_heads <= kMaxHeads && q_heads % kv_heads == 0;
}

}  // namespace lora
