// C ABI of the operators around the projections (lora_attention.h): host-side
// argument checks, then the launch on the caller's stream.  No call allocates,
// synchronises or keeps state.

#include "cache_checks.hpp"

namespace lora {
hipError_t launch_rms_norm(const uint16_t* x, int64_t ldx, const uint16_t* residual, int64_t ldr,
                           const uint16_t* weight, double eps, int num_tokens, int hidden,
                           uint16_t* sum, int64_t lds, uint16_t* y, int64_t ldy, uint8_t* y8,
                           int64_t ldy8, float* scales, int group, hipStream_t stream);
hipError_t launch_kv_append(const uint16_t* qkv, int64_t ldqkv, const int32_t* positions,
                            const int64_t* slots, const float* rope, int rope_rows, int rot_dim,
                            int interleaved, int num_tokens, int q_heads, int kv_heads,
                            int head_dim, uint16_t* q_out, int64_t ldq, uint8_t* cache,
                            int num_pages, int page_shift, hipStream_t stream);
hipError_t launch_kv_read(const int64_t* slots, int num_tokens, int kv_heads, int head_dim,
                          const uint8_t* cache, int num_pages, int page_shift, uint16_t* k_out,
                          int64_t ldk, uint16_t* v_out, int64_t ldv, hipStream_t stream);
int64_t kv_attention_workspace_bytes(int num_seqs, int max_query_len, int max_seq_len, int q_heads,
                                     int kv_heads, int head_dim);
}  // namespace lora

using namespace lora;

namespace {

constexpr int32_t kMaxHidden = 65536;
constexpr int32_t kHidden512 = 32768;    // longer rows take 1024 threads

}  // namespace

extern "C" {

lora_status_t lora_rms_norm(const uint16_t* x, int64_t ldx, const uint16_t* residual, int64_t ldr,
                            const uint16_t* weight, double eps, int32_t num_tokens, int32_t hidden,
                            uint16_t* residual_out, int64_t ldo, uint16_t* y, int64_t ldy,
                            uint8_t* y8, int64_t ldy8, float* scales, int32_t group,
                            hipStream_t stream) {
  if (num_tokens < 0 || num_tokens > kMaxTokens || hidden < 8 || hidden > kMaxHidden ||
      hidden % 8 != 0 || !(eps >= 0.0) || !isfinite(eps))
    return LORA_ERR_INVALID_ARGUMENT;
  if (num_tokens > 0) {
    if (!residual_out && !y && !y8) return LORA_ERR_INVALID_ARGUMENT;
    if ((residual_out && !residual) || !y8 != !scales) return LORA_ERR_INVALID_ARGUMENT;
    if (y8 && (group < 1 || hidden % group != 0)) return LORA_ERR_INVALID_ARGUMENT;
    if (!rows_ok(x, ldx, hidden) || !rows_ok(weight, hidden, hidden) ||
        (residual && !rows_ok(residual, ldr, hidden)) ||
        (residual_out && !rows_ok(residual_out, ldo, hidden)) || (y && !rows_ok(y, ldy, hidden)))
      return LORA_ERR_INVALID_ARGUMENT;
    if (y8 && (!aligned(y8, 8) || !aligned(scales, 4) || ldy8 < hidden || ldy8 % 8 != 0))
      return LORA_ERR_INVALID_ARGUMENT;
  }
  if (y8 && group != hidden && group != 32 && group != 64 && group != 128 && group != 256)
    return LORA_ERR_UNSUPPORTED;
  if (num_tokens == kMaxTokens && hidden > kHidden512) return LORA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return LORA_OK;
  return launch_status(lora::launch_rms_norm(x, ldx, residual, ldr, weight, eps, num_tokens, hidden,
                                             residual_out, ldo, y, ldy, y8, ldy8, scales,
                                             y8 ? group : hidden, stream));
}

lora_status_t lora_kv_append(const uint16_t* qkv, int64_t ldqkv, const int32_t* positions,
                             const int64_t* slots, const float* rope, int32_t rope_rows,
                             int32_t rot_dim, int32_t interleaved, int32_t num_tokens,
                             int32_t q_heads, int32_t kv_heads, int32_t head_dim, uint16_t* q_out,
                             int64_t ldq, uint8_t* cache, int32_t num_pages, int32_t page_size,
                             hipStream_t stream) {
  if (num_tokens < 0 || num_tokens > kMaxTokens || q_heads < 1 || q_heads > kMaxHeads)
    return LORA_ERR_INVALID_ARGUMENT;
  const lora_status_t st = cache_ok(num_tokens > 0, cache, num_pages, page_size, kv_heads, head_dim);
  if (st == LORA_ERR_INVALID_ARGUMENT) return st;
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16 != 0 || interleaved < 0 || interleaved > 1)
    return LORA_ERR_INVALID_ARGUMENT;
  const int64_t q_width = static_cast<int64_t>(q_heads) * head_dim;
  const int64_t width = q_width + 2 * static_cast<int64_t>(kv_heads) * head_dim;
  if (num_tokens > 0 && (!rows_ok(qkv, ldqkv, width) || !rows_ok(q_out, ldq, q_width) || !slots))
    return LORA_ERR_INVALID_ARGUMENT;
  if (num_tokens > 0 && rot_dim > 0 && (!positions || !rope || !aligned(rope, 16) || rope_rows < 1))
    return LORA_ERR_INVALID_ARGUMENT;
  if (st != LORA_OK) return st;
  if (num_tokens == 0) return LORA_OK;
  return launch_status(lora::launch_kv_append(qkv, ldqkv, positions, slots, rope, rope_rows, rot_dim,
                                              interleaved, num_tokens, q_heads, kv_heads, head_dim,
                                              q_out, ldq, cache, num_pages, page_shift(page_size),
                                              stream));
}

lora_status_t lora_kv_read(const int64_t* slots, int32_t num_tokens, int32_t kv_heads,
                           int32_t head_dim, const uint8_t* cache, int32_t num_pages,
                           int32_t page_size, uint16_t* k_out, int64_t ldk, uint16_t* v_out,
                           int64_t ldv, hipStream_t stream) {
  if (num_tokens < 0 || num_tokens > kMaxTokens || (num_tokens > 0 && !k_out && !v_out))
    return LORA_ERR_INVALID_ARGUMENT;
  const lora_status_t st = cache_ok(num_tokens > 0, cache, num_pages, page_size, kv_heads, head_dim);
  if (st == LORA_ERR_INVALID_ARGUMENT) return st;
  const int64_t width = static_cast<int64_t>(kv_heads) * head_dim;
  if (num_tokens > 0 && (!slots || (k_out && !rows_ok(k_out, ldk, width)) ||
                         (v_out && !rows_ok(v_out, ldv, width))))
    return LORA_ERR_INVALID_ARGUMENT;
  if (st != LORA_OK) return st;
  if (num_tokens == 0) return LORA_OK;
  return launch_status(lora::launch_kv_read(slots, num_tokens, kv_heads, head_dim, cache, num_pages,
                                            page_shift(page_size), k_out, ldk, v_out, ldv, stream));
}

int64_t lora_kv_attention_workspace_bytes(int32_t num_seqs, int32_t max_query_len,
                                          int32_t max_seq_len, int32_t q_heads, int32_t kv_heads,
                                          int32_t head_dim) {
  if (!attention_sizes_ok(num_seqs, max_query_len, max_seq_len, q_heads, kv_heads) ||
      (head_dim != 64 && head_dim != 128) ||
      static_cast<int64_t>(max_query_len) * (q_heads / kv_heads) > kMaxRows)
    return 0;
  return lora::kv_attention_workspace_bytes(num_seqs, max_query_len, max_seq_len, q_heads, kv_heads,
                                            head_dim);
}

lora_status_t lora_kv_attention(const uint16_t* q, int64_t ldq, const int32_t* query_start,
                                const int32_t* seq_lens, const int32_t* page_table,
                                int64_t ld_table, const uint8_t* cache, int32_t num_pages,
                                int32_t page_size, int32_t num_tokens, int32_t num_seqs,
                                int32_t max_query_len, int32_t max_seq_len, int32_t q_heads,
                                int32_t kv_heads, int32_t head_dim, float scale, int32_t window,
                                uint16_t* out, int64_t ldo, void* workspace,
                                int64_t workspace_bytes, hipStream_t stream) {
  if (num_tokens < 0 || num_tokens > kMaxTokens ||
      !attention_sizes_ok(num_seqs, max_query_len, max_seq_len, q_heads, kv_heads) ||
      !isfinite(scale) || window < 0)
    return LORA_ERR_INVALID_ARGUMENT;
  const bool used = num_tokens > 0 && num_seqs > 0;
  const lora_status_t st = cache_ok(used, cache, num_pages, page_size, kv_heads, head_dim);
  if (st == LORA_ERR_INVALID_ARGUMENT) return st;
  if (used &&
      (!query_start || !seq_lens || !page_table ||
       ld_table < (static_cast<int64_t>(max_seq_len) + page_size - 1) / page_size))
    return LORA_ERR_INVALID_ARGUMENT;
  const int64_t width = static_cast<int64_t>(q_heads) * head_dim;
  if (used && (!rows_ok(q, ldq, width) || !rows_ok(out, ldo, width)))
    return LORA_ERR_INVALID_ARGUMENT;
  if (st != LORA_OK) return st;
  if (static_cast<int64_t>(max_query_len) * (q_heads / kv_heads) > kMaxRows)
    return LORA_ERR_UNSUPPORTED;
  if (!used) return LORA_OK;
  const int64_t need = lora_kv_attention_workspace_bytes(num_seqs, max_query_len, max_seq_len,
                                                         q_heads, kv_heads, head_dim);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
    return LORA_ERR_INVALID_ARGUMENT;
  return launch_status(lora::launch_kv_attention(
      q, ldq, query_start, seq_lens, page_table, ld_table, cache, num_pages, page_shift(page_size),
      num_tokens, num_seqs, max_query_len, max_seq_len, q_heads, kv_heads, head_dim, scale, window,
      nullptr, 0, false, out, ldo, nullptr, 0, workspace, stream));
}

}  // extern "C"
