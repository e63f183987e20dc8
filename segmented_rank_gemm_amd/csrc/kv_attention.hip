// lora_kv_attention: softmax(scale q K^T) V of each sequence's queries over its
// cached keys and values, read from the 4-bit paged cache.
//
// One wave a (query, query head): lane j scores key base + j, the running
// maximum and sum of the softmax are kept in fp32, and the lanes then share out
// the head's elements to add the 64 weighted values up.

#include "kv_format.hpp"

namespace lora {

struct AttentionArgs {
  const uint16_t* q;
  const int32_t* query_start;
  const int32_t* seq_lens;
  const int32_t* page_table;
  uint16_t* out;
  Cache<const uint8_t> cache;
  int64_t ldq, ldo, ld_table;
  int num_tokens, max_query_len, max_seq_len, q_heads, window;
  float scale_log2;  // scale * log2(e): the softmax runs in powers of two
};

__device__ __forceinline__ float code_value(uint32_t c) {
  const uint32_t m = c & 7u;
  const float u = m < 4 ? 0.5f * m : (m < 6 ? m - 2.f : 2.f * m - 8.f);
  return c & 8u ? -u : u;
}

template <int D>
__global__ __launch_bounds__(kWave) void kv_attention_kernel(AttentionArgs a) {
  const int seq = static_cast<int>(blockIdx.z);
  const int head = static_cast<int>(blockIdx.y);
  const int i = static_cast<int>(blockIdx.x);
  const int start = a.query_start[seq], end = a.query_start[seq + 1];
  if (start < 0 || start >= a.num_tokens - i || end <= start) return;
  const int queries = end - start;
  if (i >= queries) return;
  int length = a.seq_lens[seq];
  length = length < 0 ? 0 : (length > a.max_seq_len ? a.max_seq_len : length);
  const int kv_head = head / (a.q_heads / a.cache.kv_heads);
  const int place = length - queries + i;
  const int last = place + 1 < length ? place + 1 : length;
  int first = a.window ? place - a.window + 1 : 0;
  first = first < 0 ? 0 : first;

  __shared__ float qs[D], ps[kWave];
  __shared__ int pages[kWave];
  const int lane = lane_id();
  const int64_t row = start + i;
  for (int e = lane; e < D; e += kWave)
    qs[e] = __uint_as_float(static_cast<uint32_t>(a.q[row * a.ldq + head * D + e]) << 16);
  __syncthreads();
  const int psize = a.cache.page_size();
  float top = -INFINITY, total = 0.f;
  float acc[D / kWave] = {};
  for (int base = first; base < last; base += kWave) {
    const int t = base + lane;
    int page = -1;
    float s = -INFINITY;
    if (t < last) {
      page = a.page_table[seq * a.ld_table + (t >> a.cache.page_shift)];
      if (page < 0 || page >= a.cache.num_pages) page = -1;
      if (page >= 0) {
        const uint8_t* block = a.cache.template block<D>(page, 0, kv_head);
        const int at = t & (psize - 1);
        float dot = 0.f;
        for (int b = 0; b < D / kBlock; ++b) {
          const uint32_t sb = block[a.cache.template scales_at<D>() + (b << a.cache.page_shift) + at];
          const u32x4 w = load16(block + at * (D / 2) + b * 16);
          float part = 0.f;
          for (int k = 0; k < 32; ++k)
            part += code_value((w[k >> 3] >> (4 * (k & 7))) & 15u) * qs[b * 32 + k];
          dot += part * (sb == kScaleNan ? NAN : scale_value(sb));
        }
        s = dot * a.scale_log2;
      }
    }
    pages[lane] = page;
    float m = s;
    for (int x = 1; x < kWave; x <<= 1) m = fmaxf(m, __shfl_xor(m, x));
    const float now = fmaxf(top, m);
    // a NaN score stays NaN; a run of skipped tokens leaves `now` at -infinity
    const float p = s == -INFINITY ? 0.f : exp2f(s - now);
    const float shrink = top == -INFINITY ? 0.f : exp2f(top - now);
    float sum = p;
    for (int x = 1; x < kWave; x <<= 1) sum += __shfl_xor(sum, x);
    total = total * shrink + sum;
    top = now;
    ps[lane] = p;
    __syncthreads();
    for (int j = 0; j < D / kWave; ++j) acc[j] *= shrink;
    const int n = last - base < kWave ? last - base : kWave;
    for (int k = 0; k < n; ++k) {
      const int pg = pages[k];
      if (pg < 0) continue;
      const uint8_t* block = a.cache.template block<D>(pg, 1, kv_head);
      const int at = (base + k) & (psize - 1);
      for (int j = 0; j < D / kWave; ++j) {
        const int e = j * kWave + lane;
        const uint32_t sb =
            block[a.cache.template scales_at<D>() + ((e / kBlock) << a.cache.page_shift) + at];
        const uint32_t c = (block[at * (D / 2) + e / 2] >> (4 * (e & 1))) & 15u;
        acc[j] += ps[k] * code_value(c) * (sb == kScaleNan ? NAN : scale_value(sb));
      }
    }
    __syncthreads();
  }
  for (int j = 0; j < D / kWave; ++j) {
    const float v = total == 0.f ? 0.f : acc[j] / total;
    a.out[row * a.ldo + head * D + j * kWave + lane] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
  }
}

int64_t kv_attention_workspace_bytes(int num_seqs, int max_query_len, int max_seq_len, int q_heads,
                                     int kv_heads, int head_dim) {
  return 0;
}

hipError_t launch_kv_attention(const uint16_t* q, int64_t ldq, const int32_t* query_start,
                               const int32_t* seq_lens, const int32_t* page_table,
                               int64_t ld_table, const uint8_t* cache, int num_pages,
                               int page_shift, int num_tokens, int num_seqs, int max_query_len,
                               int max_seq_len, int q_heads, int kv_heads, int head_dim,
                               float scale, int window, uint16_t* out, int64_t ldo,
                               void* workspace, hipStream_t stream) {
  const AttentionArgs a = {q, query_start, seq_lens, page_table, out,
                           {cache, num_pages, page_shift, kv_heads},
                           ldq, ldo, ld_table, num_tokens, max_query_len, max_seq_len, q_heads,
                           window, scale * 1.44269504f};
  const dim3 grid(max_query_len, q_heads, num_seqs), block(kWave);
  if (head_dim == 64) kv_attention_kernel<64><<<grid, block, 0, stream>>>(a);
  else kv_attention_kernel<128><<<grid, block, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace lora
