// lora_draft_masks: which drafted tokens of its sequence each one descends from, as
// bits, and its position, from the parents:
//   mask[i] = bit i | mask[parent[i]],  position[i] = first + depth[i]
//
// A workgroup a sequence.  The parents are staged in shared memory, and each thread
// climbs from its own token to the root, marking the bits of its row there: as many
// steps as the tree is deep.  Parents lie before their children (others are taken for
// roots), so that every climb ends.
//
// Bound by latency: two dependent loads, the climb and the stores, and where trees are
// deep by the climb, two dependent reads of shared memory a step (us, an empty launch 1.9;
// random trees / chains: 1 sequence of 26 drafts 2.2 / 3.5, of 64 2.3 / 6.0, of 512
// 5.1 / 65; 16 of 32 2.6 / 4.5.  Behind an attention over 47 MB, whose lines have taken
// the caches, 16 of 32 took 4.6 in a trace and 2.7 by themselves).

#include "kv_attention.hpp"

namespace lora {

constexpr int kMaskThreads = 256;
constexpr int kMaxDrafts = 64 * kDraftWords;

__global__ __launch_bounds__(kMaskThreads) void draft_masks_kernel(
    const int32_t* parents, const int32_t* query_start, int num_tokens, int64_t* masks, int words,
    const int32_t* first_positions, int32_t* positions) {
  const int seq = static_cast<int>(blockIdx.x), tid = static_cast<int>(threadIdx.x);
  const int start = query_start[seq], end = query_start[seq + 1];
  const int first = first_positions ? first_positions[seq] : 0;
  if (start < 0 || start >= num_tokens || end <= start) return;
  int rows = end - start;
  rows = rows < num_tokens - start ? rows : num_tokens - start;
  rows = rows < 64 * words ? rows : 64 * words;

  __shared__ int16_t parent[kMaxDrafts];
  __shared__ unsigned long long bits[kMaxDrafts][kDraftWords];
  for (int i = tid; i < rows; i += kMaskThreads) {
    const int p = parents[start + i];
    parent[i] = static_cast<int16_t>(p >= 0 && p < i ? p : -1);
    for (int w = 0; w < words; ++w) bits[i][w] = 0;
  }
  __syncthreads();
  for (int i = tid; i < rows; i += kMaskThreads) {
    int depth = -1;
    for (int p = i; p >= 0; p = parent[p]) {
      bits[i][p >> 6] |= 1ull << (p & 63);
      ++depth;
    }
    if (positions) positions[start + i] = first + depth;
  }
  if (!masks) return;
  __syncthreads();
  for (int i = tid; i < rows * words; i += kMaskThreads)
    masks[static_cast<int64_t>(start) * words + i] = static_cast<int64_t>(bits[i / words][i % words]);
}

hipError_t launch_draft_masks(const int32_t* parents, const int32_t* query_start, int num_tokens,
                              int num_seqs, int64_t* masks, int words, const int32_t* first_positions,
                              int32_t* positions, hipStream_t stream) {
  hipLaunchKernelGGL(draft_masks_kernel, dim3(num_seqs), dim3(kMaskThreads), 0, stream, parents, query_start,
                     num_tokens, masks, words, first_positions, positions);
  return hipGetLastError();
}

}  // namespace lora
