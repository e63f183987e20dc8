// lora_kv_compact: kept tokens to the places in front, codes, scales and weights:
//   place first + j  <-  place first + kept[j]
//
// A workgroup a (sequence, key head, keys or values) where this is done in place.  It
// takes the list in blocks from the front: everything a block moves is in registers
// before any of it is written.  As kept[j] >= j, a block's places lie in front of all
// that later blocks still have to read, so that every place gets what its source held
// before the call; and no other workgroup touches these bytes.
// Into other pages nothing has to be waited for, and the list is shared out.
//
// A thread moves 16 bytes of codes and one scale byte, of which a token's head has as
// many pieces each; the first piece's takes the weight along.

#include "kv_format.hpp"

namespace lora {

constexpr int kCompactThreads = 1024;

struct CompactArgs {
  const int32_t* kept;
  const int32_t* counts;
  const int32_t* first;       // may be null
  const int32_t* table;
  const int32_t* dst_table;   // may be null: in place
  int64_t ld_table, ld_dst;
  Cache<uint8_t> cache;
  float* mass;                // may be null
  int lists, max_kept, pages, dst_pages;
};

template <int D>
__global__ __launch_bounds__(kCompactThreads) void kv_compact_kernel(CompactArgs a) {
  constexpr int kPieces = D / 32;
  constexpr int kTokens = kCompactThreads / kPieces;  // a step's
  const int head = static_cast<int>(blockIdx.x) >> 1, part = static_cast<int>(blockIdx.x) & 1;
  const int seq = static_cast<int>(blockIdx.y);
  const int tid = static_cast<int>(threadIdx.x), piece = tid % kPieces;
  int count = a.counts[seq];
  count = count < a.max_kept ? count : a.max_kept;
  const int64_t first = a.first ? a.first[seq] : 0;
  const int shift = a.cache.page_shift, in = (1 << shift) - 1;
  const int32_t* kept = a.kept + (static_cast<int64_t>(seq) * a.lists + (a.lists > 1 ? head : 0)) * a.max_kept;
  const int32_t* table = a.table + seq * a.ld_table;
  const int32_t* dst_table = a.dst_table ? a.dst_table + seq * a.ld_dst : table;
  const int64_t places = static_cast<int64_t>(a.pages) << shift;
  const int64_t dst_places = static_cast<int64_t>(a.dst_table ? a.dst_pages : a.pages) << shift;
  const bool weights = a.mass && part == 0 && piece == 0;

  const int step = static_cast<int>(gridDim.z) * kTokens;
  for (int base = static_cast<int>(blockIdx.z) * kTokens; base < count; base += step) {
    const int j = base + tid / kPieces;
    u32x4 codes = {0, 0, 0, 0};
    uint8_t scale = 0;
    float weight = 0.f;
    int to_page = -1;
    const int64_t to = first + j;
    if (j < count && first >= 0 && to < dst_places) {
      const int32_t number = kept[j];
      const int64_t from = first + number;
      // in place, a token that stays where it is stays; one from further ahead is skipped
      if (number >= 0 && from < places && (a.dst_table || number > j)) {
        const int page = table[from >> shift], dst = dst_table[to >> shift];
        if (page >= 0 && page < a.cache.num_pages && dst >= 0 && dst < a.cache.num_pages) {
          const uint8_t* block = a.cache.block<D>(page, part, head);
          const int at = static_cast<int>(from) & in;
          codes = load16(block + at * (D / 2) + piece * 16);
          scale = block[a.cache.scales_at<D>() + (piece << shift) + at];
          if (weights) weight = a.mass[((static_cast<int64_t>(page) * a.cache.kv_heads + head) << shift) + at];
          to_page = dst;
        }
      }
    }
    if (!a.dst_table) {
      // what this block reads has arrived before any of it is written
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
    }
    if (to_page >= 0) {
      uint8_t* block = a.cache.block<D>(to_page, part, head);
      const int at = static_cast<int>(to) & in;
      store16(block + at * (D / 2) + piece * 16, codes);
      block[a.cache.scales_at<D>() + (piece << shift) + at] = scale;
      if (weights) a.mass[((static_cast<int64_t>(to_page) * a.cache.kv_heads + head) << shift) + at] = weight;
    }
  }
}

hipError_t launch_kv_compact(const int32_t* kept, int lists, int max_kept, const int32_t* counts,
                             const int32_t* first, const int32_t* page_table, int64_t ld_table, int pages,
                             const int32_t* dst_table, int64_t ld_dst, int dst_pages, uint8_t* cache,
                             int num_pages, int page_shift, int num_seqs, int kv_heads, int head_dim,
                             float* mass, hipStream_t stream) {
  const CompactArgs a = {kept, counts, first, page_table, dst_table, ld_table, ld_dst,
                         {cache, num_pages, page_shift, kv_heads}, mass, lists, max_kept, pages, dst_pages};
  const int tokens = kCompactThreads / (head_dim / 32);
  int64_t ranges = 1;
  if (dst_table) {
    const int64_t units = static_cast<int64_t>(num_seqs) * kv_heads * 2, most = (max_kept + tokens - 1) / tokens;
    ranges = (8 * kCus + units - 1) / units;
    ranges = ranges < most ? ranges : most;
  }
  const dim3 grid(2 * kv_heads, num_seqs, static_cast<unsigned>(ranges));
  if (head_dim == 64) hipLaunchKernelGGL(kv_compact_kernel<64>, grid, dim3(kCompactThreads), 0, stream, a);
  else hipLaunchKernelGGL(kv_compact_kernel<128>, grid, dim3(kCompactThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace lora
