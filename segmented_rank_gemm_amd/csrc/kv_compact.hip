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
// A wave moves 64 tokens at a time, kUnits of them in flight: each lane finds out where
// one token is and goes, and moves its scale bytes and its weight; the codes are moved
// by as many lanes a token as it has 16-byte pieces, which ask that lane.

#include "kv_format.hpp"

namespace lora {

constexpr int kCompactThreads = 1024;  // at most
constexpr int kUnits = 4;

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
  constexpr int kPieces = D / 32;  // of a token's codes; and its scale bytes
  constexpr int kAtOnce = kWave / kPieces;
  const int head = static_cast<int>(blockIdx.x) >> 1, part = static_cast<int>(blockIdx.x) & 1;
  const int seq = static_cast<int>(blockIdx.y);
  const int lane = lane_id(), wave = wave_index(), waves = static_cast<int>(blockDim.x) / kWave;
  const int piece = lane % kPieces;
  int count = a.counts[seq];
  count = count < a.max_kept ? count : a.max_kept;
  const int64_t first = a.first ? a.first[seq] : 0;
  if (first < 0) return;
  const int shift = a.cache.page_shift, in = (1 << shift) - 1;
  const int32_t* kept = a.kept + (static_cast<int64_t>(seq) * a.lists + (a.lists > 1 ? head : 0)) * a.max_kept;
  const int32_t* table = a.table + seq * a.ld_table;
  const int32_t* dst_table = a.dst_table ? a.dst_table + seq * a.ld_dst : table;
  const int64_t places = static_cast<int64_t>(a.pages) << shift;
  const int64_t dst_places = static_cast<int64_t>(a.dst_table ? a.dst_pages : a.pages) << shift;
  const bool weights = a.mass && part == 0;
  const int64_t block_bytes = static_cast<int64_t>(D / 2 + kPieces) << shift;
  const int64_t page_bytes = 2 * a.cache.kv_heads * block_bytes;
  uint8_t* mine = a.cache.data + (part * a.cache.kv_heads + head) * block_bytes;  // of page 0

  const int tokens = waves * kUnits * kWave;
  const int step = static_cast<int>(gridDim.z) * tokens;
  for (int base = static_cast<int>(blockIdx.z) * tokens; base < count; base += step) {
    int page[kUnits], to_page[kUnits], at[kUnits];  // at: places in the two pages
    u32x4 codes[kUnits][kPieces];
    uint8_t scales[kUnits][kPieces];
    float weight[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int j = base + (wave * kUnits + u) * kWave + lane;
      const int number = kept[j < count ? j : count - 1];
      const int64_t from = first + number, to = first + j;
      // in place, a token that stays where it is stays; one from further ahead is skipped
      const bool moves = j < count && number >= 0 && from < places && to < dst_places && (a.dst_table || number > j);
      page[u] = moves ? table[from >> shift] : -1;
      to_page[u] = moves ? dst_table[to >> shift] : -1;
      at[u] = (static_cast<int>(from) & in) | (static_cast<int>(to) & in) << 16;
    }
    bool any = false;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const bool moves = page[u] >= 0 && page[u] < a.cache.num_pages && to_page[u] >= 0 && to_page[u] < a.cache.num_pages;
      if (!moves) to_page[u] = -1;
      if (!moves) page[u] = 0;  // which is there, and is not written to
      any |= moves;
    }
    any = __any(any);
    if (any) {
      // (loads without conditions: the wait before a use counts the loads behind it)
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          const int of = p * kAtOnce + lane / kPieces;
          const int from = __shfl(at[u], of) & 0xFFFF;
          codes[u][p] = load16(mine + __shfl(page[u], of) * page_bytes + from * (D / 2) + piece * 16);
        }
        const uint8_t* s = mine + page[u] * page_bytes + ((D / 2) << shift) + (at[u] & 0xFFFF);
#pragma unroll
        for (int p = 0; p < kPieces; ++p) scales[u][p] = s[p << shift];
      }
      if (weights) {
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
          weight[u] = a.mass[((static_cast<int64_t>(page[u]) * a.cache.kv_heads + head) << shift) + (at[u] & 0xFFFF)];
      }
    }
    if (!a.dst_table) {
      // what this block reads has arrived before any of it is written
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
    }
    if (!any) continue;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const int of = p * kAtOnce + lane / kPieces;
        const int to = __shfl(to_page[u], of), place = __shfl(at[u], of) >> 16;
        if (to >= 0) store16(mine + to * page_bytes + place * (D / 2) + piece * 16, codes[u][p]);
      }
      if (to_page[u] < 0) continue;
      uint8_t* s = mine + to_page[u] * page_bytes + ((D / 2) << shift) + (at[u] >> 16);
#pragma unroll
      for (int p = 0; p < kPieces; ++p) s[p << shift] = scales[u][p];
      if (weights)
        a.mass[((static_cast<int64_t>(to_page[u]) * a.cache.kv_heads + head) << shift) + (at[u] >> 16)] = weight[u];
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
  // In place as many waves as the list keeps busy, up to 16; into other pages four, and
  // as many workgroups as fill the device.
  const int64_t waves = (static_cast<int64_t>(max_kept) + kUnits * kWave - 1) / (kUnits * kWave);
  const int64_t most = dst_table ? 4 : kCompactThreads / kWave;
  const int threads = static_cast<int>(waves < most ? waves : most) * kWave;
  int64_t ranges = 1;
  if (dst_table) {
    const int64_t units = static_cast<int64_t>(num_seqs) * kv_heads * 2, all = (waves + most - 1) / most;
    ranges = (8 * kCus + units - 1) / units;
    ranges = ranges < all ? ranges : all;
  }
  const dim3 grid(2 * kv_heads, num_seqs, static_cast<unsigned>(ranges));
  if (head_dim == 64) hipLaunchKernelGGL(kv_compact_kernel<64>, grid, dim3(threads), 0, stream, a);
  else hipLaunchKernelGGL(kv_compact_kernel<128>, grid, dim3(threads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace lora
