// lora_kv_compact: kept tokens to the places in front, codes, scales and weights:
//   place first + j  <-  place first + kept[j]
//
// Into other pages nothing has to be waited for, and the list is shared out.
// In place a workgroup has a (sequence, key head, keys or values) and takes the list in
// blocks from the front: everything a block moves is in registers before any of it is
// written.  As kept[j] >= j, a block's places lie in front of all that later blocks
// still have to read, so that every place gets what its source held before the call;
// and no other workgroup touches these bytes.
//
// Long lists of few key heads leave the device idle that way (2 x 8 workgroups, 65536
// tokens: 248 us).  Where the tokens lie a thousand places ahead of where they go, and
// further on always do, the moves are followed from the other end: a place that is no
// source itself takes its token, whose place takes its own, and so on.  These chains
// have nothing in common, each step is a thousand places long, and there are as many of
// them as tokens were left out.  What lies before goes in blocks first, in a launch of
// its own (that list: 71 us in all).
//
// A wave moves 64 tokens at a time, several times that in flight: each lane finds out
// where one token is and goes, and moves its scale bytes and its weight; the codes are
// moved by as many lanes a token as it has 16-byte pieces, which ask that lane.
//
// Bound by: HBM's lines of 128 bytes, of which a token's codes are 64 and its scale bytes
// one each (16 sequences of up to 8192 tokens, half of them into new pages, heads of 128,
// with the mass: 42 us, the 149 MB that have to move at 3.6 TB/s, 175 MB as counted at
// 4.2; chains, whose neighbours go different ways: 71 us, 242 MB as counted).

#include "kv_format.hpp"

namespace lora {

constexpr int kCompactThreads = 1024;  // at most
constexpr int kUnits = 4;              // of 64 tokens in flight
constexpr int kNearBlock = 1024;       // tokens of a block, where the rest goes by chains
constexpr int kFar = 1024;             // places that a chain's steps have at least
constexpr int kChainWaves = 4;

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

// One (sequence, key head, keys or values) of a call.
template <int D>
struct Mover {
  static constexpr int kPieces = D / 32;  // of a token's codes; and its scale bytes
  const int32_t* kept;
  const int32_t* table;
  const int32_t* dst_table;
  uint8_t* bytes;       // of page 0
  float* mass;          // of page 0; null where the weights are not this one's to move
  int64_t first, places, dst_places, page_bytes, mass_stride;
  int count, shift, in, num_pages;

  // What a wave holds of 64 tokens.
  struct Held {
    u32x4 codes[kPieces];
    uint8_t scales[kPieces];
    float weight;
  };

  __device__ __forceinline__ Mover(const CompactArgs& a, int seq, int head, int part) {
    count = a.counts[seq];
    count = count < a.max_kept ? count : a.max_kept;
    first = a.first ? a.first[seq] : 0;
    if (first < 0) count = 0;
    shift = a.cache.page_shift;
    in = (1 << shift) - 1;
    num_pages = a.cache.num_pages;
    kept = a.kept + (static_cast<int64_t>(seq) * a.lists + (a.lists > 1 ? head : 0)) * a.max_kept;
    table = a.table + seq * a.ld_table;
    dst_table = a.dst_table ? a.dst_table + seq * a.ld_dst : table;
    places = static_cast<int64_t>(a.pages) << shift;
    dst_places = static_cast<int64_t>(a.dst_table ? a.dst_pages : a.pages) << shift;
    const int64_t block_bytes = static_cast<int64_t>(D / 2 + kPieces) << shift;
    page_bytes = 2 * a.cache.kv_heads * block_bytes;
    bytes = a.cache.data + (part * a.cache.kv_heads + head) * block_bytes;
    mass = a.mass && part == 0 ? a.mass + (static_cast<int64_t>(head) << shift) : nullptr;
    mass_stride = static_cast<int64_t>(a.cache.kv_heads) << shift;
  }
  __device__ __forceinline__ bool has(int page) const { return page >= 0 && page < num_pages; }
  // at: each lane's token's place in its page.  (Loads without conditions, of a page that
  // is there: the wait before a use counts the loads behind it.)
  __device__ __forceinline__ void load(Held& h, int page, int at) const {
    const int lane = lane_id();
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      const int of = p * (kWave / kPieces) + lane / kPieces;
      h.codes[p] = load16(bytes + __shfl(page, of) * page_bytes + __shfl(at, of) * (D / 2) + lane % kPieces * 16);
    }
    const uint8_t* s = bytes + page * page_bytes + ((D / 2) << shift) + at;
#pragma unroll
    for (int p = 0; p < kPieces; ++p) h.scales[p] = s[p << shift];
  }
  __device__ __forceinline__ void load_weight(Held& h, int page, int at) const {
    if (mass) h.weight = mass[page * mass_stride + at];
  }
  // page: -1 for a token that does not move.
  __device__ __forceinline__ void store(const Held& h, int page, int at) const {
    const int lane = lane_id();
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      const int of = p * (kWave / kPieces) + lane / kPieces;
      const int to = __shfl(page, of), place = __shfl(at, of);
      if (to >= 0) store16(bytes + to * page_bytes + place * (D / 2) + lane % kPieces * 16, h.codes[p]);
    }
    if (page < 0) return;
    uint8_t* s = bytes + page * page_bytes + ((D / 2) << shift) + at;
#pragma unroll
    for (int p = 0; p < kPieces; ++p) s[p << shift] = h.scales[p];
    if (mass) mass[page * mass_stride + at] = h.weight;
  }
};

// The list's entries from `base` on, as many as the workgroup's waves take with U units each.
template <int D, int U>
__device__ __forceinline__ void move_block(const Mover<D>& m, bool in_place, int base) {
  const int lane = lane_id(), wave = wave_index();
  int page[U], to_page[U], at[U], to_at[U];
  typename Mover<D>::Held held[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int j = base + (wave * U + u) * kWave + lane;
    const int number = m.kept[j < m.count ? j : m.count - 1];
    const int64_t from = m.first + number, to = m.first + j;
    // in place, a token that stays where it is stays; one from further ahead is skipped
    const bool moves = j < m.count && number >= 0 && from < m.places && to < m.dst_places && (!in_place || number > j);
    page[u] = moves ? m.table[from >> m.shift] : -1;
    to_page[u] = moves ? m.dst_table[to >> m.shift] : -1;
    at[u] = static_cast<int>(from) & m.in;
    to_at[u] = static_cast<int>(to) & m.in;
  }
  bool any = false;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool moves = m.has(page[u]) && m.has(to_page[u]);
    if (!moves) to_page[u] = -1;
    if (!moves) page[u] = 0;
    any |= moves;
  }
  any = __any(any);
  if (any) {
#pragma unroll
    for (int u = 0; u < U; ++u) m.load(held[u], page[u], at[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) m.load_weight(held[u], page[u], at[u]);
  }
  if (in_place) {
    // what this block reads has arrived before any of it is written
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  }
  if (!any) return;
#pragma unroll
  for (int u = 0; u < U; ++u) m.store(held[u], to_page[u], to_at[u]);
}

template <int D>
__device__ __forceinline__ Mover<D> mover_of(const CompactArgs& a) {
  return Mover<D>(a, static_cast<int>(blockIdx.y), static_cast<int>(blockIdx.x) >> 1, static_cast<int>(blockIdx.x) & 1);
}

// U: units of a wave.
template <int D, int U>
__global__ __launch_bounds__(kCompactThreads) void kv_compact_kernel(CompactArgs a) {
  const Mover<D> m = mover_of<D>(a);
  const int tokens = static_cast<int>(blockDim.x) * U;
  const int step = static_cast<int>(gridDim.z) * tokens;
  for (int base = static_cast<int>(blockIdx.z) * tokens; base < m.count; base += step)
    move_block<D, U>(m, !a.dst_table, base);
}

// The first block of the list whose tokens come from far (the list's end if none does).
template <int D>
__device__ __forceinline__ int first_far(const Mover<D>& m) {
  for (int base = 0; base < m.count; base += kWave * kNearBlock) {
    const int64_t j = base + static_cast<int64_t>(lane_id()) * kNearBlock;
    const unsigned long long far = __ballot(j < m.count && m.kept[j < m.count ? j : 0] - j >= kFar);
    if (far) return base + (__ffsll(static_cast<long long>(far)) - 1) * kNearBlock;
  }
  return m.count;
}

// In place, the blocks before it: several at a time as long as there are as many.
template <int D>
__global__ __launch_bounds__(kNearBlock) void kv_compact_near_kernel(CompactArgs a) {
  const Mover<D> m = mover_of<D>(a);
  const int end = first_far(m);
  for (int base = 0; base < end;) {
    if (end == m.count || end - base >= kUnits * kNearBlock) {
      move_block<D, kUnits>(m, true, base);
      base += kUnits * kNearBlock;
    } else {
      move_block<D, 1>(m, true, base);
      base += kNearBlock;
    }
  }
}

// The rest of the list, in place, by chains.
template <int D>
__global__ __launch_bounds__(kChainWaves * kWave) void kv_compact_chain_kernel(CompactArgs a) {
  const Mover<D> m = mover_of<D>(a);
  const int lane = lane_id(), wave = wave_index();
  const int from = first_far(m);
  __shared__ uint32_t sources[kChainWaves][kWave];
  const int step = static_cast<int>(gridDim.z) * kChainWaves * kWave;
  for (int start = from + (static_cast<int>(blockIdx.z) * kChainWaves + wave) * kWave; start < m.count; start += step) {
    // The first entry from `start` on: of 64 even parts the one that it is in, until
    // they are single entries.  (Those below 0, behind all others, count as large.)
    int low = from, high = m.count;
    while (high > low) {
      const int part = (high - low + kWave - 1) / kWave;
      const int64_t probe = low + static_cast<int64_t>(lane) * part;
      const uint32_t entry = static_cast<uint32_t>(m.kept[probe < high ? probe : low]);
      const int before = static_cast<int>(__popcll(__ballot(probe < high && entry < static_cast<uint32_t>(start))));
      if (before == 0) break;
      const int64_t next = low + static_cast<int64_t>(before) * part;
      low = low + (before - 1) * part + 1;
      high = next < high ? static_cast<int>(next) : high;
    }
    // Which of the 64 places from `start` on are sources: they stand there, ascending.
    sources[wave][lane] = 0;
    __builtin_amdgcn_wave_barrier();
    const int64_t entry = static_cast<int64_t>(low) + lane;
    const int source = entry < m.count ? m.kept[entry] : -1;
    if (source >= start && source - start < kWave) sources[wave][source - start] = 1;
    __builtin_amdgcn_wave_barrier();
    int place = start + lane;
    bool active = place < m.count && sources[wave][lane] == 0;
    __builtin_amdgcn_wave_barrier();
    // Every step goes ahead, so that each chain ends at the list's.
    int next = active ? m.kept[place] : 0;
    int to_page = active && m.first + place < m.places ? m.table[(m.first + place) >> m.shift] : -1;
    while (__any(active)) {
      const int64_t at = m.first + next;
      const bool ahead = active && next > place && at < m.places;
      int page = ahead ? m.table[at >> m.shift] : -1;
      const int to_at = static_cast<int>(m.first + place) & m.in;
      const bool moves = ahead && m.has(page) && m.has(to_page);
      active = ahead && next < m.count;
      const int after = active ? m.kept[next] : 0;
      typename Mover<D>::Held held;
      const int from_page = moves ? page : 0, from_at = static_cast<int>(at) & m.in;
      m.load(held, from_page, from_at);
      m.load_weight(held, from_page, from_at);
      m.store(held, moves ? to_page : -1, to_at);
      place = next;
      next = after;
      to_page = page;
    }
  }
}

template <int D>
static void launch_compact(const CompactArgs& a, int num_seqs, hipStream_t stream) {
  const int64_t units = static_cast<int64_t>(num_seqs) * a.cache.kv_heads * 2;
  const dim3 grid(2 * a.cache.kv_heads, num_seqs, 1);
  // By chains where the device has more compute units than half of them could use, and
  // the list more than a few blocks (us, chains / blocks, half of the tokens, 8 heads of
  // 128: 5000 entries of one sequence 16.8 / 18.6, 16384 22 / 47, 65536 72 / 248; of 4
  // sequences, 64 units, 5000 22.4 / 22.1, 16384 65 / 78, 32768 130 / 154, where the bytes
  // that move take 27 and 54).  A list that leaves out next to nothing has few chains (16
  // tokens of 65552: 147 / 141).
  if (!a.dst_table && units <= kCus / 4 && a.max_kept > 4 * kNearBlock) {
    hipLaunchKernelGGL(kv_compact_near_kernel<D>, grid, dim3(kNearBlock), 0, stream, a);
    const int64_t all = (static_cast<int64_t>(a.max_kept) + kChainWaves * kWave - 1) / (kChainWaves * kWave);
    int64_t ranges = (16 * kCus + units - 1) / units;
    ranges = ranges < all ? ranges : all;
    hipLaunchKernelGGL(kv_compact_chain_kernel<D>, dim3(grid.x, grid.y, static_cast<unsigned>(ranges)),
                       dim3(kChainWaves * kWave), 0, stream, a);
    return;
  }
  // A few accepted drafts: a wave's lanes hold a list, and wait for no others' loads
  // (64 sequences of 6: 3.0 us, with four times as many in flight 4.5).
  if (a.max_kept <= kNearBlock) {
    const int threads = (a.max_kept + kWave - 1) / kWave * kWave;
    hipLaunchKernelGGL((kv_compact_kernel<D, 1>), grid, dim3(threads), 0, stream, a);
    return;
  }
  // In place as many waves as the list keeps busy, up to 16; into other pages four, and
  // as many workgroups as fill the device.
  const int64_t waves = (static_cast<int64_t>(a.max_kept) + kUnits * kWave - 1) / (kUnits * kWave);
  const int64_t most = a.dst_table ? 4 : kCompactThreads / kWave;
  const int threads = static_cast<int>(waves < most ? waves : most) * kWave;
  int64_t ranges = 1;
  if (a.dst_table) {
    const int64_t all = (waves + most - 1) / most;
    ranges = (8 * kCus + units - 1) / units;
    ranges = ranges < all ? ranges : all;
  }
  hipLaunchKernelGGL((kv_compact_kernel<D, kUnits>), dim3(grid.x, grid.y, static_cast<unsigned>(ranges)),
                     dim3(threads), 0, stream, a);
}

hipError_t launch_kv_compact(const int32_t* kept, int lists, int max_kept, const int32_t* counts,
                             const int32_t* first, const int32_t* page_table, int64_t ld_table, int pages,
                             const int32_t* dst_table, int64_t ld_dst, int dst_pages, uint8_t* cache,
                             int num_pages, int page_shift, int num_seqs, int kv_heads, int head_dim,
                             float* mass, hipStream_t stream) {
  const CompactArgs a = {kept, counts, first, page_table, dst_table, ld_table, ld_dst,
                         {cache, num_pages, page_shift, kv_heads}, mass, lists, max_kept, pages, dst_pages};
  if (head_dim == 64) launch_compact<64>(a, num_seqs, stream);
  else launch_compact<128>(a, num_seqs, stream);
  return hipGetLastError();
}

}  // namespace lora
