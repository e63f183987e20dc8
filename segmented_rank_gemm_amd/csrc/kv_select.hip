// lora_kv_select: which tokens of a sequence that has more than `budget` of them each
// key head keeps: the first `sinks`, the last `recent`, and of the others the heaviest;
// of equal ones the first.  Their numbers come out ascending.
//
// A workgroup a (sequence, key head).  The weight of the last one that is kept is found
// exactly, digit by digit of the weights' bits (in an order in which bits compare as the
// numbers do): a histogram of the digit over what the digits before left, and the bin in
// which the count from the top passes what is still to be kept.  Then one ordered pass
// writes those above it and the first of those equal to it.

#include "kv_format.hpp"

namespace lora {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWaves = kSelectThreads / kWave;
constexpr int kDigit = 8;
constexpr int kBins = 1 << kDigit;
constexpr int kCopies = 16;  // of the histogram, so that a wave's lanes seldom meet in one

struct SelectArgs {
  const float* mass;
  const int32_t* seq_lens;
  const int32_t* page_table;
  int64_t ld_table;
  int32_t* kept;
  int32_t* new_lens;
  int num_pages, page_shift, kv_heads, max_seq_len, sinks, recent, budget;
};

// Bits that compare as the weights do; a NaN counts as -infinity, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) w = -INFINITY;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b >> 31 ? ~b : b | 0x80000000u;
}

// The weights of tokens [token, token + 4) in that order, token a multiple of 4.  A
// page that does not exist weighs -infinity.
__device__ __forceinline__ u32x4 orders_at(const SelectArgs& a, const int32_t* table, int head, int token) {
  const int page = table[(token < a.max_seq_len ? token : a.max_seq_len - 1) >> a.page_shift];
  const bool ok = token < a.max_seq_len && page >= 0 && page < a.num_pages;
  const u32x4 w = load16(a.mass + (((static_cast<int64_t>(ok ? page : 0) * a.kv_heads + head) << a.page_shift) +
                                   (token & ((1 << a.page_shift) - 1))));
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = order_of(ok ? __uint_as_float(w[i]) : -INFINITY);
  return o;
}

__global__ __launch_bounds__(kSelectThreads) void kv_select_kernel(SelectArgs a) {
  const int head = static_cast<int>(blockIdx.x), seq = static_cast<int>(blockIdx.y);
  const int tid = static_cast<int>(threadIdx.x), wave = wave_index(), lane = lane_id();
  int n = a.seq_lens[seq];
  n = n < 0 ? 0 : (n < a.max_seq_len ? n : a.max_seq_len);
  int32_t* kept = a.kept + (static_cast<int64_t>(seq) * a.kv_heads + head) * a.budget;
  if (head == 0 && tid == 0) a.new_lens[seq] = n < a.budget ? n : a.budget;
  if (n <= a.budget) {
    for (int i = tid; i < a.budget; i += kSelectThreads) kept[i] = i < n ? i : -1;
    return;
  }
  const int32_t* table = a.page_table + seq * a.ld_table;
  const int low = a.sinks, high = n - a.recent;  // those between are weighed
  __shared__ uint32_t bins[kCopies][kBins + 1];
  __shared__ uint32_t found[2];  // the digit, and how many are still to be kept in it
  uint32_t prefix = 0, known = 0;  // digits found so far, and their bits
  uint32_t need = static_cast<uint32_t>(a.budget - a.sinks - a.recent);
  for (int shift = 32 - kDigit; shift >= 0 && need > 0; shift -= kDigit) {
    for (int i = tid; i < kCopies * (kBins + 1); i += kSelectThreads) (&bins[0][0])[i] = 0;
    __syncthreads();
    for (int token = 4 * tid; token < high; token += 4 * kSelectThreads) {
      const u32x4 o = orders_at(a, table, head, token);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (token + i >= low && token + i < high && (o[i] & known) == prefix)
          atomicAdd(&bins[lane % kCopies][(o[i] >> shift) & (kBins - 1)], 1u);
    }
    __syncthreads();
    if (wave == 0) {
      // lane l has the bins [4 l, 4 l + 4), and of those above, the sum
      uint32_t sums[4], mine = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        sums[b] = 0;
        for (int k = 0; k < kCopies; ++k) sums[b] += bins[k][4 * lane + b];
        mine += sums[b];
      }
      uint32_t above = mine;
#pragma unroll
      for (int d = 1; d < kWave; d *= 2) {
        const uint32_t other = __shfl_down(above, d);
        above += lane + d < kWave ? other : 0u;
      }
      above -= mine;
#pragma unroll
      for (int b = 3; b >= 0; --b) {
        if (above < need && above + sums[b] >= need) {
          found[0] = static_cast<uint32_t>(4 * lane + b);
          found[1] = need - above;
        }
        above += sums[b];
      }
    }
    __syncthreads();
    prefix |= found[0] << shift;
    known |= static_cast<uint32_t>(kBins - 1) << shift;
    need = found[1];
  }
  const bool choose = a.budget > a.sinks + a.recent;

  // In order: how many are kept before each, and how many equal the last one that is.
  __shared__ uint32_t totals[2][kSelectWaves];
  int kept_before = 0, equal_before = 0;
  for (int base = 0, flip = 0; base < n; base += 4 * kSelectThreads, flip ^= 1) {
    const int token = base + 4 * tid;
    const u32x4 o = orders_at(a, table, head, token);
    bool keep[4], equal[4];
    int mine = 0;  // kept ones below, equal ones above
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = token + i;
      const bool weighed = at >= low && at < high;
      keep[i] = at < n && (!weighed || (choose && o[i] > prefix));
      equal[i] = choose && weighed && o[i] == prefix;
      mine += (keep[i] ? 1 : 0) + (equal[i] ? 1 << 16 : 0);
    }
    int before = wave_exclusive_sum(mine & 0xFFFF) + (wave_exclusive_sum(mine >> 16) << 16);
    if (lane == kWave - 1) totals[flip][wave] = static_cast<uint32_t>(before + mine);
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < kSelectWaves; ++w) {
      const int of = static_cast<int>(totals[flip][w]);
      if (w < wave) before += of;
      all += of;
    }
    int k = kept_before + (before & 0xFFFF), e = equal_before + (before >> 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int taken = e < static_cast<int>(need) ? e : static_cast<int>(need);
      if (keep[i] || (equal[i] && e < static_cast<int>(need))) kept[k + taken] = token + i;
      k += keep[i] ? 1 : 0;
      e += equal[i] ? 1 : 0;
    }
    kept_before += all & 0xFFFF;
    equal_before += all >> 16;
  }
}

hipError_t launch_kv_select(const float* mass, int num_pages, int page_shift, const int32_t* seq_lens,
                            const int32_t* page_table, int64_t ld_table, int num_seqs, int kv_heads,
                            int max_seq_len, int sinks, int recent, int32_t* kept, int budget,
                            int32_t* new_lens, hipStream_t stream) {
  const SelectArgs a = {mass, seq_lens, page_table, ld_table, kept, new_lens, num_pages, page_shift,
                        kv_heads, max_seq_len, sinks, recent, budget};
  hipLaunchKernelGGL(kv_select_kernel, dim3(kv_heads, num_seqs), dim3(kSelectThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace lora
