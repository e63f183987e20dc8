// lora_kv_select: which tokens of a sequence that has more than `budget` of them each
// key head keeps: the first `sinks`, the last `recent`, and of the others the heaviest;
// of equal ones the first.  Their numbers come out ascending.
//
// A workgroup a (sequence, key head); each of its waves has a run of the tokens.  The
// weight of the last one that is kept is found exactly, digit by digit of the weights'
// bits: a histogram of the digit over what the digits before left, and the bin in which
// the count from the top passes what is still to be kept.  Then every wave knows how
// many are kept before its run, and writes its own.
//
// The weights are read once, into registers, where max_seq_len tokens fit (32 a thread).
// Longer sequences are read once for the first digit, once for those that share it with
// the last one kept, which go on from shared memory, and once to write.
//
// Non-negative numbers compare as their bits do.  Where there are others (NaNs, which
// count as -infinity, and pages that do not exist, which weigh as much, among them),
// which the first reading finds out, the bits are turned into ones that do.

#include "kv_format.hpp"

namespace lora {

// Waves of a workgroup.  Several workgroups of 8 share a compute unit; of 16, two do not.
constexpr int kFewWaves = 8, kManyWaves = 16;
constexpr int kVector = 4 * kWave;  // tokens of a wave's load
constexpr int kInFlight = 4;        // of them, for long sequences
constexpr int kBins = 2048;         // digits of 11, 11 and 10 bits
constexpr int kShared = 32;         // weights of a thread's that go on from shared memory

struct SelectArgs {
  const float* mass;
  const int32_t* seq_lens;
  const int32_t* page_table;
  int64_t ld_table;
  int32_t* kept;
  int32_t* new_lens;
  int num_pages, page_shift, kv_heads, max_seq_len, sinks, recent, budget;
};

constexpr uint32_t kInfinity = 0x7F800000u, kNegative = 0x80000000u;

// Bits that compare as any weights do; -0 as 0.
__device__ __forceinline__ uint32_t order_of(uint32_t bits) {
  const float w = __uint_as_float(bits);
  const int b = __float_as_int(w == w ? w + 0.f : -INFINITY);
  return static_cast<uint32_t>(b ^ (b >> 31 | static_cast<int>(kNegative)));
}

// A key head's weights as a lane finds them.  A vector starts at a multiple of 256
// tokens, and so of the page size: where a lane's four lie in their page is always the
// same, and of their address only the page is looked up.
struct Source {
  const char* base;      // of this lane's tokens in page 0
  uint32_t page_bytes;   // from one page to the next
  uint32_t num_pages;
  const int32_t* table;
  int shift, last;       // the table's last entry that may be read
};
__device__ __forceinline__ Source source_of(const SelectArgs& a, int seq, int head) {
  Source s;
  const int in = (1 << a.page_shift) - 1;
  s.base = reinterpret_cast<const char*>(a.mass + (head << a.page_shift) + (4 * lane_id() & in));
  s.page_bytes = static_cast<uint32_t>(a.kv_heads) << (a.page_shift + 2);
  s.num_pages = static_cast<uint32_t>(a.num_pages);
  s.table = a.page_table + seq * a.ld_table;
  s.shift = a.page_shift;
  s.last = (a.max_seq_len - 1) >> a.page_shift;
  return s;
}

// The pages of N vectors of a run, from token `first` of the wave on.
template <int N>
__device__ __forceinline__ void look_up(const Source& s, int first, uint32_t (&page)[N]) {
#pragma unroll
  for (int r = 0; r < N; ++r) {
    const int entry = ((first + r * kVector) >> s.shift) + (4 * lane_id() >> s.shift);
    page[r] = static_cast<uint32_t>(s.table[static_cast<uint32_t>(entry < s.last ? entry : s.last)]);
  }
}

// Their weights.
template <int N>
struct Weights {
  bool there[N];  // the page exists
  u32x4 w[N];

  __device__ __forceinline__ void load(const Source& s, const uint32_t (&page)[N]) {
#pragma unroll
    for (int r = 0; r < N; ++r) {
      there[r] = page[r] < s.num_pages;
      w[r] = load16(s.base + static_cast<uint64_t>(there[r] ? page[r] : 0u) * s.page_bytes);
    }
  }
  __device__ __forceinline__ void check_pages() {
#pragma unroll
    for (int r = 0; r < N; ++r)
      if (__any(!there[r]) && !there[r]) w[r] = u32x4{kNegative | kInfinity, kNegative | kInfinity, kNegative | kInfinity, kNegative | kInfinity};
  }
  __device__ __forceinline__ void order() {
#pragma unroll
    for (int r = 0; r < N; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) w[r][i] = order_of(w[r][i]);
  }
};

// What has been found of the last one kept: its digits so far (prefix, under known), and
// how many of those with these digits are kept.
struct Border {
  uint32_t prefix, known, need;
  __device__ __forceinline__ bool shares(uint32_t w) const { return (w & known) == prefix; }
  __device__ __forceinline__ uint32_t top() const { return prefix | ~known; }  // of those that share them
};

struct Finder {
  uint32_t bins[kBins];
  uint32_t above[kManyWaves];
  uint32_t digit, need, count;
};

template <int WAVES>
__device__ __forceinline__ void clear_bins(Finder& f) {
  for (int i = static_cast<int>(threadIdx.x); i < kBins; i += WAVES * kWave) f.bins[i] = 0;
  __syncthreads();
}

// The digit at `shift` of the last one kept, from the histogram; the number of weights
// that share it with the digits before is returned.
template <int WAVES>
__device__ __forceinline__ uint32_t find_digit(Finder& f, Border& b, int shift, int bits) {
  const int tid = static_cast<int>(threadIdx.x), wave = wave_index(), lane = lane_id();
  __syncthreads();
  constexpr int kMine = kBins / (WAVES * kWave);  // bins of a thread
  uint32_t sums[kMine], mine = 0;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    sums[i] = f.bins[kMine * tid + i];
    mine += sums[i];
  }
  uint32_t above = mine;  // this thread's bins' and those above them in the wave
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const uint32_t other = __shfl_down(above, d);
    above += lane + d < kWave ? other : 0u;
  }
  if (lane == 0) f.above[wave] = above;
  __syncthreads();
  above -= mine;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) above += w > wave ? f.above[w] : 0u;
#pragma unroll
  for (int i = kMine - 1; i >= 0; --i) {
    if (above < b.need && above + sums[i] >= b.need) {
      f.digit = static_cast<uint32_t>(kMine * tid + i);
      f.need = b.need - above;
      f.count = sums[i];
    }
    above += sums[i];
  }
  __syncthreads();
  b.prefix |= f.digit << shift;
  b.known |= ((1u << bits) - 1) << shift;
  b.need = f.need;
  return f.count;
}

// Does `visit(first, weights)` for a wave's run [begin, end) of a long sequence, the next
// vectors on their way meanwhile.
template <typename Visit>
__device__ __forceinline__ void run_of(const Source& s, int begin, int end, bool turned, const Visit& visit) {
  if (begin >= end) return;
  constexpr int kStep = kInFlight * kVector;
  uint32_t pages[kInFlight];
  Weights<kInFlight> next;
  look_up(s, begin, pages);
  next.load(s, pages);
  look_up(s, begin + kStep, pages);
  for (int first = begin; first < end; first += kStep) {
    Weights<kInFlight> now = next;
    now.check_pages();
    if (turned) now.order();
    next.load(s, pages);
    look_up(s, first + 2 * kStep, pages);
#pragma unroll
    for (int r = 0; r < kInFlight; ++r)
      if (first + r * kVector < end) visit(first + r * kVector, now.w[r]);
  }
}

// R: vectors of a thread that are kept in registers; 0: sequences that do not fit.
template <int R, int WAVES>
__global__ __launch_bounds__(WAVES * kWave) void kv_select_kernel(SelectArgs a) {
  const int head = static_cast<int>(blockIdx.x), seq = static_cast<int>(blockIdx.y);
  const int tid = static_cast<int>(threadIdx.x), wave = wave_index(), lane = lane_id();
  const Source source = source_of(a, seq, head);
  Weights<R ? R : 1> own;
  if constexpr (R > 0) {  // beside the length
    uint32_t pages[R];
    look_up(source, wave * R * kVector, pages);
    own.load(source, pages);
  }
  int n = a.seq_lens[seq];
  n = n < 0 ? 0 : (n < a.max_seq_len ? n : a.max_seq_len);
  int32_t* kept = a.kept + (static_cast<int64_t>(seq) * a.kv_heads + head) * a.budget;
  if (head == 0 && tid == 0) a.new_lens[seq] = n < a.budget ? n : a.budget;
  if (n <= a.budget) {
    for (int i = tid; i < a.budget; i += WAVES * kWave) kept[i] = i < n ? i : -1;
    return;
  }
  const int low = a.sinks, high = n - a.recent;  // those between are weighed
  // This wave's run.
  const int length = R ? R * kVector : (n + WAVES * kVector - 1) / (WAVES * kVector) * kVector;
  const int begin = wave * length < n ? wave * length : n;
  const int end = begin + length < n ? begin + length : n;
  bool turned = false;
  const auto all = [&](const auto& visit) {
    if constexpr (R > 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) visit(begin + r * kVector, own.w[r]);
    } else {
      run_of(source, begin, end, turned, visit);
    }
  };
  // f(w, is it weighed) of a vector's, by the whole wave
  const auto weighed = [&](int first, const u32x4& w, const auto& f) {
    if (first >= low && first + kVector <= high) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f(w[i], true);
    } else if (first + kVector > low && first < high) {
      const int token = first + 4 * lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) f(w[i], token + i >= low && token + i < high);
    }
  };
  __shared__ Finder f;
  __shared__ uint32_t shared[R ? 1 : kShared][R ? 1 : WAVES * kWave];
  __shared__ uint32_t totals[2][WAVES];

  Border b = {0, 0, static_cast<uint32_t>(a.budget - a.sinks - a.recent)};
  uint32_t above = 0, mine = 0;  // of the run, above the first digit; of this thread's, that share it
  bool gathered = false;
  if (b.need == 0) {
    b.prefix = b.known = 0xFFFFFFFFu;  // none is above, and none of the equal ones is taken
  } else {
    clear_bins<WAVES>(f);
    const auto first_digit = [&] {
      uint32_t most = 0;
      all([&](int first, const u32x4& w) {
        weighed(first, w, [&](uint32_t x, bool in) {
          if (!in) return;
          most = x > most ? x : most;
          atomicAdd(&f.bins[x >> 21], 1u);
        });
      });
      return most;
    };
    if constexpr (R > 0) {
      own.check_pages();
      uint32_t most = 0;
      all([&](int first, const u32x4& w) { weighed(first, w, [&](uint32_t x, bool in) { most = in && x > most ? x : most; }); });
      turned = __syncthreads_or(most > kInfinity);
      if (turned) own.order();
      first_digit();
    } else {
      turned = __syncthreads_or(first_digit() > kInfinity);
      if (turned) {
        clear_bins<WAVES>(f);
        first_digit();
      }
    }
    uint32_t same = find_digit<WAVES>(f, b, 21, 11);
    // Done as soon as all that share the digits are kept.
    if (same != b.need) {
      clear_bins<WAVES>(f);
      if constexpr (R == 0) {
        const uint32_t top = b.top(), bottom = b.prefix, width = top - bottom;
        all([&](int first, const u32x4& w) {
          weighed(first, w, [&](uint32_t x, bool in) {
            above += static_cast<uint32_t>(__popcll(__ballot(in && x > top)));
            if (in && x - bottom <= width) {
              if (mine < kShared) shared[mine][tid] = x;
              ++mine;
            }
          });
        });
        gathered = !__syncthreads_or(mine > kShared);
      }
      // f(w) of those that share the first digit, at least
      const auto left = [&](const auto& f) {
        if (gathered) {
          for (uint32_t i = 0; i < mine; ++i) f(shared[i][tid], true);
        } else {
          all([&](int first, const u32x4& w) { weighed(first, w, f); });
        }
      };
      left([&](uint32_t x, bool in) {
        if (in && b.shares(x)) atomicAdd(&f.bins[x >> 10 & 2047u], 1u);
      });
      same = find_digit<WAVES>(f, b, 10, 11);
      if (same != b.need) {
        clear_bins<WAVES>(f);
        left([&](uint32_t x, bool in) {
          if (in && b.shares(x)) atomicAdd(&f.bins[x & 1023u], 1u);
        });
        find_digit<WAVES>(f, b, 0, 10);
      }
    }
  }

  // How many of the run are kept, and how many equal the last one that is (as far as its
  // digits were looked for).
  const uint32_t top = b.top(), bottom = b.prefix, need = b.need;
  // The lanes with a weight that is kept, and with one that is equal to the last one that
  // is, by the weight's place in the vector.
  struct Lanes {
    unsigned long long keep[4], equal[4];
  };
  const auto lanes_of = [&](int first, const u32x4& w) {
    Lanes l;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      l.keep[i] = __ballot(w[i] > top);
      l.equal[i] = __ballot(w[i] >= bottom) & ~l.keep[i];
    }
    if (first < low || first + kVector > high) {
      const int token = first + 4 * lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned long long weighed = __ballot(token + i >= low && token + i < high);
        l.keep[i] = (l.keep[i] & weighed) | (__ballot(token + i < n) & ~weighed);
        l.equal[i] &= weighed;
      }
    }
    return l;
  };
  uint32_t keeps = 0, equals = 0;
  if (gathered) {
    uint32_t k = 0, e = 0;
    for (uint32_t i = 0; i < mine; ++i) {
      const uint32_t x = shared[i][tid];
      k += x > top ? 1u : 0u;
      e += x >= bottom && x <= top ? 1u : 0u;
    }
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
      k += __shfl_xor(k, d);
      e += __shfl_xor(e, d);
    }
    // and those that are not weighed
    const int sinks = low < end ? low : end, last = high > begin ? high : begin;
    keeps = above + k + static_cast<uint32_t>((sinks > begin ? sinks - begin : 0) + (end > last ? end - last : 0));
    equals = e;
  } else {
    all([&](int first, const u32x4& w) {
      const Lanes l = lanes_of(first, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        keeps += static_cast<uint32_t>(__popcll(l.keep[i]));
        equals += static_cast<uint32_t>(__popcll(l.equal[i]));
      }
    });
  }
  if (lane == 0) {
    totals[0][wave] = keeps;
    totals[1][wave] = equals;
  }
  __syncthreads();
  uint32_t k0 = lane < wave ? totals[0][lane] : 0u, e0 = lane < wave ? totals[1][lane] : 0u;
#pragma unroll
  for (int d = 1; d < WAVES; d *= 2) {
    k0 += __shfl_xor(k0, d);
    e0 += __shfl_xor(e0, d);
  }
  k0 = __builtin_amdgcn_readfirstlane(k0);  // kept, and equal, before the vector
  e0 = __builtin_amdgcn_readfirstlane(e0);

  // (inside the list also where another stream writes the mass meanwhile)
  const auto put = [&](uint32_t at, int token) {
    if (at < static_cast<uint32_t>(a.budget)) kept[at] = token;
  };
  all([&](int first, const u32x4& w) {
    const Lanes l = lanes_of(first, w);
    const int token = first + 4 * lane;
    // in the lanes below, from `from` on; and in all
    const auto before = [](const unsigned long long (&m)[4], uint32_t from, uint32_t& all) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        from = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(m[i] >> 32),
                                         __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(m[i]), from));
        all += static_cast<uint32_t>(__popcll(m[i]));
      }
      return from;
    };
    const uint32_t taken = e0 < need ? e0 : need;
    uint32_t k = before(l.keep, k0, k0);
    const bool some = (l.equal[0] | l.equal[1] | l.equal[2] | l.equal[3]) != 0;
    if (!some && first >= low && first + kVector <= high) {
      k += taken;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (w[i] > top) put(k++, token + i);
    } else {
      uint32_t e = before(l.equal, e0, e0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool keep = l.keep[i] >> lane & 1, equal = l.equal[i] >> lane & 1;
        if (keep || (equal && e < need)) put(k + (e < need ? e : need), token + i);
        k += keep ? 1u : 0u;
        e += equal ? 1u : 0u;
      }
    }
  });
}

hipError_t launch_kv_select(const float* mass, int num_pages, int page_shift, const int32_t* seq_lens,
                            const int32_t* page_table, int64_t ld_table, int num_seqs, int kv_heads,
                            int max_seq_len, int sinks, int recent, int32_t* kept, int budget,
                            int32_t* new_lens, hipStream_t stream) {
  const SelectArgs a = {mass, seq_lens, page_table, ld_table, kept, new_lens, num_pages, page_shift,
                        kv_heads, max_seq_len, sinks, recent, budget};
  const dim3 grid(kv_heads, num_seqs), few(kFewWaves * kWave), many(kManyWaves * kWave);
  constexpr int kFit = kFewWaves * kVector;  // tokens of a vector a thread
  if (max_seq_len <= kFit) hipLaunchKernelGGL((kv_select_kernel<1, kFewWaves>), grid, few, 0, stream, a);
  else if (max_seq_len <= 2 * kFit) hipLaunchKernelGGL((kv_select_kernel<2, kFewWaves>), grid, few, 0, stream, a);
  else if (max_seq_len <= 4 * kFit) hipLaunchKernelGGL((kv_select_kernel<4, kFewWaves>), grid, few, 0, stream, a);
  else if (max_seq_len <= 8 * kFit) hipLaunchKernelGGL((kv_select_kernel<4, kManyWaves>), grid, many, 0, stream, a);
  else hipLaunchKernelGGL((kv_select_kernel<0, kManyWaves>), grid, many, 0, stream, a);
  return hipGetLastError();
}

}  // namespace lora
