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
// A compute unit takes 15 us to read 131072 weights into a histogram, so a few long lists
// are cut into pieces of 8192 tokens, a workgroup each, and the digits into launches: each
// of them joins the histograms that the one before left (which also say how many are kept
// before the piece), and reads the piece again from the caches.
//
// Bound by: the histogram's additions in shared memory and the steps that follow from each
// other (64 sequences of 4097 to 8192 tokens, 8 key heads: 13.9 us, the 21 MB at 1.5 TB/s:
// up to the first histogram's end 6, then the digits 4, counting and writing 4; with 16
// waves 15.4); of few long lists what their pieces join: behind the first launch each
// piece reads the histograms of all of its list, 4 KB a piece (131072 tokens, 16 pieces:
// launches of 3.4, 5.8, 5.4 and 7 us, 21 in all, whole 58; 1048576 tokens, 128 pieces:
// 8.8, 35, 40 and 42); of many long lists HBM, for the three readings (64 sequences of
// 131072: 890 MB read and 135 written, 5.8 TB/s).
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
  uint32_t* work;  // of the pieces; NULL without
};

// A list in pieces: its stages are launches, between which each piece leaves its part of
// the digit's histogram (two bins a word), and what it knows.
constexpr int kPieceVectors = 2;                            // of a thread
constexpr int kPiece = kPieceVectors * kManyWaves * kVector;  // tokens
constexpr int kMostPieces = 128, kMostLists = 32;
constexpr int kWhole = -1, kLastStage = 3;  // stages 0, 1 and 2 count a digit; the last one writes
struct Known {
  uint32_t prefix, known, need;  // the border
  uint32_t keeps, equals;        // before the piece, of those above the border and at it
  uint32_t done, unused[2];      // nothing is left to be found
};
struct Pieces {
  uint32_t* counts;  // of the list's first piece
  Known* known;
  int number;

  static __host__ __device__ constexpr int64_t words(int pieces) {
    return pieces * static_cast<int64_t>(2 * (kBins / 2) + sizeof(Known) / sizeof(uint32_t));
  }
  __device__ __forceinline__ Pieces(const SelectArgs& a, int64_t list) : number((a.max_seq_len + kPiece - 1) / kPiece) {
    counts = a.work + list * words(number);
    known = reinterpret_cast<Known*>(counts + number * kBins);
  }
  // two histograms take turns: one is read while the next one is written
  __device__ __forceinline__ uint32_t* counts_of(int piece, int stage) const {
    return counts + (2 * piece + (stage & 1)) * (kBins / 2);
  }
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

// Sums over the lanes below.
__device__ __forceinline__ uint32_t sum_below(uint32_t v) {
  int x = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x138, 0xF, 0xF, false);  // the lane below's
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);  // within 16 lanes, 1, 2, 4 and 8 below
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);  // the last lane's of the 16 below,
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);  // and of the 32
  return static_cast<uint32_t>(x);
}

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
  uint32_t digit, need, count, equals;
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

// The digit at `shift` from the pieces' histograms of `stage`, of a list of n tokens; and
// what lies before this piece.
template <int WAVES>
__device__ __forceinline__ void join_pieces(Finder& f, Border& b, Known& k, const Pieces& pieces, int piece,
                                            int n, int stage, int shift, int bits) {
  static_assert(WAVES * kWave * 2 == kBins, "a word a thread");
  const int tid = static_cast<int>(threadIdx.x);
  const int number = (n + kPiece - 1) / kPiece;
  uint32_t all[2] = {0, 0}, before[2] = {0, 0};
#pragma unroll 8
  for (int p = 0; p < number; ++p) {
    const uint32_t two = pieces.counts_of(p, stage)[tid];
    if (p == piece) {
      before[0] = all[0];
      before[1] = all[1];
    }
    all[0] += two & 0xFFFFu;
    all[1] += two >> 16;
  }
  f.bins[2 * tid] = all[0];
  f.bins[2 * tid + 1] = all[1];
  const uint32_t same = find_digit<WAVES>(f, b, shift, bits);
  const uint32_t digit = f.digit, first = 2u * static_cast<uint32_t>(tid);
  uint32_t above = (first > digit ? before[0] : 0u) + (first + 1 > digit ? before[1] : 0u);
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) above += __shfl_xor(above, d);
  if (lane_id() == 0) f.above[wave_index()] = above;
  if (digit >> 1 == static_cast<uint32_t>(tid)) f.equals = before[digit & 1];
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WAVES; ++w) k.keeps += f.above[w];
  k.equals = f.equals;
  k.done = same == b.need;
}

// R: vectors of a thread that are kept in registers; 0: sequences that do not fit.
// STAGE: of a list in pieces, of which the workgroup has one; kWhole: it has the list.
template <int R, int WAVES, int STAGE = kWhole>
__global__ __launch_bounds__(WAVES * kWave) void kv_select_kernel(SelectArgs a) {
  static_assert(STAGE == kWhole || (R == kPieceVectors && WAVES == kManyWaves), "a piece");
  const int head = static_cast<int>(blockIdx.x), seq = static_cast<int>(blockIdx.y);
  const int piece = STAGE == kWhole ? 0 : static_cast<int>(blockIdx.z), start = piece * kPiece;
  const int tid = static_cast<int>(threadIdx.x), wave = wave_index(), lane = lane_id();
  const Source source = source_of(a, seq, head);
  Weights<R ? R : 1> own;
  if constexpr (R > 0) {  // beside the length
    uint32_t pages[R];
    look_up(source, start + wave * R * kVector, pages);
    own.load(source, pages);
  }
  int n = a.seq_lens[seq];
  n = n < 0 ? 0 : (n < a.max_seq_len ? n : a.max_seq_len);
  int32_t* kept = a.kept + (static_cast<int64_t>(seq) * a.kv_heads + head) * a.budget;
  if constexpr (STAGE == kWhole || STAGE == kLastStage) {
    if (head == 0 && piece == 0 && tid == 0) a.new_lens[seq] = n < a.budget ? n : a.budget;
    if (n <= a.budget) {
      const int step = (STAGE == kWhole ? 1 : static_cast<int>(gridDim.z)) * WAVES * kWave;
      for (int i = piece * WAVES * kWave + tid; i < a.budget; i += step) kept[i] = i < n ? i : -1;
      return;
    }
  } else if (n <= a.budget) {
    return;
  }
  if (STAGE != kWhole && start >= n) return;
  const int low = a.sinks, high = n - a.recent;  // those between are weighed
  // This wave's run.
  const int length = R ? R * kVector : (n + WAVES * kVector - 1) / (WAVES * kVector) * kVector;
  const int at = start + wave * length, begin = at < n ? at : n;
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
  Known k = {};
  if constexpr (STAGE != kWhole) {
    // digits of 11, 11 and 10 bits, as below
    constexpr int kShift[] = {21, 10, 0}, kBits[] = {11, 11, 10};
    const Pieces pieces(a, static_cast<int64_t>(seq) * a.kv_heads + head);
    if constexpr (STAGE > 1) {
      k = pieces.known[piece];
      b = {k.prefix, k.known, k.need};
    } else if (b.need == 0) {
      b.prefix = b.known = 0xFFFFFFFFu;
      k.done = 1;
    }
    if constexpr (STAGE > 0) {
      if (!k.done) join_pieces<WAVES>(f, b, k, pieces, piece, n, STAGE - 1, kShift[STAGE - 1], kBits[STAGE - 1]);
      if (STAGE < kLastStage && tid == 0)
        pieces.known[piece] = {b.prefix, b.known, b.need, k.keeps, k.equals, k.done, {0, 0}};
    }
    own.check_pages();
    own.order();
    if constexpr (STAGE < kLastStage) {
      if (k.done) return;
      clear_bins<WAVES>(f);
      all([&](int first, const u32x4& w) {
        weighed(first, w, [&](uint32_t x, bool in) {
          if (in && b.shares(x)) atomicAdd(&f.bins[x >> kShift[STAGE] & ((1u << kBits[STAGE]) - 1)], 1u);
        });
      });
      __syncthreads();
      pieces.counts_of(piece, STAGE)[tid] = f.bins[2 * tid] | f.bins[2 * tid + 1] << 16;
      return;
    }
  } else if (b.need == 0) {
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
  // In registers (vector by vector, as below, it took 2.5 of 16.4 us more and spilled
  // scalars): this lane's that are kept, and that are equal to the last one that is, as
  // bits, and how many of each vector are so in the lanes below (at most 252), as bytes.
  uint32_t kept_bits = 0, equal_bits = 0, kept_below = 0, equal_below = 0;
  uint32_t kept_of[R ? R : 1] = {}, equal_of[R ? R : 1] = {};  // of the wave's vectors
  bool some_equal = false;
  // Elsewhere, vector by vector: the lanes with a weight that is kept, and with one that is
  // equal to the last one that is, by the weight's place in the vector.
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
  if constexpr (R > 0) {
    uint32_t kept_own = 0, equal_own = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int first = begin + r * kVector, token = first + 4 * lane;
      const bool inside = first >= low && first + kVector <= high;
      uint32_t k = 0, e = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = own.w[r][i];
        k |= (w > top ? 1u : 0u) << i;
        e |= (w >= bottom ? 1u : 0u) << i;
      }
      if (!inside) {
        uint32_t in = 0, there = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          in |= (token + i >= low && token + i < high ? 1u : 0u) << i;
          there |= (token + i < n ? 1u : 0u) << i;
        }
        k = (k & in) | (there & ~in);
        e = (e & in) | k;
      }
      e &= ~k;
      kept_bits |= k << (4 * r);
      equal_bits |= e << (4 * r);
      kept_own |= static_cast<uint32_t>(__popc(k)) << (8 * r);
      equal_own |= static_cast<uint32_t>(__popc(e)) << (8 * r);
    }
    kept_below = sum_below(kept_own);
    some_equal = __any(equal_own != 0);
    if (some_equal) equal_below = sum_below(equal_own);
    const uint32_t k1 = __builtin_amdgcn_readlane(kept_below, kWave - 1), k2 = __builtin_amdgcn_readlane(kept_own, kWave - 1);
    const uint32_t e1 = __builtin_amdgcn_readlane(equal_below, kWave - 1), e2 = __builtin_amdgcn_readlane(equal_own, kWave - 1);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      kept_of[r] = (k1 >> (8 * r) & 255u) + (k2 >> (8 * r) & 255u);
      equal_of[r] = (e1 >> (8 * r) & 255u) + (e2 >> (8 * r) & 255u);
      keeps += kept_of[r];
      equals += equal_of[r];
    }
  } else if (gathered) {
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
  if constexpr (STAGE != kWhole) {
    k0 += k.keeps + static_cast<uint32_t>((low < start ? low : start) + (start > high ? start - high : 0));
    e0 += k.equals;
  }
  k0 = __builtin_amdgcn_readfirstlane(k0);  // kept, and equal, before the vector
  e0 = __builtin_amdgcn_readfirstlane(e0);

  // (inside the list also where another stream writes the mass meanwhile)
  const auto put = [&](uint32_t at, int token) {
    if (at < static_cast<uint32_t>(a.budget)) kept[at] = token;
  };
  if constexpr (R > 0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int token = begin + r * kVector + 4 * lane;
      uint32_t k = k0 + (kept_below >> (8 * r) & 255u);
      if (!some_equal) {
        k += e0 < need ? e0 : need;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (kept_bits >> (4 * r + i) & 1u) put(k++, token + i);
      } else {
        uint32_t e = e0 + (equal_below >> (8 * r) & 255u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool keep = kept_bits >> (4 * r + i) & 1u, equal = equal_bits >> (4 * r + i) & 1u;
          if (keep || (equal && e < need)) put(k + (e < need ? e : need), token + i);
          k += keep ? 1u : 0u;
          e += equal ? 1u : 0u;
        }
      }
      k0 += kept_of[r];
      e0 += equal_of[r];
    }
    return;
  }
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

// Pieces of each list; 0: it is left whole.  Pieces use the compute units that a few whole
// lists leave idle, but their four launches read the weights four times, and every piece
// all histograms.  us in pieces / whole, by lists:
//   65536 tokens    8: 16 / 34    32: 21 / 35    128: 61 / 37
//   131072 tokens   8: 21 / 58    16: 22 / 59     64: 67 / 62
//   262144 tokens   8: 25 / 106                   64: 142 / 111
//   524288 tokens   8: 48 / 200   32: 161 / 206
//   1048576 tokens  1: 35 / 384    8: 123 / 390
// and 3 pieces 17 / 17 for 8 lists, 20 / 19 for 32.
static int pieces_of(int num_seqs, int kv_heads, int max_seq_len) {
  const int pieces = (max_seq_len - 1) / kPiece + 1;
  return pieces > 3 && pieces <= kMostPieces && static_cast<int64_t>(num_seqs) * kv_heads <= kMostLists ? pieces : 0;
}

int64_t kv_select_workspace_bytes(int num_seqs, int kv_heads, int max_seq_len) {
  return static_cast<int64_t>(num_seqs) * kv_heads * Pieces::words(pieces_of(num_seqs, kv_heads, max_seq_len)) *
         static_cast<int64_t>(sizeof(uint32_t));
}

hipError_t launch_kv_select(const float* mass, int num_pages, int page_shift, const int32_t* seq_lens,
                            const int32_t* page_table, int64_t ld_table, int num_seqs, int kv_heads,
                            int max_seq_len, int sinks, int recent, int32_t* kept, int budget,
                            int32_t* new_lens, void* workspace, hipStream_t stream) {
  const SelectArgs a = {mass, seq_lens, page_table, ld_table, kept, new_lens, num_pages, page_shift,
                        kv_heads, max_seq_len, sinks, recent, budget, static_cast<uint32_t*>(workspace)};
  const dim3 grid(kv_heads, num_seqs), few(kFewWaves * kWave), many(kManyWaves * kWave);
  if (const int pieces = pieces_of(num_seqs, kv_heads, max_seq_len)) {
    const dim3 parts(kv_heads, num_seqs, pieces);
    hipLaunchKernelGGL((kv_select_kernel<kPieceVectors, kManyWaves, 0>), parts, many, 0, stream, a);
    hipLaunchKernelGGL((kv_select_kernel<kPieceVectors, kManyWaves, 1>), parts, many, 0, stream, a);
    hipLaunchKernelGGL((kv_select_kernel<kPieceVectors, kManyWaves, 2>), parts, many, 0, stream, a);
    hipLaunchKernelGGL((kv_select_kernel<kPieceVectors, kManyWaves, kLastStage>), parts, many, 0, stream, a);
    return hipGetLastError();
  }
  constexpr int kFit = kFewWaves * kVector;  // tokens of a vector a thread
  if (max_seq_len <= kFit) hipLaunchKernelGGL((kv_select_kernel<1, kFewWaves>), grid, few, 0, stream, a);
  else if (max_seq_len <= 2 * kFit) hipLaunchKernelGGL((kv_select_kernel<2, kFewWaves>), grid, few, 0, stream, a);
  else if (max_seq_len <= 4 * kFit) hipLaunchKernelGGL((kv_select_kernel<4, kFewWaves>), grid, few, 0, stream, a);
  else if (max_seq_len <= 8 * kFit) hipLaunchKernelGGL((kv_select_kernel<4, kManyWaves>), grid, many, 0, stream, a);
  else hipLaunchKernelGGL((kv_select_kernel<0, kManyWaves>), grid, many, 0, stream, a);
  return hipGetLastError();
}

}  // namespace lora
