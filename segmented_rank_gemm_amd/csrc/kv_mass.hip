// lora_kv_attention_mass: how much attention each cached token drew in a step, by key
// head, from the queries, the cached keys and the logarithms of the rows' sums that
// attention left:
//   drawn[t] = sum over the rows that see t of exp(scale * q . k_t - lse)
// added to what earlier steps left for the tokens before the queries, and put in the
// place of whatever was there for the queries' own.
//
// The scores are 16x16 matrix products with the rows on one side (A) and tokens on the
// other (B): column c of the j-th of a chunk's four products is token 4 c + j, so that
// lane (g, c) (lane = 16 g + c) gets, for the rows [4 g, 4 g + 4), the scores of four
// neighbouring tokens.  It adds up its rows, tile after tile, in four registers; the
// four lanes that share the tokens are joined once, at the end.  Every token has one
// writer, and its sum is always taken in the same order.
//
// Few rows: a wave walks chunks of 64 tokens of a key head, the next ones' keys on
// their way, with the rows in shared memory.  Many: a wave keeps the keys of one chunk
// in registers, and the rows come by.
//
// Bound by: HBM with one tile of rows (64 sequences of up to 8192 tokens, 8 key heads of
// 128: 39.5 us, 4.1 TB/s where a copy reaches 5.0 to 5.5); with many rows by the
// instructions that the units take in turn (8 sequences in pieces of 129 to 512 queries, 8
// key heads of 8: 157 us, 780 TFLOP/s; vector instructions 51% of the cycles, of which the
// exponentials, their arguments and sums are 48 of 89 a tile and chunk, the matrix unit
// 31%).  For heads of 128 that kernel keeps 17 registers (27 with masks) in scratch memory,
// stored at its start and read again once a chunk, not in the loop over the rows: 47 MB of
// writes where its output is 1 MB.

#include "kv_attention.hpp"

namespace lora {

constexpr int kMassWaves = 8;
constexpr int kMassThreads = kMassWaves * kWave;
// Tiles of 16 rows, at most, for the kernel of few: as many as two workgroups a compute
// unit have room for in shared memory, beside a tree's masks (us, this kernel / that of
// many: 16 sequences of 4096 tokens, 8 key heads: 32 rows 15 / 64, 128 rows 28 / 81, 256
// rows 46 / 97; one of 32768: 128 rows 18 / 36).
__host__ __device__ constexpr int few_tiles(int V) { return V == kTree ? 14 : 16; }
constexpr int kShares = 4;         // of the rows, for that of many: waves that share a chunk
constexpr float kLog2e = 1.44269504f;

struct MassArgs {
  SumArgs a;
  float* mass;
  float scale_log2;  // scale * log2(e), with its sign
  uint32_t inverse;  // ceil(2^32 / group): the high half of a product with a row below 2^22 is its query
};

__device__ __forceinline__ int query_of(const MassArgs& m, int row) {
  return static_cast<int>(m.a.group == 1 ? static_cast<uint32_t>(row) : __umulhi(static_cast<uint32_t>(row), m.inverse));
}

// A row's sum as the power that its scores are taken relative to; a row without a sum
// counts for nothing, whatever its query holds.
__device__ __forceinline__ float relative_to(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }
// Of a row that is not there and has a query of zeros: its powers are zero.
constexpr float kNoRow = 3.402823466e38f;

// What the rows [4 g, 4 g + 4) of a tile see (seen_by_rows), without those that count for
// nothing: a NaN score less their infinity would be NaN.
__device__ __forceinline__ uint32_t unless_silent(uint32_t seen, f32x4 top) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (top[i] == INFINITY) seen &= ~(15u << (4 * i));
  return seen;
}

// Sums over the four lanes with the same c.
__device__ __forceinline__ float over_groups(float v) {
  const uint32_t a = __float_as_uint(v);
  const auto rows = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  const uint32_t b = __float_as_uint(__uint_as_float(rows[0]) + __uint_as_float(rows[1]));
  const auto halves = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return __uint_as_float(halves[0]) + __uint_as_float(halves[1]);
}

// The chunk's tokens that the rows [4 g, 4 g + 4) of a tile see: bit 4 i + j for row i and
// token 4 c + j.  Row 0 of the tile is head head0 of query query0; past `rows`, none.
template <int V>
__device__ __forceinline__ uint32_t seen_by_rows(const AttentionArgs& a, const RowTile& t, const Draft* drafts,
                                                 int base, int query0, int head0, int rows) {
  const int lane = lane_id(), g = lane >> 4;
  const int token = base + 4 * (lane & 15);
  uint32_t seen = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 4 * g + i;
    const int query = row_of(a, query0, head0, row).query;
    uint32_t bits;
    if constexpr (V == kTree) {
      const Draft& d = drafts[row < rows ? query : 0];
      const int o = token - t.before;
      bits = bits_between(token, 0, t.before);
      if (o > -4) {
        const int w = o >> 5, shift = o & 31;
        const uint32_t m0 = w >= 0 && w < 2 * kDraftWords ? d.mask[w] : 0u;
        const uint32_t m1 = w >= -1 && w + 1 < 2 * kDraftWords ? d.mask[w + 1] : 0u;
        bits |= static_cast<uint32_t>((static_cast<unsigned long long>(m1) << 32 | m0) >> shift);
      }
      bits &= bits_between(token, d.from, token + 4);
    } else {
      const int place = t.before + query;
      bits = bits_between(token, a.window ? place - a.window + 1 : 0, place + 1);
    }
    seen |= (row < rows ? bits & 15u : 0u) << (4 * i);
  }
  return seen;
}

// exp(scores - sums) of one tile and chunk, s[j][i] of row 4 g + i and token 4 c + j,
// added up over the rows.
__device__ __forceinline__ void add_rows(f32x4& sums, const f32x4 (&s)[4], f32x4 top, float scale_log2) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __builtin_amdgcn_exp2f(fmaf(s[j][i], scale_log2, -top[i]));
    sums[j] += (p[0] + p[1]) + (p[2] + p[3]);
  }
}
__device__ __forceinline__ void add_seen_rows(f32x4& sums, const f32x4 (&s)[4], f32x4 top, float scale_log2,
                                              uint32_t seen) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = __builtin_amdgcn_exp2f(fmaf(s[j][i], scale_log2, -top[i]));
      if (!(seen >> (4 * i + j) & 1u)) p[i] = 0.f;
    }
    sums[j] += (p[0] + p[1]) + (p[2] + p[3]);
  }
}

// Where lane (g, c) finds its part of the keys, and the mass of token 4 c + g, of a chunk.
template <int D>
struct MassReader {
  Reader<D> keys;
  float* mass;          // of page 0
  int64_t mass_stride;  // from one page to the next

  __device__ __forceinline__ int page(int base) const { return keys.page_at(base + 16 * ((lane_id() & 15) >> 2)); }
  __device__ __forceinline__ void load(Keys<D>& k, int page, int base) const { keys.load(k, Pages{page, page}, base); }
  // (of page 0 where there is none: it is not written)
  __device__ __forceinline__ float* at(int page, int base) const {
    const int lane = lane_id();
    const int in = (base + 4 * (lane & 15) + (lane >> 4)) & ((1 << keys.shift) - 1);
    return mass + (page < 0 ? 0 : page) * mass_stride + in;
  }
};
template <int D>
__device__ __forceinline__ MassReader<D> mass_reader_of(const MassArgs& m, int seq, int kv_head) {
  const int shift = m.a.cache.page_shift;
  return MassReader<D>{reader_of<D>(m.a, seq, kv_head), m.mass + (static_cast<int64_t>(kv_head) << shift),
                       static_cast<int64_t>(m.a.cache.kv_heads) << shift};
}

// Of a lane's joined sums, that of token 4 c + g.
__device__ __forceinline__ float of_group(const f32x4 sums) {
  const int g = lane_id() >> 4;
  const float s0 = sums[0], s1 = sums[1], s2 = sums[2], s3 = sums[3];
  const float low = g & 1 ? s1 : s0, high = g & 1 ? s3 : s2;
  return g & 2 ? high : low;
}

// One tile of rows (T = 1), or up to T.
template <int D, int V, int T>
__global__ __launch_bounds__(kMassThreads, 4) void kv_mass_kernel(MassArgs m) {
  constexpr int kSteps = D / 32;
  const SumArgs& a = m.a;
  const int wave = wave_index(), lane = lane_id(), g = lane >> 4, c = lane & 15;
  const int kv_head = static_cast<int>(blockIdx.x);
  const int seq = sequence_at(a, static_cast<int>(blockIdx.z));
  const MassReader<D> reader = mass_reader_of<D>(m, seq, kv_head);
  const int step = kMassWaves * static_cast<int>(gridDim.y);
  int chunk = static_cast<int>(blockIdx.y) * kMassWaves + wave;
  int first_page = -1;
  if (!a.window) first_page = reader.page(chunk * kChunk);  // beside the lengths
  RowTile t;
  if (!tile_of<V>(a, seq, 0, t, true)) return;
  const int length = t.before + t.queries;
  const int end = (length + kChunk - 1) / kChunk;
  chunk += t.chunk0;
  if (t.chunk0 + static_cast<int>(blockIdx.y) * kMassWaves >= end) return;  // the whole workgroup
  if (a.window) first_page = reader.page(chunk * kChunk);

  // What a wave has on its way, with one tile: two chunks' keys, and the mass of their
  // tokens; with several, whose products take longer, the next chunk's page.  (Loads
  // without conditions: past the last chunk the last one's once more.)
  struct Ahead {
    Keys<D> keys;
    float mass;
    int page;
  };
  const auto base_of = [&](int at) { return (at < end ? at : end - 1) * kChunk; };
  const auto fetch = [&](Ahead& x, int page, int at) {
    x.page = page;
    reader.load(x.keys, page, base_of(at));
    x.mass = *reader.at(page, base_of(at));
  };
  Ahead ahead[2];
  int pages[2];  // of the chunks after those
  fetch(ahead[0], first_page, chunk);
  if constexpr (T == 1) {
    fetch(ahead[1], reader.page(base_of(chunk + step)), chunk + step);
    pages[0] = reader.page(base_of(chunk + 2 * step));
    pages[1] = reader.page(base_of(chunk + 3 * step));
  } else {
    pages[0] = reader.page(base_of(chunk + step));
  }

  const int tiles = (t.rows + kTile - 1) / kTile;
  __shared__ u32x4 q[T * kSteps][kWave];
  __shared__ f32x4 tops[T * 4];
  __shared__ unsigned long long silent[kMassWaves];  // rows that count for nothing
  __shared__ Draft drafts[V == kTree ? T * kTile : 1];
  for (int f = wave; f < tiles * kSteps; f += kMassWaves) {
    const int row = (f / kSteps) * kTile + c;
    u32x4 w = {0, 0, 0, 0};
    if (row < t.rows) {
      const RowOf at = row_of(a, 0, 0, row);
      w = load16(a.q + static_cast<int64_t>(t.start + at.query) * a.ldq + (kv_head * a.group + at.head) * D +
                 g * (D / 4) + 8 * (f % kSteps));
    }
    q[f][lane] = w;
  }
  static_assert(T * kTile <= kMassThreads, "a row a thread");
  {
    const int row = static_cast<int>(threadIdx.x);
    float top = kNoRow;
    if (row < t.rows) {
      const RowOf at = row_of(a, 0, 0, row);
      top = relative_to(a.lse[static_cast<int64_t>(t.start + at.query) * a.ldl + kv_head * a.group + at.head]);
    }
    if (row < T * kTile) reinterpret_cast<float*>(tops)[row] = top;
    const unsigned long long out = __ballot(top == INFINITY);
    if (lane == 0) silent[wave] = out;
  }
  if constexpr (V == kTree) stage_drafts(a, t, drafts, tiles * kTile, kMassThreads);
  __syncthreads();
  // bit n: of tile n, some row counts for nothing
  const unsigned long long silent_tiles =
      __ballot(lane < T && reinterpret_cast<const uint16_t*>(silent)[lane < T ? lane : 0] != 0);

  // Adds up one tile's rows.
  const auto add = [&](f32x4& sums, const f32x4 (&s)[4], int base, bool masked, int n) {
    const f32x4 top = tops[4 * n + g];
    if (masked || (silent_tiles >> n & 1)) {
      const int query0 = n * kTile / a.group;
      const uint32_t seen =
          seen_by_rows<V>(a, t, drafts, base, query0, n * kTile - query0 * a.group, t.rows - n * kTile);
      add_seen_rows(sums, s, top, m.scale_log2, unless_silent(seen, top));
    } else {
      add_rows(sums, s, top, m.scale_log2);
    }
  };
  const auto store = [&](f32x4& sums, int base, int page, float before) {
#pragma unroll
    for (int j = 0; j < 4; ++j) sums[j] = over_groups(sums[j]);
    const float drawn = of_group(sums);
    const int token = base + 4 * c + g;
    if (token < length && page >= 0) *reader.at(page, base) = token >= t.before ? drawn : before + drawn;
  };
  const auto key = [&](const Keys<D>& keys, int i, int j) {
    return __builtin_bit_cast(bf16x8, word_to_bf16(keys.w[j][i], __uint_as_float(byte_scale(keys.scales, j))));
  };
  if constexpr (T == 1) {
    const auto take = [&](Ahead& x, int& next_page) {
      const int base = chunk * kChunk, page = x.page;
      const float before = x.mass;
      f32x4 s[4];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const bf16x8 rows = __builtin_bit_cast(bf16x8, q[i][lane]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[j] = mfma(rows, key(x.keys, i, j), i == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : s[j]);
      }
      fetch(x, next_page, chunk + 2 * step);
      next_page = reader.page(base_of(chunk + 4 * step));
      f32x4 sums = {0.f, 0.f, 0.f, 0.f};
      add(sums, s, base, base < t.all_first || base + kChunk > t.all_last, 0);
      store(sums, base, page, before);
      chunk += step;
    };
    while (chunk < end) {
      take(ahead[0], pages[0]);
      if (chunk >= end) break;
      take(ahead[1], pages[1]);
    }
  } else {
    for (; chunk < end; chunk += step) {
      const int base = chunk * kChunk, page = ahead[0].page;
      const float before = ahead[0].mass;
      bf16x8 k[4][kSteps];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < kSteps; ++i) k[j][i] = key(ahead[0].keys, i, j);
      f32x4 sums = {0.f, 0.f, 0.f, 0.f};
      const bool masked = base < t.all_first || base + kChunk > t.all_last;
#pragma unroll 1
      for (int n = 0; n < tiles; ++n) {
        f32x4 s[4];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const bf16x8 rows = __builtin_bit_cast(bf16x8, q[n * kSteps + i][lane]);
#pragma unroll
          for (int j = 0; j < 4; ++j) s[j] = mfma(rows, k[j][i], i == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : s[j]);
        }
        add(sums, s, base, masked, n);
      }
      store(sums, base, page, before);
      fetch(ahead[0], pages[0], chunk + step);
      pages[0] = reader.page(base_of(chunk + 2 * step));
    }
  }
}

// Any number of rows: a workgroup has two chunks, each wave the keys of one of them, and
// the four waves of a chunk share the rows, a tile of 16 of a step's 64 each.  Tiles come
// by in shared memory, staged as the matrix unit's operands, in two buffers of a step.
template <int D, int V>
__global__ __launch_bounds__(kMassThreads, 4) void kv_mass_rows_kernel(MassArgs m) {
  constexpr int kSteps = D / 32;
  constexpr int kChunks = kMassWaves / kShares;  // of a workgroup
  constexpr int kStageRows = kShares * kTile;      // a tile for each
  const SumArgs& a = m.a;
  const int wave = wave_index(), lane = lane_id(), g = lane >> 4, c = lane & 15;
  const int share = wave / kChunks;
  const int kv_head = static_cast<int>(blockIdx.x);
  const int seq = sequence_at(a, static_cast<int>(blockIdx.z));
  RowTile t;
  if (!tile_of<V>(a, seq, 0, t, true)) return;
  const int length = t.before + t.queries;
  const int end = (length + kChunk - 1) / kChunk;
  const MassReader<D> reader = mass_reader_of<D>(m, seq, kv_head);

  __shared__ u32x4 q[2][kShares][kSteps][kWave];
  __shared__ float tops[2][kStageRows];
  __shared__ float joined[kMassWaves][kWave];
  __shared__ int again;  // chunks that have to be done once more
  __shared__ Draft drafts[V == kTree ? 64 * kDraftWords : 1];
  if constexpr (V == kTree) stage_drafts(a, t, drafts, t.query1 + 1, kMassThreads);  // (a barrier comes below)

  // Where a sum comes out as NaN, the chunks are done once more with care: it may be of a
  // row that counts for nothing, whose infinity leaves a NaN score NaN.  Its query and
  // such keys are then staged as finite ones.  (A look for such rows at every tile cost
  // registers: 8 sequences in pieces 157 -> 161 us, 16 trees of 32 drafts behind 4096
  // tokens 118 -> 138; this 158 and 120.)
  bool careful = false;
  if (threadIdx.x == 0) again = -1;
  for (int first = t.chunk0 + static_cast<int>(blockIdx.y) * kChunks; first < end;) {
    const int chunk = first + wave % kChunks, base = chunk * kChunk;
    const bool mine = chunk < end;
    const int loaded = mine ? base : (end - 1) * kChunk;
    const int page = reader.page(loaded);
    Keys<D> keys;
    reader.load(keys, page, loaded);
    if (careful) {
      // (rows that see such a key, and count, have NaN for their sum)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (((keys.scales >> (8 * j)) & 255u) == kScaleNan) keys.scales &= ~(255u << (8 * j));
    }

    // The rows that see some of these chunks; tiles are counted from the first of them on.
    int from = 0, to = t.rows;
    if constexpr (V != kTree) {
      const int q0 = first * kChunk - t.before;  // the first query that sees their first token
      from = q0 > t.query1 ? t.rows : (q0 > 0 ? q0 * a.group : 0);
      if (a.window) {
        const int64_t q1 = static_cast<int64_t>(first + kChunks) * kChunk - 1 + a.window - t.before;  // past the last
        to = q1 <= 0 ? 0 : (q1 * a.group < to ? static_cast<int>(q1 * a.group) : to);
      }
    }
    // Steps of kStageRows rows, of whose operands each wave brings kLoads, and the first
    // one the sums: by registers, since the compiler lets no read of shared memory pass a
    // load into it.  (Past the last step the last row's once more, which nobody reads.)
    constexpr int kLoads = kShares * kSteps / kMassWaves;
    u32x4 part[kLoads];
    float lse = 0.f;
    // Where a step is a whole number of queries, its rows lie as far behind those of the
    // step before as these do; elsewhere, and where rows are missing, they are looked for.
    const bool whole = kStageRows % a.group == 0;
    const int64_t queries = kStageRows / a.group;  // (for that case)
    const uint16_t* at_row[kLoads];
    const float* at_lse = a.lse;
    const auto ask = [&](int row0) {
      if (whole && row0 > from && row0 + kStageRows <= t.rows) {
#pragma unroll
        for (int f = 0; f < kLoads; ++f) at_row[f] += queries * a.ldq;
        at_lse += queries * a.ldl;
      } else {
        const int first_row = row0 < t.rows ? row0 : t.rows - 1, left = t.rows - 1 - first_row;
        const int query0 = query_of(m, first_row), head0 = first_row - query0 * a.group;
#pragma unroll
        for (int f = 0; f < kLoads; ++f) {
          const int at = f * kMassWaves + wave, row = at / kSteps * kTile + c;
          const RowOf of = row_of(a, query0, head0, row < left ? row : left);
          at_row[f] = a.q + static_cast<int64_t>(t.start + of.query) * a.ldq + (kv_head * a.group + of.head) * D +
                      g * (D / 4) + 8 * (at % kSteps);
        }
        const RowOf of = row_of(a, query0, head0, lane < left ? lane : left);
        at_lse = a.lse + static_cast<int64_t>(t.start + of.query) * a.ldl + kv_head * a.group + of.head;
      }
#pragma unroll
      for (int f = 0; f < kLoads; ++f) part[f] = load16(at_row[f]);
      if (wave == 0) lse = *at_lse;
    };
    const auto put = [&](int buffer, int row0) {
#pragma unroll
      for (int f = 0; f < kLoads; ++f) {
        const int at = f * kMassWaves + wave;
        u32x4 w = part[f];
        if (careful) {
          const int row = row0 + at / kSteps * kTile + c, of = row < t.rows ? row : t.rows - 1;
          const int query = query_of(m, of), head = of - query * a.group;
          if (a.lse[static_cast<int64_t>(t.start + query) * a.ldl + kv_head * a.group + head] == -INFINITY)
            w = u32x4{0, 0, 0, 0};
        }
        q[buffer][at / kSteps][at % kSteps][lane] = w;
      }
      if (wave == 0 && lane < kStageRows) tops[buffer][lane] = row0 + lane < to ? relative_to(lse) : INFINITY;
    };
    int row0 = from;
    ask(row0);
    put(0, row0);
    ask(row0 + kStageRows);
    bf16x8 k[4][kSteps];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        k[j][i] = __builtin_bit_cast(bf16x8, word_to_bf16(keys.w[j][i], __uint_as_float(byte_scale(keys.scales, j))));
    f32x4 sums = {0.f, 0.f, 0.f, 0.f};
    for (int buffer = 0; row0 < to; row0 += kStageRows, buffer ^= 1) {
      __syncthreads();  // this step's tiles are there, and the other buffer has been read
      put(buffer ^ 1, row0 + kStageRows);
      ask(row0 + 2 * kStageRows);
      const int tile0 = row0 + share * kTile;
      if (!mine || tile0 >= to) continue;
      f32x4 s[4];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const bf16x8 rows = __builtin_bit_cast(bf16x8, q[buffer][share][i][lane]);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = mfma(rows, k[j][i], i == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : s[j]);
      }
      const f32x4 top = *reinterpret_cast<const f32x4*>(&tops[buffer][share * kTile + 4 * g]);
      const int query0 = query_of(m, tile0), last = query_of(m, tile0 + kTile - 1);
      bool masked;
      if constexpr (V == kTree) masked = base < t.all_first || base + kChunk > t.all_last;
      else masked = base + kChunk > t.before + query0 + 1 || (a.window && base <= t.before + last - a.window);
      if (masked) {
        // (not known to be the same each time: what follows from it takes no registers
        // through the loop)
        int here = base;
        asm volatile("" : "+s"(here));
        add_seen_rows(sums, s, top, m.scale_log2,
                      seen_by_rows<V>(a, t, drafts, here, query0, tile0 - query0 * a.group, to - tile0));
      } else {
        add_rows(sums, s, top, m.scale_log2);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) sums[j] = over_groups(sums[j]);
    const float drawn = of_group(sums);
    joined[wave][lane] = drawn;
    if (!careful && __any(drawn != drawn)) again = first;  // (a sum of rows, so a barrier came before)
    __syncthreads();
    careful = !careful && again == first;
    if (careful) continue;
    const int token = base + 4 * c + g;
    if (share == 0 && mine && token < length && page >= 0) {
      float* at = reader.at(page, base);
      float all = drawn;
#pragma unroll
      for (int n = 1; n < kShares; ++n) all += joined[n * kChunks + wave][lane];
      *at = token >= t.before ? all : *at + all;
    }
    __syncthreads();  // the sums have been read
    first += kChunks * static_cast<int>(gridDim.y);
  }
}

template <int D, int V>
static void launch_mass(const MassArgs& m, int num_seqs, hipStream_t stream) {
  const int heads = m.a.cache.kv_heads;
  const int64_t rows = static_cast<int64_t>(m.a.max_query_len) * m.a.group;
  const int64_t units = static_cast<int64_t>(num_seqs) * heads;
  // tokens that a sequence's rows see, and its own
  int64_t longest = m.a.max_seq_len;
  if (m.a.window) {
    const int64_t seen = static_cast<int64_t>(m.a.window) + m.a.max_query_len + kChunk;
    longest = longest < seen ? longest : seen;
  }
  const int64_t chunks = (longest + kChunk - 1) / kChunk;
  const bool few = rows <= few_tiles(V) * kTile;
  // Of few rows as many workgroups as the device holds (64 sequences of up to 8192 tokens:
  // 40 us, with twice as many 46), of many, whose work differs in the rows as well, several
  // times that.
  const int64_t most = few ? (chunks + kMassWaves - 1) / kMassWaves : (chunks * kShares + kMassWaves - 1) / kMassWaves;
  int64_t groups = ((few ? 2 : 16) * kCus + units - 1) / units;
  groups = groups < most ? groups : most;
  const dim3 grid(heads, static_cast<unsigned>(groups), num_seqs), block(kMassThreads);
  if (rows <= kTile) hipLaunchKernelGGL((kv_mass_kernel<D, V, 1>), grid, block, 0, stream, m);
  else if (few) hipLaunchKernelGGL((kv_mass_kernel<D, V, few_tiles(V)>), grid, block, 0, stream, m);
  else hipLaunchKernelGGL((kv_mass_rows_kernel<D, V>), grid, block, 0, stream, m);
}

hipError_t launch_kv_attention_mass(const uint16_t* q, int64_t ldq, const float* lse, int64_t ldl,
                                    const int32_t* query_start, const int32_t* seq_lens,
                                    const int32_t* page_table, int64_t ld_table, const uint8_t* cache,
                                    int num_pages, int page_shift, int num_tokens, int num_seqs,
                                    int max_query_len, int max_seq_len, int q_heads, int kv_heads,
                                    int head_dim, float scale, int window, const int64_t* masks,
                                    int64_t words, float* mass, hipStream_t stream) {
  const int group = q_heads / kv_heads;
  if (window >= max_seq_len) window = 0;
  MassArgs m;
  m.a = SumArgs{{q, query_start, seq_lens, page_table, nullptr,
                 {cache, num_pages, page_shift, kv_heads},
                 ldq, 0, ld_table, num_tokens, max_query_len, max_seq_len, q_heads, window,
                 0.f, 0u, group, ((1 << 21) + group - 1) / group,
                 1, 1, 0, 0, nullptr, nullptr},
                masks, words, const_cast<float*>(lse), ldl};
  m.mass = mass;
  m.inverse = static_cast<uint32_t>(((1ull << 32) + group - 1) / group);
  m.scale_log2 = fminf(fmaxf(scale * kLog2e, -3.402823466e38f), 3.402823466e38f);
  if (masks) {
    if (head_dim == 64) launch_mass<64, kTree>(m, num_seqs, stream);
    else launch_mass<128, kTree>(m, num_seqs, stream);
  } else {
    if (head_dim == 64) launch_mass<64, kPlain>(m, num_seqs, stream);
    else launch_mass<128, kPlain>(m, num_seqs, stream);
  }
  return hipGetLastError();
}

}  // namespace lora
