// lora_kv_attention: softmax(scale q K^T) V of each sequence's queries over its
// cached keys and values, read from the 4-bit paged cache.
//
// The rows that share a key head (a sequence's queries times its query heads a
// key head) are the columns of 16x16 matrix products, tokens their rows:
//   S^T[t][row] = sum_e K[t][e] q[row][e]          (A: keys, B: queries)
//   O^T[e][row] = sum_t V[t][e] P[row][t]          (A: values, B: weights)
// A wave walks the tokens in chunks of 64.  All three index orders of a product
// are free as long as both operands agree, and are chosen so that nothing has
// to move between lanes:
//   - row r of the j-th of a chunk's four S tiles is token 4 r + j, so that lane
//     (g, c) of the result (lane = 16 g + c) holds the 16 scores of the tokens
//     [16 g, 16 g + 16) for row c: after the softmax just the B operand that the
//     second product wants of it;
//   - the A operand of the second product is then read as 16 tokens by D / 16
//     neighbouring elements a lane, element m of each lane making up the m-th
//     product, so lane (g, c) ends up with D / 4 neighbouring outputs of row c.
// Codes become bf16 with their scale in one conversion for two (exact: 4 bits
// times a power of two).  Scores, maxima, sums and outputs are fp32; the weights
// are rounded to bf16 for the second product, as the matrix unit takes them, and it
// is the rounded ones that are summed: what the values are divided by is what they
// were multiplied by, so that equal values come back as they are (sums of the
// unrounded ones were off by up to 2^-8 of the result where few tokens are seen; 282
// against 293 us for prompts in pieces, the same for single queries).
//
// Bound by: HBM (136 bytes a token and key head at D = 128) as long as the rows of
// a key head fit one tile (4.8 TB/s at 64 sequences of up to 8192 tokens, where this
// library's copy reaches 5.5); for prompts by the vector unit beside the matrix unit,
// which one wave uses in turn (1015 TFLOP/s at 8 sequences of 2048 queries over 8192
// tokens, where a library product reaches 1335; for prompts in pieces vector
// instructions take 55% of the cycles, the matrix unit 33%, shared memory 27%).
//
// lora_kv_tree_attention is the same kernels with another view of the tokens: causal with
// the rows' sums (kSums), or what masks of drafts say (kTree).  A tree's drafts lie in the
// last chunks alone; elsewhere a row sees all of a chunk, and the walk is the plain one.
// With 256 to 512 rows a key head it is bound like prompts (16 sequences of up to 4096
// tokens and 32 drafts, 64 query heads on 8: 67 us, vector instructions 59% and the matrix
// unit 21% of the cycles, and at the end the longest sequences' workgroups alone: 1.6 of 2
// waves a SIMD; 64 drafts of 32768 tokens: 95 us and 5 for the join, 65% and 27%); with few
// rows by latency (26 drafts behind 500 tokens: 10 us and 2 for the masks).  Sums without
// masks beside plain attention, us: 64 single queries to 8192 tokens 65 / 64, one of 131072
// 40 / 38, pieces of prompts 316 / 292.

#include <type_traits>

#include "kv_attention.hpp"

namespace lora {

// Waves that share out the tokens of a tile of mt * 16 rows.  Two workgroups fit
// a compute unit: four waves a SIMD at 128 registers, or two at 256.
__host__ __device__ constexpr int split_waves(int mt) { return mt == 1 ? 8 : 4; }
// Many rows: waves of a workgroup, and 16-row tiles of a wave.
constexpr int kRowWaves = 4;
constexpr int kRowTiles = 2;
constexpr int kManyRows = 128;
constexpr float kNoScore = -3.402823466e38f;  // the running maximum before any score
// The running maximum moves only when a score passes it by this many powers of
// two; weights up to 2^8 lose nothing in fp32 sums or bf16 mantissas.
constexpr float kMaxLag = 8.f;

// The rows of one wave: MT tiles of 16.
template <int D, int MT, int V>
struct Rows {
  f32x4 acc[MT][D / 16];
  float top[MT], sum[MT];
  int place[MT];  // of row c of the tile: the last token that it sees
};
// Where sums of exponentials are asked for, those of the unrounded ones too: the
// logarithm of the rounded ones' would be off by up to 2^-8.
template <int D, int MT>
struct SumRows {
  f32x4 acc[MT][D / 16];
  float top[MT], sum[MT], full[MT];
  int place[MT];
};
template <int D, int MT>
struct Rows<D, MT, kSums> : SumRows<D, MT> {};
template <int D, int MT>
struct Rows<D, MT, kTree> : SumRows<D, MT> {
  const Draft* drafts[MT];  // of row c of the tile: what it sees
  int before;
};

template <int D, int MT, int V>
__device__ __forceinline__ uint32_t seen_by(const Rows<D, MT, V>& r, int mt, const Span& at) {
  if constexpr (V == kTree) return seen_bits(at, *r.drafts[mt], r.before);
  else return seen_bits(at, r.place[mt]);
}

// The first half of the running softmax over one chunk's scores of row tile mt,
// s[j][i] of token 16 g + 4 i + j: hides what a row does not see and moves the
// running maximum.
template <int D, int MT, int V>
__device__ __forceinline__ void raise(Rows<D, MT, V>& r, int mt, f32x4 (&s)[4], const Span& at,
                                      float scale_log2) {
  if (at.masked) {
    const uint32_t seen = seen_by(r, mt, at);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!(seen >> (4 * i + j) & 1u)) s[j][i] = -INFINITY;
  }
  float m = s[0][0];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, s[j][i]);
  m *= scale_log2;
  if (__any(m > r.top[mt] + kMaxLag)) {
    m = fmaxf(m, __shfl_xor(m, 16));
    m = fmaxf(m, __shfl_xor(m, 32));
    const float now = fmaxf(r.top[mt], m);
    const float shrink = __builtin_amdgcn_exp2f(r.top[mt] - now);
    r.top[mt] = now;
    r.sum[mt] *= shrink;
    if constexpr (V != kPlain) r.full[mt] *= shrink;
#pragma unroll
    for (int n = 0; n < D / 16; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) r.acc[mt][n][i] *= shrink;
  }
}

// The second half, a quarter of it: the weights of the tokens 16 g + 4 i + j, in
// bf16 (pairs of tokens 16 g + 2 i, + 1), and the sum of what they were rounded to.
template <int D, int MT, int V>
__device__ __forceinline__ void powers(uint32_t (&weights)[8], Rows<D, MT, V>& r, int mt,
                                       const f32x4 (&s)[4], int i, float scale_log2) {
  float p[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = __builtin_amdgcn_exp2f(fmaf(s[j][i], scale_log2, -r.top[mt]));
  const uint32_t a = pack_bf16x2(p[0], p[1]), b = pack_bf16x2(p[2], p[3]);
  r.sum[mt] += (bf16_lo(a) + bf16_hi(a)) + (bf16_lo(b) + bf16_hi(b));
  if constexpr (V != kPlain) r.full[mt] += (p[0] + p[1]) + (p[2] + p[3]);
  weights[2 * i] = a;
  weights[2 * i + 1] = b;
}

// Scores of one chunk and their weights.  q: the operand [mt][D / 32][lane] in
// shared memory.
template <int D, int MT, int V>
__device__ __forceinline__ void weigh(Rows<D, MT, V>& r, uint32_t (&weights)[MT][8], const Keys<D>& k,
                                      const u32x4* q, const Span& at, float scale_log2) {
  f32x4 s[MT][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[mt][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    bf16x8 b[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
      b[mt] = __builtin_bit_cast(bf16x8, q[(mt * (D / 32) + i) * kWave + lane_id()]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u32x4 w = word_to_bf16(k.w[j][i], __uint_as_float(byte_scale(k.scales, j)));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) s[mt][j] = mfma(__builtin_bit_cast(bf16x8, w), b[mt], s[mt][j]);
    }
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    raise(r, mt, s[mt], at, scale_log2);
#pragma unroll
    for (int i = 0; i < 4; ++i) powers(weights[mt], r, mt, s[mt], i, scale_log2);
  }
}

// Bits `nan` of this lane's 16 tokens: value blocks that held a NaN and were
// taken out.  Marks the outputs that they reach: those for which the sum over
// these tokens of "seen" is not zero.
template <int D, int MT, int V>
__device__ __forceinline__ void mark_nan(Rows<D, MT, V>& r, uint32_t nan, const Span& at) {
  if (!__any(nan != 0)) return;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const uint32_t seen = seen_by(r, mt, at);
    f32x4 hit = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4 a, b;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = 8 * h + 2 * i;
        a[i] = (nan >> k & 1u ? 0x3F80u : 0u) | (nan >> (k + 1) & 1u ? 0x3F800000u : 0u);
        b[i] = (seen >> k & 1u ? 0x3F80u : 0u) | (seen >> (k + 1) & 1u ? 0x3F800000u : 0u);
      }
      hit = mfma(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), hit);
    }
    // the D / 16 elements of lane c's tokens share a block, so `hit` serves them all
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float add = hit[i] > 0.f ? NAN : 0.f;
#pragma unroll
      for (int n = 0; n < D / 16; ++n) r.acc[mt][n][i] += add;
    }
  }
}

// Values that no row sees may be anything: their weights are zero, and their
// scales are made so.  A NaN block that some rows see and others do not is
// taken out too (mark_nan).
template <int D, int MT, int V>
__device__ __forceinline__ void mask_values(Rows<D, MT, V>& r, u32x4& scales, const Span& at) {
  uint32_t nan = 0;
  const int token = at.base + 16 * (lane_id() >> 4);
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const uint32_t byte = 255u << (8 * (k & 3));
    const bool none = !at.ok || token + k >= at.last || token + k < at.first;
    const bool bad = at.several && (scales[k >> 2] & byte) == byte;
    if (bad && !none) nan |= 1u << k;
    if (bad || none) scales[k >> 2] &= ~byte;
  }
  mark_nan(r, nan, at);
}

// The weighted values of one chunk.
template <int D, int MT, int V>
__device__ __forceinline__ void add_values(Rows<D, MT, V>& r, const uint32_t (&weights)[MT][8],
                                           const Values& v, const u32x4 scales) {
  // D / 32 elements of the lane at a time: their operands are D / 8 registers
  constexpr int kPairs = D / 64;  // words of two elements
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if constexpr (MT == 1) __builtin_amdgcn_sched_barrier(0);
      uint32_t vt[2 * kPairs][4];  // [element][pair of tokens]
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = 8 * h + 2 * i;
        const float sa = __uint_as_float(byte_scale(scales[k >> 2], k & 3));
        const float sb = __uint_as_float(byte_scale(scales[k >> 2], (k + 1) & 3));
        uint32_t a[2], b[2];
        if (half == 0) {
          a[0] = codes_to_bf16<0>(v.w[k], sa);
          b[0] = codes_to_bf16<0>(v.w[k + 1], sb);
          if constexpr (kPairs == 2) {
            a[1] = codes_to_bf16<1>(v.w[k], sa);
            b[1] = codes_to_bf16<1>(v.w[k + 1], sb);
          }
        } else {
          a[0] = codes_to_bf16<kPairs>(v.w[k], sa);
          b[0] = codes_to_bf16<kPairs>(v.w[k + 1], sb);
          if constexpr (kPairs == 2) {
            a[1] = codes_to_bf16<3>(v.w[k], sa);
            b[1] = codes_to_bf16<3>(v.w[k + 1], sb);
          }
        }
#pragma unroll
        for (int n = 0; n < kPairs; ++n) {
          vt[2 * n][i] = __builtin_amdgcn_perm(b[n], a[n], 0x05040100u);
          vt[2 * n + 1][i] = __builtin_amdgcn_perm(b[n], a[n], 0x07060302u);
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const bf16x8 p = as_bf16x8(weights[mt][4 * h], weights[mt][4 * h + 1],
                                   weights[mt][4 * h + 2], weights[mt][4 * h + 3]);
#pragma unroll
        for (int n = 0; n < 2 * kPairs; ++n) {
          const int at = half * 2 * kPairs + n;
          r.acc[mt][at] = mfma(as_bf16x8(vt[n][0], vt[n][1], vt[n][2], vt[n][3]), p, r.acc[mt][at]);
        }
      }
    }
  }
}

// The parts of a tile that hold anything; 1 also where nothing is seen.
__device__ __forceinline__ int parts_of(const AttentionArgs& a, const RowTile& t) {
  const int n = (t.chunk1 - t.chunk0 + a.part_chunks - 1) / a.part_chunks;
  return n > 1 ? n : 1;
}

__device__ __forceinline__ int64_t unit_of(const AttentionArgs& a, int seq, int tile, int kv_head) {
  return (static_cast<int64_t>(seq) * a.row_tiles + tile) * a.cache.kv_heads + kv_head;
}

// A call's arguments behind a loop that does not need them; of the views with more of
// them they are loaded once more: kept in registers through it they put others out.
// Only for kernels whose one parameter they are, at the front of their argument segment
// (launch_for looks at that).
template <int V>
struct LateArgs {
  SumArgs args;
  __device__ __forceinline__ explicit LateArgs(const SumArgs&) {
    using Word = const __attribute__((address_space(4))) uint64_t;
    Word* p = (Word*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    uint64_t words[sizeof(SumArgs) / 8];
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(SumArgs) / 8); ++i) words[i] = p[i];
    args = __builtin_bit_cast(SumArgs, words);
  }
};
template <>
struct LateArgs<kPlain> {
  const AttentionArgs& args;
  __device__ __forceinline__ explicit LateArgs(const AttentionArgs& a) : args(a) {}
};

// ln of the sum of a row's exponentials, from the sum relative to the power `top` of
// two; -infinity for a row that saw nothing.
__device__ __forceinline__ float log_sum(float top, float full) {
  return (top + __builtin_amdgcn_logf(full)) * 0.693147181f;
}

__device__ __forceinline__ void store_lse(const SumArgs& a, const RowTile& t, int kv_head, int row,
                                          float top, float full) {
  const RowOf at = row_of(a, t.query0, t.head0, row);
  if (a.lse)
    a.lse[static_cast<int64_t>(t.start + at.query) * a.ldl + kv_head * a.group + at.head] = log_sum(top, full);
}

// Four neighbouring outputs of a row, divided by its sum; a row that saw nothing
// gets zeros.
__device__ __forceinline__ void store_out(const AttentionArgs& a, const RowTile& t, int kv_head, int row,
                                          int d, int e, f32x4 o, float total) {
  const RowOf at = row_of(a, t.query0, t.head0, row);
  const float inv = total == 0.f ? 0.f : 1.f / total;
  *(LORA_GLOBAL u32x2*)(a.out + static_cast<int64_t>(t.start + at.query) * a.ldo +
                        (kv_head * a.group + at.head) * d + e) =
      u32x2{pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv)};
}

// A part's maximum and sums for one row.
template <int V>
__device__ __forceinline__ void store_stats(const AttentionArgs& a, int64_t at, float top, float total,
                                            float full) {
  if constexpr (V == kPlain)
    *(LORA_GLOBAL u32x2*)(a.stats + at * 2) = u32x2{__float_as_uint(top), __float_as_uint(total)};
  else
    store16(a.stats + at * 4, u32x4{__float_as_uint(top), __float_as_uint(total), __float_as_uint(full), 0u});
}

// Few rows: the workgroup's waves share out the tokens of one row tile, and the
// workgroups of a unit (sequence, key head, row tile) its parts.
template <int D, int MT, int V>
__global__ __launch_bounds__(split_waves(MT) * kWave, MT == 1 ? 4 : 2) void kv_attention_kernel(typename ArgsOf<V>::type a) {
  constexpr int kWaves = split_waves(MT);
  const int tid = static_cast<int>(threadIdx.x);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int lane = lane_id(), g = lane >> 4, c = lane & 15;

  // blockIdx: key head, then row tile (or workgroup of tiles) and part, then
  // sequence.  Neighbours go to other XCDs; with a multiple of 8 key heads the
  // workgroups of one head share an XCD and find its cache in their L2.
  const int kv_head = static_cast<int>(blockIdx.x);
  const int seq = sequence_at(a, static_cast<int>(blockIdx.z));
  const int tile = static_cast<int>(blockIdx.y) / a.parts;
  const int part = static_cast<int>(blockIdx.y) - tile * a.parts;

  const Reader<D> reader = reader_of<D>(a, seq, kv_head);
  // Without a window the first chunk does not depend on the lengths: its pages
  // are looked up beside them.
  int chunk = part * a.part_chunks + wave;
  Pages pages = {-1, -1};
  if (!a.window) pages = reader.pages(chunk * kChunk);

  RowTile t;
  if (!tile_of<V>(a, seq, tile, t)) return;
  const int active = parts_of(a, t);
  if (part >= active) return;
  chunk += t.chunk0;
  int stop = t.chunk0 + (part + 1) * a.part_chunks;
  stop = stop < t.chunk1 ? stop : t.chunk1;
  if (a.window) pages = reader.pages(chunk * kChunk);

  // The queries as B operands, for all waves.
  __shared__ u32x4 q[MT * (D / 32)][kWave];
  // Loads are never behind a condition inside the loop: the wait before a use
  // counts the loads after it, and where paths with and without some meet, it
  // waits for those too.  The last step loads its own chunk once more instead.
  Keys<D> keys;
  Values values;
  const auto next_of = [&](int at) { return at + kWaves < stop ? at + kWaves : at; };
  int next = next_of(chunk);
  Pages ahead = {-1, -1};
  if (chunk < stop) {
    reader.load(keys, pages, chunk * kChunk);
    reader.load(values, pages, chunk * kChunk);
    ahead = reader.pages(next * kChunk);
  }
  for (int f = wave; f < MT * (D / 32); f += kWaves)
    q[f][lane] = query_operand<D>(a, t, kv_head, (f / (D / 32)) * kTile + c, f % (D / 32));
  __shared__ Draft drafts[V == kTree ? MT * kTile : 1];
  if constexpr (V == kTree) stage_drafts(a, t, drafts, MT * kTile, kWaves * kWave);
  Rows<D, MT, V> r;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    if constexpr (V == kTree) {
      r.drafts[mt] = drafts + (row_of(a, t.query0, t.head0, mt * kTile + c).query - t.query0);
      r.before = t.before;
    } else {
      r.place[mt] = t.before + row_of(a, t.query0, t.head0, mt * kTile + c).query;
    }
    r.top[mt] = kNoScore;
    r.sum[mt] = 0.f;
    if constexpr (V != kPlain) r.full[mt] = 0.f;
#pragma unroll
    for (int n = 0; n < D / 16; ++n) r.acc[mt][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  __syncthreads();

  // The next chunk's keys are on their way from the scores on, its values from
  // the products on, and the pages of the one after it are looked up.
  for (; chunk < stop; chunk += kWaves) {
    const int after = next_of(next);
    Span at;
    at.base = chunk * kChunk;
    at.first = t.first;
    at.last = t.last;
    at.window = a.window;
    at.several = V == kTree || t.query1 != t.query0;
    at.ok = pages.v >= 0;
    at.masked = at.base < t.all_first || at.base + kChunk > t.all_last ||
                !__all(pages.v >= 0 && pages.k >= 0);
    uint32_t weights[MT][8];
    weigh(r, weights, keys, &q[0][0], at, a.scale_log2);
    reader.load(keys, ahead, next * kChunk);
    u32x4 scales = values.scales;
    if (at.masked) mask_values(r, scales, at);
    add_values(r, weights, values, scales);
    reader.load(values, ahead, next * kChunk);
    pages = ahead;
    next = after;
    ahead = reader.pages(next * kChunk);
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    r.sum[mt] += __shfl_xor(r.sum[mt], 16);
    r.sum[mt] += __shfl_xor(r.sum[mt], 32);
    if constexpr (V != kPlain) {
      r.full[mt] += __shfl_xor(r.full[mt], 16);
      r.full[mt] += __shfl_xor(r.full[mt], 32);
    }
  }

  // The waves' results, joined in a fixed order.
  // (rows 4 words apart from a multiple of the banks)
  __shared__ float outs[kWaves][kTile][D + 4];
  __shared__ float tops[kWaves][kTile], sums[kWaves][kTile], fulls[V == kPlain ? 1 : kWaves][kTile];
  const LateArgs<V> late(a);
  const auto& b = late.args;
  constexpr int kLanes = D / 4;  // threads a row, four elements each
  constexpr int kRowsAtOnce = kWaves * kWave / kLanes;
  const int e = (tid % kLanes) * 4;
  const int64_t slot =
      (unit_of(b, seq, tile, kv_head) * b.parts + part) * (MT * kTile);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    if (mt > 0) __syncthreads();  // the tile before has been read
    if (g == 0) {
      tops[wave][c] = r.top[mt];
      sums[wave][c] = r.sum[mt];
      if constexpr (V != kPlain) fulls[wave][c] = r.full[mt];
    }
    __syncthreads();
    float top = kNoScore;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, tops[w][c]);
    const float f = __builtin_amdgcn_exp2f(r.top[mt] - top);
    if (mt * kTile + c < t.rows) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < D / 16; ++n)
          outs[wave][c][g * (D / 4) + i * (D / 16) + n] = r.acc[mt][n][i] * f;
    }
    __syncthreads();
    for (int row = tid / kLanes; row < kTile && mt * kTile + row < t.rows; row += kRowsAtOnce) {
      top = kNoScore;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = fmaxf(top, tops[w][row]);
      float total = 0.f, full = 0.f;
      f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        total += sums[w][row] * __builtin_amdgcn_exp2f(tops[w][row] - top);
        if constexpr (V != kPlain) full += fulls[w][row] * __builtin_amdgcn_exp2f(tops[w][row] - top);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += outs[w][row][e + i];
      }
      if (active == 1) {
        store_out(b, t, kv_head, mt * kTile + row, D, e, o, total);
        if constexpr (V != kPlain)
          if (e == 0) store_lse(b, t, kv_head, mt * kTile + row, top, full);
      } else {
        const int64_t at = slot + mt * kTile + row;
        store16(b.partial + at * D + e, __builtin_bit_cast(u32x4, o));
        if (e == 0) store_stats<V>(b, at, top, total, full);
      }
    }
  }
}

// Many rows (pieces of prompts): each of the workgroup's waves has kRowTiles * 16
// rows of its own, and all walk the same chunks.  A chunk's codes are turned into
// bf16 operands once for all of them: each wave takes a quarter of the keys and of
// the values, and leaves its operands in shared memory in the order in which the
// matrix unit's lanes take them (16 bytes a lane, so neither side has bank
// conflicts).  Two buffers and one barrier a chunk; the codes of the next chunk
// are on their way meanwhile.
template <int D, int V>
__global__ __launch_bounds__(kRowWaves * kWave, 2) void kv_attention_rows_kernel(typename ArgsOf<V>::type a) {
  constexpr int MT = kRowTiles;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int lane = lane_id(), g = lane >> 4, c = lane & 15;
  const int kv_head = static_cast<int>(blockIdx.x);
  const int seq = sequence_at(a, static_cast<int>(blockIdx.z));
  // the last rows of a sequence see the most
  const int tile = static_cast<int>(gridDim.y - 1 - blockIdx.y);
  RowTile t;
  if (!tile_of<V>(a, seq, tile, t)) return;
  const Reader<D> reader = reader_of<D>(a, seq, kv_head);

  // This wave's rows, and what they see.
  const int row0 = wave * (MT * kTile);
  const int left = t.rows - row0;
  const int mine = left < 0 ? 0 : (left < MT * kTile ? left : MT * kTile);
  int first = 0, last = 0, all_first = 0, all_last = 0;
  if (V == kTree) {
    if (mine > 0) {
      first = t.first;
      last = t.last;
      all_first = t.all_first;
      all_last = t.all_last;
    }
  } else if (mine > 0) {
    const int place0 = t.before + row_of(a, t.query0, t.head0, row0).query;
    const int place1 = t.before + row_of(a, t.query0, t.head0, row0 + mine - 1).query;
    last = place1 + 1;
    first = a.window && place0 >= a.window ? place0 - a.window + 1 : 0;
    all_first = a.window && place1 >= a.window ? place1 - a.window + 1 : 0;
    all_last = place0 + 1;
  }
  __shared__ Draft drafts[V == kTree ? kRowWaves * MT * kTile : 1];
  if constexpr (V == kTree) stage_drafts(a, t, drafts, kRowWaves * MT * kTile, kRowWaves * kWave);  // (a barrier comes below)
  bf16x8 q[MT][D / 32];
  Rows<D, MT, V> r;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int row = row0 + mt * kTile + c;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      q[mt][i] = __builtin_bit_cast(bf16x8, query_operand<D>(a, t, kv_head, row, i));
    if constexpr (V == kTree) {
      r.drafts[mt] = drafts + (row_of(a, t.query0, t.head0, row).query - t.query0);
      r.before = t.before;
    } else {
      r.place[mt] = t.before + row_of(a, t.query0, t.head0, row).query;
    }
    r.top[mt] = kNoScore;
    r.sum[mt] = 0.f;
    if constexpr (V != kPlain) r.full[mt] = 0.f;
#pragma unroll
    for (int n = 0; n < D / 16; ++n) r.acc[mt][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  __shared__ u32x4 keys[2][4][D / 32][kWave];    // [buffer][tile j][step i][lane]
  __shared__ u32x4 values[2][2][D / 16][kWave];  // [buffer][half of the tokens][element][lane]
  __shared__ uint32_t nans[2][2][4][D / kBlock];  // [buffer][half][g][block]: bits of 8 tokens

  // What this wave turns into operands: the keys of tile j = wave, and of the
  // values the tokens' half `half` and the elements' half `side`.
  const int half = wave >> 1, side = wave & 1;
  uint32_t kw[D / 32], vw[8];
  uint32_t kscale;
  u32x2 vscale;
  bool ok = false, all_ok = false;
  auto load = [&](Pages p, int base) {
    ok = p.v >= 0;
    all_ok = __all(p.v >= 0 && p.k >= 0);
    const int in = (1 << reader.shift) - 1;
    const int ka = (base + 4 * c) & in, va = (base + 16 * g) & in;
    const uint8_t* kb = reader.keys + (p.k < 0 ? 0 : p.k) * reader.page_stride;
    const uint8_t* vb = reader.values + (p.v < 0 ? 0 : p.v) * reader.page_stride;
    const uint8_t* kr = kb + (ka + wave) * (D / 2) + g * (D / 8);
    const uint8_t* vr = vb + (va + 8 * half) * (D / 2) + c * (D / 32);
    if constexpr (D == 128) {
      const u32x4 w = load16(kr);
#pragma unroll
      for (int i = 0; i < 4; ++i) kw[i] = w[i];
    } else {
      const u32x2 w = load8(kr);
      kw[0] = w[0];
      kw[1] = w[1];
    }
    kscale = *(const LORA_GLOBAL uint32_t*)(kb + (((D / 2) + g * (D / 4) / kBlock) << reader.shift) + ka);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if constexpr (D == 128) vw[k] = *(const LORA_GLOBAL uint32_t*)(vr + k * (D / 2));
      else vw[k] = *(const LORA_GLOBAL uint16_t*)(vr + k * (D / 2));
    }
    vscale = load8(vb + (((D / 2) + c * (D / 16) / kBlock) << reader.shift) + va + 8 * half);
  };
  // True if some row of the workgroup does not see all of the chunk at `base`.
  auto partial = [&](int base) {
    return base < t.all_first || base + kChunk > t.all_last || !all_ok;
  };
  auto stage = [&](int buffer, int base) {
    const float ks = __uint_as_float(((kscale >> (8 * wave)) & 255u) << 23);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) keys[buffer][wave][i][lane] = word_to_bf16(kw[i], ks);
    if (partial(base)) {
      // as mask_values, for the tokens that no row of the workgroup sees
      const bool several = V == kTree || t.query1 != t.query0;
      uint32_t nan = 0;
      const int token = base + 16 * g + 8 * half;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t byte = 255u << (8 * (k & 3));
        const bool none = !ok || token + k >= t.last || token + k < t.first;
        const bool bad = several && (vscale[k >> 2] & byte) == byte;
        if (bad && !none) nan |= 1u << k;
        if (bad || none) vscale[k >> 2] &= ~byte;
      }
      constexpr int kLanesABlock = kBlock / (D / 16);
      if (side == 0 && c % kLanesABlock == 0) nans[buffer][half][g][c / kLanesABlock] = nan;
    }
    constexpr int kPairs = D / 64;  // words of two elements
    uint32_t vt[2 * kPairs][4];     // [element][pair of tokens]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = 2 * i;
      const float sa = __uint_as_float(byte_scale(vscale[k >> 2], k & 3));
      const float sb = __uint_as_float(byte_scale(vscale[k >> 2], (k + 1) & 3));
      // this side's elements in the low bytes
      const uint32_t wa = vw[k] >> (8 * kPairs * side), wb = vw[k + 1] >> (8 * kPairs * side);
      uint32_t ea[2], eb[2];
      ea[0] = codes_to_bf16<0>(wa, sa);
      eb[0] = codes_to_bf16<0>(wb, sb);
      if constexpr (kPairs == 2) {
        ea[1] = codes_to_bf16<1>(wa, sa);
        eb[1] = codes_to_bf16<1>(wb, sb);
      }
#pragma unroll
      for (int n = 0; n < kPairs; ++n) {
        vt[2 * n][i] = __builtin_amdgcn_perm(eb[n], ea[n], 0x05040100u);
        vt[2 * n + 1][i] = __builtin_amdgcn_perm(eb[n], ea[n], 0x07060302u);
      }
    }
#pragma unroll
    for (int n = 0; n < 2 * kPairs; ++n)
      values[buffer][half][side * 2 * kPairs + n][lane] = u32x4{vt[n][0], vt[n][1], vt[n][2], vt[n][3]};
  };

  int chunk = t.chunk0;
  bool chunk_partial = false, lane_ok = false, pages_ok = false;
  // (as above: loads without conditions, past the end of the last chunk)
  const int end = t.chunk1 - 1;
  auto upto = [&](int at) { return (at < end ? at : end) * kChunk; };
  Pages ahead = {-1, -1};
  if (chunk < t.chunk1) {
    load(reader.pages(chunk * kChunk), chunk * kChunk);
    chunk_partial = partial(chunk * kChunk);
    lane_ok = ok;
    pages_ok = all_ok;
    stage(0, chunk * kChunk);
    load(reader.pages(upto(chunk + 1)), upto(chunk + 1));
    ahead = reader.pages(upto(chunk + 2));
  }
  __syncthreads();
  for (int buffer = 0; chunk < t.chunk1; ++chunk, buffer ^= 1) {
    Span at;
    at.base = chunk * kChunk;
    at.first = t.first;
    at.last = t.last;
    at.window = a.window;
    at.several = V == kTree || t.query1 != t.query0;
    at.ok = lane_ok;
    at.masked = at.base < all_first || at.base + kChunk > all_last || !pages_ok;
    const bool whole = !chunk_partial;
    if (at.base < last && at.base + kChunk > first) {  // some row of this wave sees some of it
      static_assert(MT == 2, "the two row tiles take turns");
      f32x4 s[MT][4];
      uint32_t weights[MT][8];
      // The matrix products of one row tile beside the powers of the other, for
      // which keys and values are read from shared memory once a tile (8 sequences
      // of up to 4608 tokens in pieces: 3% less time; told to interleave them in
      // fixed patterns the compiler did worse, by 5 to 17%).
      auto scores = [&](int mt, int i) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[mt][j] = mfma(__builtin_bit_cast(bf16x8, keys[buffer][j][i][lane]), q[mt][i],
                          i == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : s[mt][j]);
      };
      auto products = [&](int mt, int h, int n0, int n1) {
        const bf16x8 p = as_bf16x8(weights[mt][4 * h], weights[mt][4 * h + 1], weights[mt][4 * h + 2],
                                   weights[mt][4 * h + 3]);
#pragma unroll
        for (int n = n0; n < n1; ++n)
          r.acc[mt][n] = mfma(__builtin_bit_cast(bf16x8, values[buffer][h][n][lane]), p, r.acc[mt][n]);
      };
      constexpr int kEvery = 4 / (D / 32);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) scores(0, i);
      raise(r, 0, s[0], at, a.scale_log2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i % kEvery == 0) scores(1, i / kEvery);
        powers(weights[0], r, 0, s[0], i, a.scale_log2);
      }
      raise(r, 1, s[1], at, a.scale_log2);
      if (!whole) {
        const int b = c / (kBlock / (D / 16));
        mark_nan(r, nans[buffer][0][g][b] | nans[buffer][1][g][b] << 8, at);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        products(0, i >> 1, (i & 1) * (D / 32), ((i & 1) + 1) * (D / 32));
        powers(weights[1], r, 1, s[1], i, a.scale_log2);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) products(1, h, 0, D / 16);
    }
    // past the last chunk this makes operands that nobody reads
    const int to = upto(chunk + 1);
    chunk_partial = partial(to);
    lane_ok = ok;
    pages_ok = all_ok;
    stage(buffer ^ 1, to);
    load(ahead, upto(chunk + 2));
    ahead = reader.pages(upto(chunk + 3));
    __syncthreads();
  }
  const LateArgs<V> late(a);
  const auto& b = late.args;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    float sum = r.sum[mt];
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    float full = 0.f;
    if constexpr (V != kPlain) {
      full = r.full[mt];
      full += __shfl_xor(full, 16);
      full += __shfl_xor(full, 32);
    }
    const int row = row0 + mt * kTile + c;
    if (row >= t.rows) continue;
    if constexpr (V != kPlain) {
      if (g == 0) store_lse(b, t, kv_head, row, r.top[mt], full);
    }
    const RowOf at = row_of(b, t.query0, t.head0, row);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t* dst = b.out + static_cast<int64_t>(t.start + at.query) * b.ldo +
                    (kv_head * b.group + at.head) * D + g * (D / 4);
    // lane (g, c) has elements g * D / 4 + i * D / 16 + n of row c
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[D / 32];
#pragma unroll
      for (int n = 0; n < D / 32; ++n)
        w[n] = pack_bf16x2(r.acc[mt][2 * n][i] * inv, r.acc[mt][2 * n + 1][i] * inv);
      if constexpr (D == 128) store16(dst + i * (D / 16), u32x4{w[0], w[1], w[2], w[3]});
      else *(LORA_GLOBAL u32x2*)(dst + i * (D / 16)) = u32x2{w[0], w[1]};
    }
  }
}

// Joins the parts of tiles that have several.  D / 4 threads side by side take one
// part's row; a workgroup takes 1 << rows_shift rows and, of each, as many parts at
// once as it has threads left, then adds those sums up in their order.  A launch of
// its own: one compute unit draws too little bandwidth to add a long sequence's
// parts up by itself (131072 tokens, 8 key heads, 32 parts of 8 rows each: 10 us in
// the last workgroup to arrive, 4 here).
constexpr int kJoinThreads = 256;
template <int D, int V>
__global__ __launch_bounds__(kJoinThreads) void kv_attention_join_kernel(typename ArgsOf<V>::type a,
                                                                         int rows_shift) {
  constexpr int kLanes = D / 4, kTeams = kJoinThreads / kLanes;
  const int tid = static_cast<int>(threadIdx.x);
  const int e = (tid % kLanes) * 4, team = tid / kLanes;
  const int teams = kTeams >> rows_shift;  // of a row
  const int of_row = team & (teams - 1);
  const int kv_head = static_cast<int>(blockIdx.x), seq = static_cast<int>(blockIdx.z);
  // a workgroup's rows are of one tile: tiles have whole powers of two of them
  const int index = (static_cast<int>(blockIdx.y) << rows_shift) + team / teams;
  const int tile = index / a.tile_rows;
  const int row = index - tile * a.tile_rows;
  RowTile t;
  if (!tile_of<V>(a, seq, tile, t)) return;  // the whole workgroup, here and below
  const int active = parts_of(a, t);
  if (active == 1) return;
  float top = kNoScore, total = 0.f, full = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  if (row < t.rows) {
    const int64_t slot = unit_of(a, seq, tile, kv_head) * a.parts * a.tile_rows + row;
#pragma unroll 4
    for (int p = of_row; p < active; p += teams) {
      const int64_t at = slot + static_cast<int64_t>(p) * a.tile_rows;
      u32x4 m = {0, 0, 0, 0};
      if constexpr (V == kPlain) {
        const u32x2 two = load8(a.stats + at * 2);
        m[0] = two[0];
        m[1] = two[1];
      } else {
        m = load16(a.stats + at * 4);
      }
      const f32x4 w = __builtin_bit_cast(f32x4, load16(a.partial + at * D + e));
      const float now = fmaxf(top, __uint_as_float(m[0]));
      const float fa = __builtin_amdgcn_exp2f(top - now);
      const float fb = __builtin_amdgcn_exp2f(__uint_as_float(m[0]) - now);
      top = now;
      total = total * fa + __uint_as_float(m[1]) * fb;
      if constexpr (V != kPlain) full = full * fa + __uint_as_float(m[2]) * fb;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = o[i] * fa + w[i] * fb;
    }
  }
  __shared__ f32x4 outs[kTeams][kLanes];
  __shared__ float tops[kTeams], sums[kTeams], fulls[kTeams];
  outs[team][tid % kLanes] = o;
  if (e == 0) {
    tops[team] = top;
    sums[team] = total;
    if constexpr (V != kPlain) fulls[team] = full;
  }
  __syncthreads();
  if (of_row > 0 || row >= t.rows) return;
  top = kNoScore;
  for (int i = team; i < team + teams; ++i) top = fmaxf(top, tops[i]);
  total = 0.f;
  full = 0.f;
  o = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int i = team; i < team + teams; ++i) {
    const float f = __builtin_amdgcn_exp2f(tops[i] - top);
    total += sums[i] * f;
    if constexpr (V != kPlain) full += fulls[i] * f;
    const f32x4 w = outs[i][tid % kLanes];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] += w[k] * f;
  }
  store_out(a, t, kv_head, row, D, e, o, total);
  if constexpr (V != kPlain)
    if (e == 0) store_lse(a, t, kv_head, row, top, full);
}

// How a call is cut up: a function of the sizes alone.
struct AttentionPlan {
  bool many;       // many rows a key head: the rows kernel
  int tile_rows;   // of a workgroup
  int row_tiles, parts, part_chunks;
  int64_t units;   // (sequence, key head, row tile)
  int64_t most_parts;  // no fewer than the parts of any smaller max_len
};

// views: of the views with sums.
static AttentionPlan attention_plan(bool views, int num_seqs, int max_query_len, int64_t max_len, int q_heads,
                                    int kv_heads) {
  AttentionPlan p;
  const int64_t rows = static_cast<int64_t>(max_query_len) * (q_heads / kv_heads);
  const int64_t chunks = (max_len + kChunk - 1) / kChunk;
  // One row tile a workgroup also where there are compute units for all of them and
  // their eight waves are done in up to three rounds, which four with two tiles are not
  // (us, one tile / two: 26 rows and 500 tokens, 32 key heads 12.5 / 14.6; 64 rows, 64
  // key heads of sequences, 1536 tokens 17 / 19, 2600 22.6 / 23.4, 4096 32 / 29; 512 rows
  // and 32768 tokens, 8 key heads 174 / 101), and where pairs of tiles are more than the
  // units but single ones no more than two each (9 counts of 408 to 504 tiles in 260 to 336
  // pairs, heads of 64 and 128, 300 to 4096 tokens: one took less in all 126, by 1 to
  // 25%, and with lengths from 100 to 4096 by 12 to 40%; 480 in 288, heads of 64: 300 tokens 10.4 / 12.1, 1024 14.6 / 17.1, 4096 31 / 41;
  // 468 in 260, heads of 128: 13.2 / 13.6, 19.8 / 20.2, 45 / 50; but 512 tiles in 256
  // pairs, heads of 128, 1024 tokens 20.3 / 17.3).  Where a call
  // with a window has one tile, and the workspace is sized for two and longer walks, it is
  // large enough: at most 3 parts of 16 rows, or a workgroup a compute unit, against at
  // least 7 of 32, or as many workgroups.
  // Only for the views that came later: the plain one's results are those of its tiles.
  const int64_t heads = static_cast<int64_t>(num_seqs) * kv_heads;
  const int64_t narrow = (rows + kTile - 1) / kTile * heads, pairs = (rows + 2 * kTile - 1) / (2 * kTile) * heads;
  const bool one = (narrow <= kCus && chunks <= 3 * split_waves(1)) ||
                   (narrow <= 2 * kCus && pairs > kCus && chunks <= 8 * split_waves(1));
  const int mt = rows <= kTile || (views && one) ? 1 : 2;
  // Workgroups of the rows kernel; with fewer than fill the device twice over
  // (their registers), cutting the tokens up as well gains more than sharing the
  // operands (us, split / rows: 1 sequence of 128 queries of 4096 tokens, 8 key
  // heads of 8, 64 workgroups 37 / 106; 512 queries, 256: 90 / 108; 8 sequences of
  // 128, 512: 176 / 155; 2048 of 2048, 1024: 130 / 94).
  const int64_t wide = (rows + kRowWaves * kRowTiles * kTile - 1) / (kRowWaves * kRowTiles * kTile);
  p.many = rows >= kManyRows && wide * num_seqs * kv_heads >= 2 * kCus;
  p.tile_rows = p.many ? kRowWaves * kRowTiles * kTile : mt * kTile;
  p.row_tiles = static_cast<int>((rows + p.tile_rows - 1) / p.tile_rows);
  p.units = static_cast<int64_t>(num_seqs) * kv_heads * p.row_tiles;
  p.parts = 1;
  p.most_parts = 1;
  p.part_chunks = static_cast<int>(chunks);
  if (p.many) return p;
  // About a workgroup a CU (131072 tokens, 8 key heads, one row tile: 256
  // workgroups 37 us, 1024 42, 2048 56); two for two row tiles where a part is
  // still many rounds of the waves (128 queries of 32768 tokens 201 -> 174 us).
  // A part is whole rounds of the waves.
  const int waves = split_waves(mt);
  const int64_t most = (chunks + waves - 1) / waves;
  p.most_parts = (kCus + p.units - 1) / p.units;
  if (mt == 2 && most >= 16 * p.most_parts) p.most_parts = (2 * kCus + p.units - 1) / p.units;
  p.most_parts = p.most_parts < most ? p.most_parts : most;
  // One round less is not worth the launch that joins the parts (1000 tokens, 8
  // key heads: 2 rounds 9.8 us, 2 parts of 1 round 10.3; 600: 8.6 and 9.7).
  if (most - (most + p.most_parts - 1) / p.most_parts < 2) p.most_parts = 1;
  const int64_t rounds = (most + p.most_parts - 1) / p.most_parts;
  p.part_chunks = static_cast<int>(rounds * waves);
  p.parts = static_cast<int>((most + rounds - 1) / rounds);
  return p;
}

// Bytes of the parts' maxima and sums, which lie before their outputs.
static int64_t stats_bytes(const AttentionPlan& p, View view) {
  return (p.units * p.most_parts * p.tile_rows * (view == kPlain ? 8 : 16) + 255) / 256 * 256;
}

static int64_t workspace_bytes(int num_seqs, int max_query_len, int max_seq_len, int q_heads, int kv_heads,
                               int head_dim, View view) {
  if (num_seqs < 1) return 0;
  const AttentionPlan p = attention_plan(view != kPlain, num_seqs, max_query_len, max_seq_len, q_heads, kv_heads);
  if (p.most_parts <= 1) return 0;
  return stats_bytes(p, view) + p.units * p.most_parts * p.tile_rows * head_dim * 4;
}

int64_t kv_attention_workspace_bytes(int num_seqs, int max_query_len, int max_seq_len, int q_heads,
                                     int kv_heads, int head_dim) {
  return workspace_bytes(num_seqs, max_query_len, max_seq_len, q_heads, kv_heads, head_dim, kPlain);
}

int64_t kv_tree_attention_workspace_bytes(int num_seqs, int max_query_len, int max_seq_len, int q_heads,
                                          int kv_heads, int head_dim) {
  return workspace_bytes(num_seqs, max_query_len, max_seq_len, q_heads, kv_heads, head_dim, kTree);
}

// Kernels that read their arguments by their place (LateArgs).
template <int V>
using LateKernel = void (*)(typename ArgsOf<V>::type);
template <int D, int V>
static void launch_for(const typename ArgsOf<V>::type& a, const AttentionPlan& p, int num_seqs,
                       hipStream_t stream) {
  static_assert(std::is_same_v<decltype(&kv_attention_rows_kernel<D, V>), LateKernel<V>> &&
                std::is_same_v<decltype(&kv_attention_kernel<D, 1, V>), LateKernel<V>> &&
                std::is_same_v<decltype(&kv_attention_kernel<D, 2, V>), LateKernel<V>> &&
                sizeof(SumArgs) % 8 == 0, "arguments are read as words from the segment's start");
  const int heads = a.cache.kv_heads;
  const dim3 grid(heads, p.row_tiles * p.parts, num_seqs);
  if (p.many)
    hipLaunchKernelGGL((kv_attention_rows_kernel<D, V>), grid, dim3(kRowWaves * kWave), 0, stream, a);
  else if (p.tile_rows == kTile)
    hipLaunchKernelGGL((kv_attention_kernel<D, 1, V>), grid, dim3(split_waves(1) * kWave), 0, stream, a);
  else
    hipLaunchKernelGGL((kv_attention_kernel<D, 2, V>), grid, dim3(split_waves(2) * kWave), 0, stream, a);
  if (p.parts > 1) {
    // of a workgroup's threads, as many a row as its parts keep busy
    int shift = 0;
    while ((kJoinThreads / (D / 4) >> (shift + 1)) >= p.parts) ++shift;
    const int rows = a.max_query_len * a.group;
    hipLaunchKernelGGL((kv_attention_join_kernel<D, V>),
                       dim3(heads, (rows + (1 << shift) - 1) >> shift, num_seqs),
                       dim3(kJoinThreads), 0, stream, a, shift);
  }
}

hipError_t launch_kv_attention(const uint16_t* q, int64_t ldq, const int32_t* query_start,
                               const int32_t* seq_lens, const int32_t* page_table,
                               int64_t ld_table, const uint8_t* cache, int num_pages,
                               int page_shift, int num_tokens, int num_seqs, int max_query_len,
                               int max_seq_len, int q_heads, int kv_heads, int head_dim,
                               float scale, int window, const int64_t* masks, int64_t words,
                               bool sums, uint16_t* out, int64_t ldo, float* lse, int64_t ldl,
                               void* workspace, hipStream_t stream) {
  const View view = masks ? kTree : (sums ? kSums : kPlain);
  const int group = q_heads / kv_heads;
  // A window bounds the tokens that any tile walks, beside the step's own ones (of a
  // tree as many as masks have bits, also past max_query_len); the parts are then fewer
  // than those that the workspace is sized for.
  if (window >= max_seq_len) window = 0;
  int64_t longest = max_seq_len;
  if (window) {
    const int64_t seen = window + (masks ? 64 * words : max_query_len) + kChunk;
    longest = longest < seen ? longest : seen;
  }
  const AttentionPlan p = attention_plan(view != kPlain, num_seqs, max_query_len, longest, q_heads, kv_heads);
  SumArgs a = {{q, query_start, seq_lens, page_table, out,
                     {cache, num_pages, page_shift, kv_heads},
                     ldq, ldo, ld_table, num_tokens, max_query_len, max_seq_len, q_heads, window,
                     fabsf(scale) * 1.44269504f, scale < 0.f ? 0x80008000u : 0u,
                     group, ((1 << 21) + group - 1) / group,
                     p.row_tiles, p.parts, p.part_chunks, p.tile_rows, nullptr, nullptr},
                     masks, words, lse, ldl};
  // a hidden token's -infinity must stay -infinity, and a score of zero stay zero
  if (a.scale_log2 < 1.17549435e-38f) a.scale_log2 = 1.17549435e-38f;
  if (a.scale_log2 > 3.402823466e38f) a.scale_log2 = 3.402823466e38f;
  if (p.parts > 1) {
    a.stats = static_cast<float*>(workspace);
    a.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + stats_bytes(p, view));
  }
  switch (view) {
    case kPlain:
      if (head_dim == 64) launch_for<64, kPlain>(a, p, num_seqs, stream);
      else launch_for<128, kPlain>(a, p, num_seqs, stream);
      break;
    case kSums:
      if (head_dim == 64) launch_for<64, kSums>(a, p, num_seqs, stream);
      else launch_for<128, kSums>(a, p, num_seqs, stream);
      break;
    case kTree:
      if (head_dim == 64) launch_for<64, kTree>(a, p, num_seqs, stream);
      else launch_for<128, kTree>(a, p, num_seqs, stream);
      break;
  }
  return hipGetLastError();
}

}  // namespace lora
