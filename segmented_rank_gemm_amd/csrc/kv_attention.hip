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

#include "kv_format.hpp"

namespace lora {

constexpr int kChunk = 64;       // tokens of a wave's step
constexpr int kTile = 16;        // rows of one matrix product
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

struct AttentionArgs {
  const uint16_t* q;
  const int32_t* query_start;
  const int32_t* seq_lens;
  const int32_t* page_table;
  uint16_t* out;
  Cache<const uint8_t> cache;
  int64_t ldq, ldo, ld_table;
  int num_tokens, max_query_len, max_seq_len, q_heads, window;
  float scale_log2;   // |scale| * log2(e): the softmax runs in powers of two
  uint32_t sign;      // scale's sign bits, for q (two bf16)
  int group;          // query heads a key head
  int group_inverse;  // ceil(2^21 / group)
  int row_tiles;      // of 16 * MT rows, for one sequence and key head
  int parts;          // of one row tile's tokens
  int part_chunks;
  int tile_rows;      // 16 * MT
  // Of parts, by (sequence, row tile, key head), part, row of the tile: the
  // maximum and the sum, and the outputs relative to that maximum.
  float* stats;       // [..][2]
  float* partial;     // [..][D]
};

__device__ __forceinline__ uint32_t byte_scale(uint32_t w, int j) {
  // byte j of w as the exponent of a float
  const uint32_t s = j == 0 ? w << 23 : (j == 1 ? w << 15 : (j == 2 ? w << 7 : w >> 1));
  return s & 0x7F800000u;
}

__device__ __forceinline__ bf16x8 as_bf16x8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const u32x4 v = {a, b, c, d};
  return __builtin_bit_cast(bf16x8, v);
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// A lane's part of a chunk's keys: of tokens 4 c + j, the g-th quarter of the head.
template <int D>
struct Keys {
  uint32_t w[4][D / 32];
  uint32_t scales;  // of the four tokens
};

// A lane's part of a chunk's values: of tokens 16 g + k, elements from c * D / 16.
struct Values {
  uint32_t w[16];
  u32x4 scales;  // of the sixteen tokens
};

struct Pages {
  int k, v;  // of this lane's keys and values; -1: no such page
};

// One sequence's cache from one key head's point of view.
template <int D>
struct Reader {
  const uint8_t* keys;
  const uint8_t* values;
  const int32_t* table;
  int64_t page_stride;
  int shift, num_pages, max_seq_len;

  __device__ __forceinline__ int page_at(int token) const {
    const bool there = token < max_seq_len;
    const int p = table[(there ? token : max_seq_len - 1) >> shift];
    return there && p >= 0 && p < num_pages ? p : -1;
  }
  __device__ __forceinline__ Pages pages(int base) const {
    const int lane = lane_id();
    return Pages{page_at(base + 16 * ((lane & 15) >> 2)), page_at(base + 16 * (lane >> 4))};
  }
  // A page that does not exist reads as page 0, which does, and is masked.
  __device__ __forceinline__ void load(Keys<D>& k, Pages p, int base) const {
    const int lane = lane_id(), g = lane >> 4;
    const int at = (base + 4 * (lane & 15)) & ((1 << shift) - 1);
    const uint8_t* b = keys + (p.k < 0 ? 0 : p.k) * page_stride;
    const uint8_t* row = b + at * (D / 2) + g * (D / 8);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (D == 128) {
        const u32x4 w = load16(row + j * (D / 2));
#pragma unroll
        for (int i = 0; i < 4; ++i) k.w[j][i] = w[i];
      } else {
        const u32x2 w = load8(row + j * (D / 2));
        k.w[j][0] = w[0];
        k.w[j][1] = w[1];
      }
    }
    k.scales = *(const LORA_GLOBAL uint32_t*)(b + (((D / 2) + g * (D / 4) / kBlock) << shift) + at);
  }
  __device__ __forceinline__ void load(Values& v, Pages p, int base) const {
    const int lane = lane_id(), c = lane & 15;
    const int at = (base + 16 * (lane >> 4)) & ((1 << shift) - 1);
    const uint8_t* b = values + (p.v < 0 ? 0 : p.v) * page_stride;
    const uint8_t* row = b + at * (D / 2) + c * (D / 32);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if constexpr (D == 128) v.w[k] = *(const LORA_GLOBAL uint32_t*)(row + k * (D / 2));
      else v.w[k] = *(const LORA_GLOBAL uint16_t*)(row + k * (D / 2));
    }
    v.scales = load16(b + (((D / 2) + c * (D / 16) / kBlock) << shift) + at);
  }
};

// The rows of one wave: MT tiles of 16.
template <int D, int MT>
struct Rows {
  f32x4 acc[MT][D / 16];
  float top[MT], sum[MT];
  int place[MT];  // of row c of the tile: the last token that it sees
};

// Where a chunk stands: which of its tokens are there at all.
struct Span {
  int base;           // the chunk's first token
  int first, last;    // tokens [first, last) are seen by some row
  int window;
  bool masked;        // some row does not see all 64, or a page is missing
  bool several;       // the rows are more than one query's
  bool ok;            // the page of this lane's 16 values (and scores) exists
};

// Which of this lane's 16 tokens (base + 16 g + k, bit k) a row at `place` sees.
__device__ __forceinline__ uint32_t seen_bits(const Span& at, int place) {
  const int token = at.base + 16 * (lane_id() >> 4);
  int hi = place - token, lo = at.window ? hi - at.window + 1 : 0;  // lo..hi of 0..15
  hi = hi < 15 ? hi : 15;
  lo = lo > 0 ? lo : 0;
  return at.ok && hi >= lo ? ((2u << hi) - 1u) & ~((1u << lo) - 1u) : 0u;
}

// The first half of the running softmax over one chunk's scores of row tile mt,
// s[j][i] of token 16 g + 4 i + j: hides what a row does not see and moves the
// running maximum.
template <int D, int MT>
__device__ __forceinline__ void raise(Rows<D, MT>& r, int mt, f32x4 (&s)[4], const Span& at,
                                      float scale_log2) {
  if (at.masked) {
    const uint32_t seen = seen_bits(at, r.place[mt]);
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
#pragma unroll
    for (int n = 0; n < D / 16; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) r.acc[mt][n][i] *= shrink;
  }
}

// The second half, a quarter of it: the weights of the tokens 16 g + 4 i + j, in
// bf16 (pairs of tokens 16 g + 2 i, + 1), and the sum of what they were rounded to.
__device__ __forceinline__ void powers(uint32_t (&weights)[8], float& sum, const f32x4 (&s)[4], int i,
                                       float top, float scale_log2) {
  float p[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = __builtin_amdgcn_exp2f(fmaf(s[j][i], scale_log2, -top));
  const uint32_t a = pack_bf16x2(p[0], p[1]), b = pack_bf16x2(p[2], p[3]);
  sum += (bf16_lo(a) + bf16_hi(a)) + (bf16_lo(b) + bf16_hi(b));
  weights[2 * i] = a;
  weights[2 * i + 1] = b;
}

// Scores of one chunk and their weights.  q: the operand [mt][D / 32][lane] in
// shared memory.
template <int D, int MT>
__device__ __forceinline__ void weigh(Rows<D, MT>& r, uint32_t (&weights)[MT][8], const Keys<D>& k,
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
    raise<D, MT>(r, mt, s[mt], at, scale_log2);
#pragma unroll
    for (int i = 0; i < 4; ++i) powers(weights[mt], r.sum[mt], s[mt], i, r.top[mt], scale_log2);
  }
}

// Bits `nan` of this lane's 16 tokens: value blocks that held a NaN and were
// taken out.  Marks the outputs that they reach: those for which the sum over
// these tokens of "seen" is not zero.
template <int D, int MT>
__device__ __forceinline__ void mark_nan(Rows<D, MT>& r, uint32_t nan, const Span& at) {
  if (!__any(nan != 0)) return;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const uint32_t seen = seen_bits(at, r.place[mt]);
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
template <int D, int MT>
__device__ __forceinline__ void mask_values(Rows<D, MT>& r, u32x4& scales, const Span& at) {
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
  mark_nan<D, MT>(r, nan, at);
}

// The weighted values of one chunk.
template <int D, int MT>
__device__ __forceinline__ void add_values(Rows<D, MT>& r, const uint32_t (&weights)[MT][8],
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

// Row `row` of a tile whose first row is head `head0` of query `query0`.
struct RowOf {
  int query, head;
};
__device__ __forceinline__ RowOf row_of(const AttentionArgs& a, int query0, int head0, int row) {
  // head0 + row < group + 128 <= 1152 and the inverse is at most 2^-21 too large, so the
  // product is off by less than 1152 / 2^21 < 1 / group: the quotient is right
  const int n = head0 + row;
  const int q = static_cast<int>(static_cast<uint32_t>(n * a.group_inverse) >> 21);
  return RowOf{query0 + q, n - q * a.group};
}

// One row tile of a sequence: its rows and the tokens that they see.
struct RowTile {
  int start;            // the sequence's first row of q
  int before;           // tokens before its first query (negative: queries that see none)
  int rows;             // of this tile
  int query0, head0;    // the query and head (of the group) of its first row
  int query1;           // the query of its last row
  int first, last;      // tokens [first, last) are seen by some row,
  int all_first, all_last;  // and these by all
  int chunk0, chunk1;   // the chunks that hold them
};

// False if the tile has no rows in this call.
__device__ __forceinline__ bool tile_of(const AttentionArgs& a, int seq, int tile, RowTile& t) {
  t.start = a.query_start[seq];
  const int end = a.query_start[seq + 1];
  int length = a.seq_lens[seq];
  if (t.start < 0 || t.start >= a.num_tokens || end <= t.start) return false;
  const int queries = end - t.start;
  int mine = queries < a.max_query_len ? queries : a.max_query_len;  // that this call does
  mine = mine < a.num_tokens - t.start ? mine : a.num_tokens - t.start;
  const int row0 = tile * a.tile_rows;
  t.rows = mine * a.group - row0;
  if (t.rows <= 0) return false;
  t.rows = t.rows < a.tile_rows ? t.rows : a.tile_rows;
  length = length < 0 ? 0 : (length > a.max_seq_len ? a.max_seq_len : length);
  t.before = length - queries;
  t.query0 = row0 / a.group;
  t.head0 = row0 - t.query0 * a.group;
  t.query1 = row_of(a, t.query0, t.head0, t.rows - 1).query;
  const int place0 = t.before + t.query0, place1 = t.before + t.query1;
  t.last = place1 + 1 > 0 ? place1 + 1 : 0;
  t.first = a.window && place0 >= a.window ? place0 - a.window + 1 : 0;
  t.all_first = a.window && place1 >= a.window ? place1 - a.window + 1 : 0;
  t.all_last = place0 + 1;
  t.chunk0 = t.first / kChunk;
  t.chunk1 = (t.last + kChunk - 1) / kChunk;
  return true;
}

// The parts of a tile that hold anything; 1 also where nothing is seen.
__device__ __forceinline__ int parts_of(const AttentionArgs& a, const RowTile& t) {
  const int n = (t.chunk1 - t.chunk0 + a.part_chunks - 1) / a.part_chunks;
  return n > 1 ? n : 1;
}

__device__ __forceinline__ int64_t unit_of(const AttentionArgs& a, int seq, int tile, int kv_head) {
  return (static_cast<int64_t>(seq) * a.row_tiles + tile) * a.cache.kv_heads + kv_head;
}

// The sequence that the index'th workgroups of a launch take: longest first, so
// that short ones fill the gaps at the end.  A compute unit holds two workgroups;
// where a launch has no more than that, nothing is left for gaps, and those that
// come second to their unit go shortest first, each beside a long one (64
// sequences of 17 to 8192 tokens, 8 key heads: as they come 73 us, longest first
// 69, this 62).  Every wave ranks the sequences for itself; with more of them than
// lanes, many workgroups a compute unit even the work out and they are taken as they
// come.
__device__ __forceinline__ int sequence_at(const AttentionArgs& a, int index) {
  const int n = static_cast<int>(gridDim.z);
  if (n == 1 || n > kWave) return index;
  const int lane = lane_id();
  int work = -1;
  if (lane < n) {
    work = a.seq_lens[lane];
    work = work < 0 || a.query_start[lane + 1] <= a.query_start[lane] ? 0 : work;
  }
  int rank = 0;
  for (int i = 0; i < n; ++i) {
    const int other = __builtin_amdgcn_readlane(work, i);
    rank += other > work || (other == work && i < lane) ? 1 : 0;
  }
  int wanted = index;
  const int each = static_cast<int>(gridDim.x * gridDim.y);  // workgroups of a sequence
  if (each * n > kCus && each * n <= 2 * kCus && index >= kCus / each)
    wanted = n - 1 - (index - kCus / each);
  const unsigned long long hit = __ballot(lane < n && rank == wanted);
  return __ffsll(static_cast<long long>(hit)) - 1;
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

template <int D>
__device__ __forceinline__ Reader<D> reader_of(const AttentionArgs& a, int seq, int kv_head) {
  Reader<D> r;
  const int64_t block = static_cast<int64_t>(D / 2 + D / kBlock) << a.cache.page_shift;
  r.keys = a.cache.data + kv_head * block;
  r.values = r.keys + a.cache.kv_heads * block;
  r.page_stride = 2 * a.cache.kv_heads * block;
  r.table = a.page_table + seq * a.ld_table;
  r.shift = a.cache.page_shift;
  r.num_pages = a.cache.num_pages;
  r.max_seq_len = a.max_seq_len;
  return r;
}

// Lane (g, c)'s part of the i-th B operand of 16 queries: elements g * D / 4 +
// 8 i .. + 7 of tile row `row` (c's); rows past the tile's are zero.
template <int D>
__device__ __forceinline__ u32x4 query_operand(const AttentionArgs& a, const RowTile& t, int kv_head,
                                               int row, int i) {
  u32x4 w = {0, 0, 0, 0};
  if (row < t.rows) {
    const RowOf at = row_of(a, t.query0, t.head0, row);
    w = load16(a.q + static_cast<int64_t>(t.start + at.query) * a.ldq +
               (kv_head * a.group + at.head) * D + (lane_id() >> 4) * (D / 4) + 8 * i);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] ^= a.sign;
  return w;
}

// Few rows: the workgroup's waves share out the tokens of one row tile, and the
// workgroups of a unit (sequence, key head, row tile) its parts.
template <int D, int MT>
__global__ __launch_bounds__(split_waves(MT) * kWave, MT == 1 ? 4 : 2) void kv_attention_kernel(AttentionArgs a) {
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
  if (!tile_of(a, seq, tile, t)) return;
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
  Rows<D, MT> r;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    r.place[mt] = t.before + row_of(a, t.query0, t.head0, mt * kTile + c).query;
    r.top[mt] = kNoScore;
    r.sum[mt] = 0.f;
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
    at.several = t.query1 != t.query0;
    at.ok = pages.v >= 0;
    at.masked = at.base < t.all_first || at.base + kChunk > t.all_last ||
                !__all(pages.v >= 0 && pages.k >= 0);
    uint32_t weights[MT][8];
    weigh<D, MT>(r, weights, keys, &q[0][0], at, a.scale_log2);
    reader.load(keys, ahead, next * kChunk);
    u32x4 scales = values.scales;
    if (at.masked) mask_values<D, MT>(r, scales, at);
    add_values<D, MT>(r, weights, values, scales);
    reader.load(values, ahead, next * kChunk);
    pages = ahead;
    next = after;
    ahead = reader.pages(next * kChunk);
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    r.sum[mt] += __shfl_xor(r.sum[mt], 16);
    r.sum[mt] += __shfl_xor(r.sum[mt], 32);
  }

  // The waves' results, joined in a fixed order.
  // (rows 4 words apart from a multiple of the banks)
  __shared__ float outs[kWaves][kTile][D + 4];
  __shared__ float tops[kWaves][kTile], sums[kWaves][kTile];
  constexpr int kLanes = D / 4;  // threads a row, four elements each
  constexpr int kRowsAtOnce = kWaves * kWave / kLanes;
  const int e = (tid % kLanes) * 4;
  const int64_t slot =
      (unit_of(a, seq, tile, kv_head) * a.parts + part) * (MT * kTile);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    if (mt > 0) __syncthreads();  // the tile before has been read
    if (g == 0) {
      tops[wave][c] = r.top[mt];
      sums[wave][c] = r.sum[mt];
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
      float total = 0.f;
      f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        total += sums[w][row] * __builtin_amdgcn_exp2f(tops[w][row] - top);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += outs[w][row][e + i];
      }
      if (active == 1) {
        store_out(a, t, kv_head, mt * kTile + row, D, e, o, total);
      } else {
        const int64_t at = slot + mt * kTile + row;
        store16(a.partial + at * D + e, __builtin_bit_cast(u32x4, o));
        if (e == 0)
          *(LORA_GLOBAL u32x2*)(a.stats + at * 2) =
              u32x2{__float_as_uint(top), __float_as_uint(total)};
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
template <int D>
__global__ __launch_bounds__(kRowWaves * kWave, 2) void kv_attention_rows_kernel(AttentionArgs a) {
  constexpr int MT = kRowTiles;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int lane = lane_id(), g = lane >> 4, c = lane & 15;
  const int kv_head = static_cast<int>(blockIdx.x);
  const int seq = sequence_at(a, static_cast<int>(blockIdx.z));
  // the last rows of a sequence see the most
  const int tile = static_cast<int>(gridDim.y - 1 - blockIdx.y);
  RowTile t;
  if (!tile_of(a, seq, tile, t)) return;
  const Reader<D> reader = reader_of<D>(a, seq, kv_head);

  // This wave's rows, and what they see.
  const int row0 = wave * (MT * kTile);
  const int left = t.rows - row0;
  const int mine = left < 0 ? 0 : (left < MT * kTile ? left : MT * kTile);
  int first = 0, last = 0, all_first = 0, all_last = 0;
  if (mine > 0) {
    const int place0 = t.before + row_of(a, t.query0, t.head0, row0).query;
    const int place1 = t.before + row_of(a, t.query0, t.head0, row0 + mine - 1).query;
    last = place1 + 1;
    first = a.window && place0 >= a.window ? place0 - a.window + 1 : 0;
    all_first = a.window && place1 >= a.window ? place1 - a.window + 1 : 0;
    all_last = place0 + 1;
  }
  bf16x8 q[MT][D / 32];
  Rows<D, MT> r;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int row = row0 + mt * kTile + c;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      q[mt][i] = __builtin_bit_cast(bf16x8, query_operand<D>(a, t, kv_head, row, i));
    r.place[mt] = t.before + row_of(a, t.query0, t.head0, row).query;
    r.top[mt] = kNoScore;
    r.sum[mt] = 0.f;
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
      const bool several = t.query1 != t.query0;
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
    at.several = t.query1 != t.query0;
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
      raise<D, MT>(r, 0, s[0], at, a.scale_log2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i % kEvery == 0) scores(1, i / kEvery);
        powers(weights[0], r.sum[0], s[0], i, r.top[0], a.scale_log2);
      }
      raise<D, MT>(r, 1, s[1], at, a.scale_log2);
      if (!whole) {
        const int b = c / (kBlock / (D / 16));
        mark_nan<D, MT>(r, nans[buffer][0][g][b] | nans[buffer][1][g][b] << 8, at);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        products(0, i >> 1, (i & 1) * (D / 32), ((i & 1) + 1) * (D / 32));
        powers(weights[1], r.sum[1], s[1], i, r.top[1], a.scale_log2);
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
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    float sum = r.sum[mt];
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    const int row = row0 + mt * kTile + c;
    if (row >= t.rows) continue;
    const RowOf at = row_of(a, t.query0, t.head0, row);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t* dst = a.out + static_cast<int64_t>(t.start + at.query) * a.ldo +
                    (kv_head * a.group + at.head) * D + g * (D / 4);
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
template <int D>
__global__ __launch_bounds__(kJoinThreads) void kv_attention_join_kernel(AttentionArgs a,
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
  if (!tile_of(a, seq, tile, t)) return;  // the whole workgroup, here and below
  const int active = parts_of(a, t);
  if (active == 1) return;
  float top = kNoScore, total = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  if (row < t.rows) {
    const int64_t slot = unit_of(a, seq, tile, kv_head) * a.parts * a.tile_rows + row;
#pragma unroll 4
    for (int p = of_row; p < active; p += teams) {
      const int64_t at = slot + static_cast<int64_t>(p) * a.tile_rows;
      const u32x2 m = load8(a.stats + at * 2);
      const f32x4 w = __builtin_bit_cast(f32x4, load16(a.partial + at * D + e));
      const float now = fmaxf(top, __uint_as_float(m[0]));
      const float fa = __builtin_amdgcn_exp2f(top - now);
      const float fb = __builtin_amdgcn_exp2f(__uint_as_float(m[0]) - now);
      top = now;
      total = total * fa + __uint_as_float(m[1]) * fb;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = o[i] * fa + w[i] * fb;
    }
  }
  __shared__ f32x4 outs[kTeams][kLanes];
  __shared__ float tops[kTeams], sums[kTeams];
  outs[team][tid % kLanes] = o;
  if (e == 0) {
    tops[team] = top;
    sums[team] = total;
  }
  __syncthreads();
  if (of_row > 0 || row >= t.rows) return;
  top = kNoScore;
  for (int i = team; i < team + teams; ++i) top = fmaxf(top, tops[i]);
  total = 0.f;
  o = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int i = team; i < team + teams; ++i) {
    const float f = __builtin_amdgcn_exp2f(tops[i] - top);
    total += sums[i] * f;
    const f32x4 w = outs[i][tid % kLanes];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] += w[k] * f;
  }
  store_out(a, t, kv_head, row, D, e, o, total);
}

// How a call is cut up: a function of the sizes alone.
struct AttentionPlan {
  bool many;       // many rows a key head: the rows kernel
  int tile_rows;   // of a workgroup
  int row_tiles, parts, part_chunks;
  int64_t units;   // (sequence, key head, row tile)
  int64_t most_parts;  // no fewer than the parts of any smaller max_len
};

static AttentionPlan attention_plan(int num_seqs, int max_query_len, int64_t max_len, int q_heads,
                                    int kv_heads) {
  AttentionPlan p;
  const int64_t rows = static_cast<int64_t>(max_query_len) * (q_heads / kv_heads);
  const int mt = rows <= kTile ? 1 : 2;
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
  const int64_t chunks = (max_len + kChunk - 1) / kChunk;
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
static int64_t stats_bytes(const AttentionPlan& p) {
  return (p.units * p.most_parts * p.tile_rows * 8 + 255) / 256 * 256;
}

int64_t kv_attention_workspace_bytes(int num_seqs, int max_query_len, int max_seq_len, int q_heads,
                                     int kv_heads, int head_dim) {
  if (num_seqs < 1) return 0;
  const AttentionPlan p = attention_plan(num_seqs, max_query_len, max_seq_len, q_heads, kv_heads);
  if (p.most_parts <= 1) return 0;
  return stats_bytes(p) + p.units * p.most_parts * p.tile_rows * head_dim * 4;
}

template <int D>
static void launch_for(const AttentionArgs& a, const AttentionPlan& p, int num_seqs,
                       hipStream_t stream) {
  const int heads = a.cache.kv_heads;
  const dim3 grid(heads, p.row_tiles * p.parts, num_seqs);
  if (p.many)
    hipLaunchKernelGGL(kv_attention_rows_kernel<D>, grid, dim3(kRowWaves * kWave), 0, stream, a);
  else if (p.tile_rows == kTile)
    hipLaunchKernelGGL((kv_attention_kernel<D, 1>), grid, dim3(split_waves(1) * kWave), 0, stream, a);
  else
    hipLaunchKernelGGL((kv_attention_kernel<D, 2>), grid, dim3(split_waves(2) * kWave), 0, stream, a);
  if (p.parts > 1) {
    // of a workgroup's threads, as many a row as its parts keep busy
    int shift = 0;
    while ((kJoinThreads / (D / 4) >> (shift + 1)) >= p.parts) ++shift;
    const int rows = a.max_query_len * a.group;
    hipLaunchKernelGGL(kv_attention_join_kernel<D>,
                       dim3(heads, (rows + (1 << shift) - 1) >> shift, num_seqs),
                       dim3(kJoinThreads), 0, stream, a, shift);
  }
}

hipError_t launch_kv_attention(const uint16_t* q, int64_t ldq, const int32_t* query_start,
                               const int32_t* seq_lens, const int32_t* page_table,
                               int64_t ld_table, const uint8_t* cache, int num_pages,
                               int page_shift, int num_tokens, int num_seqs, int max_query_len,
                               int max_seq_len, int q_heads, int kv_heads, int head_dim,
                               float scale, int window, uint16_t* out, int64_t ldo,
                               void* workspace, hipStream_t stream) {
  const int group = q_heads / kv_heads;
  // A window bounds the tokens that any tile walks; the parts are then fewer
  // than those that the workspace is sized for.
  if (window >= max_seq_len) window = 0;
  int64_t longest = max_seq_len;
  if (window) {
    const int64_t seen = static_cast<int64_t>(window) + max_query_len + kChunk;
    longest = longest < seen ? longest : seen;
  }
  const AttentionPlan p = attention_plan(num_seqs, max_query_len, longest, q_heads, kv_heads);
  AttentionArgs a = {q, query_start, seq_lens, page_table, out,
                     {cache, num_pages, page_shift, kv_heads},
                     ldq, ldo, ld_table, num_tokens, max_query_len, max_seq_len, q_heads, window,
                     fabsf(scale) * 1.44269504f, scale < 0.f ? 0x80008000u : 0u,
                     group, ((1 << 21) + group - 1) / group,
                     p.row_tiles, p.parts, p.part_chunks, p.tile_rows, nullptr, nullptr};
  // a hidden token's -infinity must stay -infinity, and a score of zero stay zero
  if (a.scale_log2 < 1.17549435e-38f) a.scale_log2 = 1.17549435e-38f;
  if (a.scale_log2 > 3.402823466e38f) a.scale_log2 = 3.402823466e38f;
  if (p.parts > 1) {
    a.stats = static_cast<float*>(workspace);
    a.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + stats_bytes(p));
  }
  if (head_dim == 64) launch_for<64>(a, p, num_seqs, stream);
  else launch_for<128>(a, p, num_seqs, stream);
  return hipGetLastError();
}

}  // namespace lora
