// What the kernels that walk a sequence's cached keys share (attention, and the
// weight that each token draws): a call's arguments, the cache from one key head's
// point of view, the rows of a tile and the tokens that they see, their queries as
// operands of the matrix unit.
//
// The rows that share a key head (a sequence's queries times its query heads a key
// head) are the columns of 16x16 matrix products, tokens their rows; tokens come in
// chunks of 64.  Row r of the j-th of a chunk's four score tiles is token 4 r + j, so
// that lane (g, c) of the result (lane = 16 g + c) holds the scores of the tokens
// [16 g, 16 g + 16) for row c.
#pragma once

#include "kv_format.hpp"

namespace lora {

constexpr int kChunk = 64;       // tokens of a wave's step
constexpr int kTile = 16;        // rows of one matrix product

// Which tokens a query sees.
enum View : int {
  kPlain = 0,   // those up to its own place
  kSums = 1,    // the same, and the sums of the unrounded exponentials are kept
  kTree = 2,    // the tokens before the first query, and of the queries' own tokens (the
                // drafts) those of its mask's bits; with the sums as well
};

// Drafts of a sequence, at most: words of 64 bits of a row's mask.
constexpr int kDraftWords = 8;

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
  float* stats;       // [..][2], with sums of exponentials [..][4]
  float* partial;     // [..][D]
};

// And of the other views; the plain one's kernels are not handed what they do not read.
struct SumArgs : AttentionArgs {
  const int64_t* masks;  // [num_tokens][words]
  int64_t words;
  float* lse;            // [num_tokens][ldl]; may be null
  int64_t ldl;
};
template <int V>
struct ArgsOf {
  using type = SumArgs;
};
template <>
struct ArgsOf<kPlain> {
  using type = AttentionArgs;
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

// Where a chunk stands: which of its tokens are there at all.
struct Span {
  int base;           // the chunk's first token
  int first, last;    // tokens [first, last) are seen by some row
  int window;
  bool masked;        // some row does not see all 64, or a page is missing
  bool several;       // the rows are more than one query's
  bool ok;            // the page of this lane's 16 values (and scores) exists
};

// Bits [from, to) of a lane's 16 tokens, of which the first is `token`.
__device__ __forceinline__ uint32_t bits_between(int token, int from, int to) {
  int lo = from - token, hi = to - 1 - token;
  hi = hi < 15 ? hi : 15;
  lo = lo > 0 ? lo : 0;
  return hi >= lo ? ((2u << hi) - 1u) & ~((1u << lo) - 1u) : 0u;
}

// Which of this lane's 16 tokens (base + 16 g + k, bit k) a row at `place` sees.
__device__ __forceinline__ uint32_t seen_bits(const Span& at, int place) {
  const int token = at.base + 16 * (lane_id() >> 4);
  int hi = place - token, lo = at.window ? hi - at.window + 1 : 0;  // lo..hi of 0..15
  hi = hi < 15 ? hi : 15;
  lo = lo > 0 ? lo : 0;
  return at.ok && hi >= lo ? ((2u << hi) - 1u) & ~((1u << lo) - 1u) : 0u;
}

// What a query of a tree sees: the tokens [from, before) and, of the drafts from token
// `from` on, those of its mask, which is staged in shared memory as 32-bit words
// (a word more than the masks have keeps neighbouring rows in other banks).
constexpr int kMaskStride = 2 * kDraftWords + 1;
struct Draft {
  uint32_t mask[kMaskStride];
  int from;
};

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
  int queries;          // of the sequence
  int first, last;      // tokens [first, last) are seen by some row,
  int all_first, all_last;  // and these by all
  int chunk0, chunk1;   // the chunks that hold them
};

// The tokens that some row of the tile sees, and those that all see, for a sequence of
// `length` tokens.
template <int V>
__device__ __forceinline__ void see(const typename ArgsOf<V>::type& a, RowTile& t, int length) {
  if constexpr (V == kTree) {
    // A row sees from 0 to all of the drafts that its mask has bits for, and with a
    // window so many fewer of the tokens before them.  (A sequence may have more queries
    // than those; the call is cut up for as many drafts as there are bits.)
    const int text = t.before > 0 ? t.before : 0;
    const int bits = t.before + 64 * static_cast<int>(a.words);
    const int last = bits < length ? bits : length;
    t.last = last > 0 ? last : 0;
    t.first = a.window && text > a.window ? text - a.window : 0;
    t.all_first = a.window && last > a.window ? last - a.window : 0;
    t.all_last = t.before;
  } else {
    const int place0 = t.before + t.query0, place1 = t.before + t.query1;
    t.last = place1 + 1 > 0 ? place1 + 1 : 0;
    t.first = a.window && place0 >= a.window ? place0 - a.window + 1 : 0;
    t.all_first = a.window && place1 >= a.window ? place1 - a.window + 1 : 0;
    t.all_last = place0 + 1;
  }
  t.chunk0 = t.first / kChunk;
  t.chunk1 = (t.last + kChunk - 1) / kChunk;
}

// Queries of a sequence that count, where all its tokens are walked: so many that those of
// a call see none of 2^30 tokens, and few enough that places and their differences do not
// pass 2^31.
constexpr int kMostQueries = (1 << 30) + (1 << 22);

// False if the tile has no rows in this call.  all: the tile is all of the sequence's rows.
template <int V = kPlain>
__device__ __forceinline__ bool tile_of(const typename ArgsOf<V>::type& a, int seq, int tile, RowTile& t,
                                        bool all = false) {
  t.start = a.query_start[seq];
  const int end = a.query_start[seq + 1];
  int length = a.seq_lens[seq];
  if (t.start < 0 || t.start >= a.num_tokens || end <= t.start) return false;
  int queries = end - t.start;
  if (V == kTree || all) queries = queries < kMostQueries ? queries : kMostQueries;
  int mine = queries < a.max_query_len ? queries : a.max_query_len;  // that this call does
  mine = mine < a.num_tokens - t.start ? mine : a.num_tokens - t.start;
  const int row0 = all ? 0 : tile * a.tile_rows;
  t.rows = mine * a.group - row0;
  if (t.rows <= 0) return false;
  if (!all) t.rows = t.rows < a.tile_rows ? t.rows : a.tile_rows;
  length = length < 0 ? 0 : (length > a.max_seq_len ? a.max_seq_len : length);
  t.before = length - queries;
  t.queries = queries;
  t.query0 = row0 / a.group;
  t.head0 = row0 - t.query0 * a.group;
  t.query1 = all ? mine - 1 : row_of(a, t.query0, t.head0, t.rows - 1).query;
  see<V>(a, t, length);
  return true;
}

// Stages what `count` queries from the tile's first on see, by one thread for each
// (nothing for those past the tile's last).  A query's tokens
// in their order are those before the drafts and then its mask's; with a window it
// sees the last `window` of them.  A mask's bits of drafts that are not there (past
// the sequence's, or before its first token) do not count.
__device__ __forceinline__ void stage_drafts(const SumArgs& a, const RowTile& t, Draft* drafts,
                                             int count, int threads) {
  const int words = static_cast<int>(a.words);
  const int low = t.before < 0 ? -t.before : 0, high = t.queries;
  for (int i = static_cast<int>(threadIdx.x); i < count; i += threads) {
    const bool there = t.query0 + i <= t.query1;
    const int64_t* row = a.masks + static_cast<int64_t>(t.start + (there ? t.query0 + i : t.query1)) * words;
    int seen = 0;
    for (int w = 0; w < kDraftWords; ++w) {
      unsigned long long m = w < words && there ? static_cast<unsigned long long>(row[w]) : 0ull;
      const int lo = low - 64 * w, hi = high - 64 * w;  // bits [lo, hi) of this word count
      if (hi <= 0 || lo >= 64) m = 0;
      if (hi > 0 && hi < 64) m &= (1ull << hi) - 1;
      if (lo > 0 && lo < 64) m &= ~((1ull << lo) - 1);
      drafts[i].mask[2 * w] = static_cast<uint32_t>(m);
      drafts[i].mask[2 * w + 1] = static_cast<uint32_t>(m >> 32);
      seen += __popcll(m);
    }
    int from = 0;
    if (a.window) {
      const int text = t.before > 0 ? t.before : 0;
      if (seen <= a.window) {
        from = text - (a.window - seen);
        from = from > 0 ? from : 0;
      } else {
        // past the lowest seen - window bits
        int drop = seen - a.window, w = 0;
        uint32_t m = drafts[i].mask[0];
        while (__popc(m) <= drop) {  // a later word has a bit left: seen > drop
          drop -= __popc(m);
          m = drafts[i].mask[++w];
        }
        for (; drop > 0; --drop) m &= m - 1;
        from = t.before + 32 * w + __ffs(static_cast<int>(m)) - 1;
      }
    }
    drafts[i].from = from;
  }
}

// Which of this lane's 16 tokens a query of a tree sees.
__device__ __forceinline__ uint32_t seen_bits(const Span& at, const Draft& d, int before) {
  const int token = at.base + 16 * (lane_id() >> 4);
  const int o = token - before;  // the draft's number of the first of them
  uint32_t bits = bits_between(token, 0, before);
  if (o > -16) {
    const int w = o >> 5, shift = o & 31;
    const uint32_t m0 = w >= 0 && w < 2 * kDraftWords ? d.mask[w] : 0u;
    const uint32_t m1 = w >= -1 && w + 1 < 2 * kDraftWords ? d.mask[w + 1] : 0u;
    bits |= static_cast<uint32_t>((static_cast<unsigned long long>(m1) << 32 | m0) >> shift);
  }
  return at.ok ? bits & bits_between(token, d.from, token + 16) : 0u;
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

}  // namespace lora
