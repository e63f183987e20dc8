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
// are rounded to bf16 for the second product, as the matrix unit takes them.
//
// Bound by: HBM (68 bytes a token and head at D = 128) as long as the rows of a
// key head fit one tile; by the exponentials and the matrix unit for prompts.

#include "kv_format.hpp"

namespace lora {

constexpr int kChunk = 64;       // tokens of a wave's step
constexpr int kTile = 16;        // rows of one matrix product
// Waves of a workgroup: they share out one tile's tokens (split), or have tiles
// of their own.  More row tiles a wave need the registers of four waves.
__host__ __device__ constexpr int waves_of(int mt, bool split) { return split && mt == 1 ? 8 : 4; }
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
  int row_tiles;      // of 16 * MT rows, for one sequence and key head
  int parts;          // of one row tile's tokens
  int part_chunks;
  int* arrivals;      // one counter a (sequence, key head, row tile)
  float* partial;     // [unit][part][MT * 16][D], then [..][2]: maximum and sum
};

// What a wave holds of one chunk: keys of token 4 c + j, block g (D = 128) or
// half block g (D = 64); values of the tokens 16 g + k, elements from c * D / 16.
template <int D>
struct Chunk {
  static constexpr int kKeyWords = D / 32;  // u32 of codes a key tile and lane
  uint32_t k[4][kKeyWords];
  uint32_t v[16];
  uint32_t ks;     // scales of the four keys
  u32x4 vs;        // scales of the sixteen values
  bool ok;         // the page of this lane's values (and of its 16 scores) exists
  bool all_ok;     // and that of its keys
};

struct Pages {
  int k, v;  // -1: no token there, or no such page
};

__device__ __forceinline__ uint32_t byte_scale(uint32_t w, int j) {
  // byte j of w as the exponent of a float
  const uint32_t s = j == 0 ? w << 23 : (j == 1 ? w << 15 : (j == 2 ? w << 7 : w >> 1));
  return s & 0x7F800000u;
}

template <int S>
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, S));
}

__device__ __forceinline__ bf16x8 as_bf16x8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const u32x4 v = {a, b, c, d};
  return __builtin_bit_cast(bf16x8, v);
}

// Eight codes of one word, as the A operand of one product.
__device__ __forceinline__ bf16x8 word_to_bf16(uint32_t w, float scale) {
  return as_bf16x8(codes_to_bf16<0>(w, scale), codes_to_bf16<1>(w, scale), codes_to_bf16<2>(w, scale),
                   codes_to_bf16<3>(w, scale));
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// One sequence's cache from one key head's point of view.
template <int D>
struct Reader {
  const uint8_t* keys;
  const uint8_t* values;
  const int32_t* table;
  int64_t page_stride;
  int shift, num_pages, last;

  __device__ __forceinline__ int page_at(int token) const {
    if (token >= last) return -1;
    const int p = table[token >> shift];
    return p >= 0 && p < num_pages ? p : -1;
  }
  __device__ __forceinline__ Pages pages(int base) const {
    const int lane = lane_id();
    Pages p;
    p.k = page_at(base + 16 * ((lane & 15) >> 2));
    p.v = page_at(base + 16 * (lane >> 4));
    return p;
  }
  // A page that does not exist reads as page 0, which does, and is masked.
  __device__ __forceinline__ void load(Chunk<D>& ch, Pages p, int base) const {
    const int lane = lane_id(), g = lane >> 4, c = lane & 15;
    const int in = (1 << shift) - 1;
    const int64_t scales = static_cast<int64_t>(D / 2) << shift;
    ch.ok = p.v >= 0;
    ch.all_ok = p.v >= 0 && p.k >= 0;
    const uint8_t* kb = keys + (p.k < 0 ? 0 : p.k) * page_stride;
    const uint8_t* vb = values + (p.v < 0 ? 0 : p.v) * page_stride;
    const int ka = (base + 4 * c) & in, va = (base + 16 * g) & in;
    const uint8_t* kr = kb + ka * (D / 2) + g * (D / 8);
    const uint8_t* vr = vb + va * (D / 2) + c * (D / 32);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (D == 128) {
        const u32x4 w = load16(kr + j * (D / 2));
#pragma unroll
        for (int i = 0; i < 4; ++i) ch.k[j][i] = w[i];
      } else {
        const u32x2 w = load8(kr + j * (D / 2));
        ch.k[j][0] = w[0];
        ch.k[j][1] = w[1];
      }
    }
    ch.ks = *(const LORA_GLOBAL uint32_t*)(kb + scales + ((g * (D / 4) / kBlock) << shift) + ka);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if constexpr (D == 128) ch.v[k] = *(const LORA_GLOBAL uint32_t*)(vr + k * (D / 2));
      else ch.v[k] = *(const LORA_GLOBAL uint16_t*)(vr + k * (D / 2));
    }
    ch.vs = load16(vb + scales + ((c * (D / 16) / kBlock) << shift) + va);
  }
};

// The rows of one wave: MT tiles of 16.
template <int D, int MT>
struct Rows {
  bf16x8 q[MT][D / 32];
  f32x4 acc[MT][D / 16];
  float top[MT], sum[MT];
  int place[MT];  // of row c of the tile: the last token that it sees
};

// One chunk: scores, running softmax, weighted values.  `masked`: some row does
// not see all 64 tokens, or a page is missing.
template <int D, int MT, bool kMasked>
__device__ __forceinline__ void attend(Rows<D, MT>& r, const Chunk<D>& ch, int base, int first, int last,
                                       int window, float scale_log2, bool several) {
  const int lane = lane_id(), g = lane >> 4;
  uint32_t weights[MT][8];
  uint32_t seen[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) seen[mt] = 0xFFFFu;
  if constexpr (kMasked) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      // this lane's tokens are base + 16 g + [0, 16)
      const int at = base + 16 * g;
      int hi = r.place[mt] - at, lo = window ? hi - window + 1 : 0;  // visible: lo..hi of 0..15
      hi = hi < 15 ? hi : 15;
      lo = lo > 0 ? lo : 0;
      seen[mt] = ch.ok && hi >= lo ? ((2u << hi) - 1u) & ~((1u << lo) - 1u) : 0u;
    }
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    f32x4 s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float scale = __uint_as_float(byte_scale(ch.ks, j));
      s[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < D / 32; ++i) s[j] = mfma(word_to_bf16(ch.k[j][i], scale), r.q[mt][i], s[j]);
    }
    if constexpr (kMasked) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!(seen[mt] >> (4 * i + j) & 1u)) s[j][i] = -INFINITY;
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
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float p[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[j] = __builtin_amdgcn_exp2f(fmaf(s[j][i], scale_log2, -r.top[mt]));
        if constexpr (kMasked)
          if (!(seen[mt] >> (4 * i + j) & 1u)) p[j] = 0.f;
        r.sum[mt] += p[j];
      }
      weights[mt][2 * i] = pack_bf16x2(p[0], p[1]);
      weights[mt][2 * i + 1] = pack_bf16x2(p[2], p[3]);
    }
  }
  u32x4 vs = ch.vs;
  if constexpr (kMasked) {
    // Values that no row sees may be anything; their weights are zero, their
    // scales must not be NaN.
    uint32_t nan = 0;
    const int at = base + 16 * g;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const uint32_t byte = (vs[k >> 2] >> (8 * (k & 3))) & 255u;
      const bool none = !ch.ok || at + k >= last || at + k < first;
      if (none) vs[k >> 2] &= ~(255u << (8 * (k & 3)));
      else if (several && byte == kScaleNan) {
        nan |= 1u << k;
        vs[k >> 2] &= ~(255u << (8 * (k & 3)));
      }
    }
    // A NaN block that some rows see and others do not: the sum over its tokens
    // of "seen" marks the outputs that it reaches.
    if (several && __any(nan != 0)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 a;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          a[i] = (nan >> (8 * h + 2 * i) & 1u ? 0x3F80u : 0u) |
                 (nan >> (8 * h + 2 * i + 1) & 1u ? 0x3F800000u : 0u);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          u32x4 b;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            b[i] = (seen[mt] >> (8 * h + 2 * i) & 1u ? 0x3F80u : 0u) |
                   (seen[mt] >> (8 * h + 2 * i + 1) & 1u ? 0x3F800000u : 0u);
          const f32x4 hit = mfma(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                 f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int n = 0; n < D / 16; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (hit[i] > 0.f) r.acc[mt][n][i] = NAN;
        }
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t vt[D / 16][4];  // [element][pair of tokens]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = 8 * h + 2 * i;
      const float sa = __uint_as_float(byte_scale(vs[k >> 2], k & 3));
      const float sb = __uint_as_float(byte_scale(vs[k >> 2], (k + 1) & 3));
      const bf16x8 a = word_to_bf16(ch.v[k], sa), b = word_to_bf16(ch.v[k + 1], sb);
      const u32x4 wa = __builtin_bit_cast(u32x4, a), wb = __builtin_bit_cast(u32x4, b);
#pragma unroll
      for (int n = 0; n < D / 32; ++n) {
        vt[2 * n][i] = __builtin_amdgcn_perm(wb[n], wa[n], 0x05040100u);
        vt[2 * n + 1][i] = __builtin_amdgcn_perm(wb[n], wa[n], 0x07060302u);
      }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const bf16x8 p = as_bf16x8(weights[mt][4 * h], weights[mt][4 * h + 1], weights[mt][4 * h + 2],
                                 weights[mt][4 * h + 3]);
#pragma unroll
      for (int n = 0; n < D / 16; ++n)
        r.acc[mt][n] = mfma(as_bf16x8(vt[n][0], vt[n][1], vt[n][2], vt[n][3]), p, r.acc[mt][n]);
    }
  }
}

// Four neighbouring outputs of a row, divided by its sum; a row that saw nothing
// gets zeros.
__device__ __forceinline__ void store_out(const AttentionArgs& a, int start, int head0, int row,
                                          int group, int e, int d, f32x4 o, float total) {
  const int qi = row / group;
  const float inv = total == 0.f ? 0.f : 1.f / total;
  *(LORA_GLOBAL u32x2*)(a.out + static_cast<int64_t>(start + qi) * a.ldo +
                        (head0 + row - qi * group) * d + e) =
      u32x2{pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv)};
}

// kSplit: the workgroup's waves share out the tokens of one row tile, and the
// workgroups of a unit its parts; otherwise each wave has a row tile of its own
// and walks all of that tile's tokens.
template <int D, int MT, bool kSplit>
__global__ __launch_bounds__(waves_of(MT, kSplit) * kWave) void kv_attention_kernel(
    AttentionArgs a) {
  constexpr int kWaves = waves_of(MT, kSplit);
  const int tid = static_cast<int>(threadIdx.x);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int lane = lane_id(), g = lane >> 4, c = lane & 15;
  const int kv_heads = a.cache.kv_heads;
  const int group = a.q_heads / kv_heads;

  // blockIdx.x = (row tile, or its workgroup of tiles) and part, slowest first;
  // then the sequence and key head, so that neighbours read different caches
  const int heads = static_cast<int>(blockIdx.x);
  const int kv_head = heads % kv_heads, seq = heads / kv_heads;
  const int part = kSplit ? static_cast<int>(blockIdx.y) % a.parts : 0;
  const int tile = kSplit ? static_cast<int>(blockIdx.y) / a.parts
                          : static_cast<int>(blockIdx.y) * kWaves + wave;
  const int start = a.query_start[seq], end = a.query_start[seq + 1];
  if (start < 0 || start >= a.num_tokens || end <= start) return;
  const int queries = end - start;
  int mine = queries < a.max_query_len ? queries : a.max_query_len;  // that this call does
  mine = mine < a.num_tokens - start ? mine : a.num_tokens - start;
  const int row0 = tile * kTile * MT;
  const int rows = mine * group;
  if (row0 >= rows) return;  // the whole workgroup (kSplit), or a wave that shares nothing
  int length = a.seq_lens[seq];
  length = length < 0 ? 0 : (length > a.max_seq_len ? a.max_seq_len : length);

  // Tokens that some row of the tile sees, and that all of them see.
  const int q_first = row0 / group;
  const int row_last = row0 + kTile * MT < rows ? row0 + kTile * MT - 1 : rows - 1;
  const int q_last = row_last / group;
  const int place0 = length - queries + q_first, place1 = length - queries + q_last;
  const int last = place1 + 1 > 0 ? place1 + 1 : 0;
  int first = a.window ? place0 - a.window + 1 : 0;
  first = first > 0 ? first : 0;
  int all_first = a.window ? place1 - a.window + 1 : 0;
  all_first = all_first > 0 ? all_first : 0;
  const int all_last = place0 + 1;
  const int chunk0 = first / kChunk, chunk1 = (last + kChunk - 1) / kChunk;
  const int active = kSplit ? (chunk1 - chunk0 + a.part_chunks - 1) / a.part_chunks : 1;
  if (kSplit && part >= (active > 1 ? active : 1)) return;

  Rows<D, MT> r;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int row = row0 + mt * kTile + c;
    const int qi = row / group;
    r.place[mt] = length - queries + qi;
    r.top[mt] = kNoScore;
    r.sum[mt] = 0.f;
#pragma unroll
    for (int n = 0; n < D / 16; ++n) r.acc[mt][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    const uint16_t* src = a.q + static_cast<int64_t>(start + qi) * a.ldq +
                          (kv_head * group + row - qi * group) * D + g * (D / 4);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      u32x4 w = {0, 0, 0, 0};
      if (row < rows) w = load16(src + 8 * i);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] ^= a.sign;
      r.q[mt][i] = __builtin_bit_cast(bf16x8, w);
    }
  }

  Reader<D> reader;
  const int64_t block = static_cast<int64_t>(D / 2 + D / kBlock) << a.cache.page_shift;
  reader.keys = a.cache.data + kv_head * block;
  reader.values = reader.keys + kv_heads * block;
  reader.page_stride = 2 * kv_heads * block;
  reader.table = a.page_table + seq * a.ld_table;
  reader.shift = a.cache.page_shift;
  reader.num_pages = a.cache.num_pages;
  reader.last = last;

  const int step = kSplit ? kWaves : 1;
  int chunk = chunk0, stop = chunk1;
  if constexpr (kSplit) {
    chunk = chunk0 + part * a.part_chunks + wave;
    stop = chunk0 + (part + 1) * a.part_chunks;
    stop = stop < chunk1 ? stop : chunk1;
  }
  // The pages of the chunk after next and the codes of the next are on their way
  // while a chunk is worked on.
  if (chunk < stop) {
    Chunk<D> now, next;
    reader.load(now, reader.pages(chunk * kChunk), chunk * kChunk);
    Pages ahead = reader.pages((chunk + step) * kChunk);
    for (; chunk < stop; chunk += step) {
      const int base = chunk * kChunk;
      if (chunk + step < stop) {
        reader.load(next, ahead, base + step * kChunk);
        ahead = reader.pages(base + 2 * step * kChunk);
      }
      const bool whole = base >= all_first && base + kChunk <= all_last;
      if (whole && __all(now.all_ok))
        attend<D, MT, false>(r, now, base, first, last, a.window, a.scale_log2, q_last != q_first);
      else
        attend<D, MT, true>(r, now, base, first, last, a.window, a.scale_log2, q_last != q_first);
      now = next;
    }
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    r.sum[mt] += __shfl_xor(r.sum[mt], 16);
    r.sum[mt] += __shfl_xor(r.sum[mt], 32);
  }

  if constexpr (!kSplit) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int row = row0 + mt * kTile + c;
      if (row >= rows) continue;
      const int qi = row / group;
      const float inv = r.sum[mt] == 0.f ? 0.f : 1.f / r.sum[mt];
      uint16_t* dst = a.out + static_cast<int64_t>(start + qi) * a.ldo +
                      (kv_head * group + row - qi * group) * D + g * (D / 4);
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
    return;
  } else {
    // The waves' parts, then the workgroups', added in a fixed order.
    __shared__ float outs[kWaves][kTile][D];
    __shared__ float tops[kWaves][kTile], sums[kWaves][kTile];
    __shared__ int is_last;
    constexpr int kLanes = D / 4;                    // threads a row, four elements each
    constexpr int kRowsAtOnce = kWaves * kWave / kLanes;
    constexpr int kSteps = (kTile + kRowsAtOnce - 1) / kRowsAtOnce;
    const int row_0 = tid / kLanes, e = (tid % kLanes) * 4;
    const int unit = (tile * static_cast<int>(gridDim.x)) + heads;
    const int64_t slot = static_cast<int64_t>(unit) * a.parts + part;
    const int64_t units = static_cast<int64_t>(a.row_tiles) * gridDim.x;
    float* ml = a.partial + units * a.parts * (MT * kTile * D);
    const bool alone = active <= 1;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt > 0) __syncthreads();
      if (g == 0) {
        tops[wave][c] = r.top[mt];
        sums[wave][c] = r.sum[mt];
      }
      __syncthreads();
      float top = kNoScore;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = fmaxf(top, tops[w][c]);
      const float f = __builtin_amdgcn_exp2f(r.top[mt] - top);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < D / 16; ++n)
          outs[wave][c][g * (D / 4) + i * (D / 16) + n] = r.acc[mt][n][i] * f;
      __syncthreads();
#pragma unroll
      for (int at_row = 0; at_row < kSteps; ++at_row) {
        const int row_t = row_0 + at_row * kRowsAtOnce;
        const int row = row0 + mt * kTile + row_t;
        if (row_t >= kTile || row >= rows) break;
        top = kNoScore;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) top = fmaxf(top, tops[w][row_t]);
        float total = 0.f;
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          total += sums[w][row_t] * __builtin_amdgcn_exp2f(tops[w][row_t] - top);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] += outs[w][row_t][e + i];
        }
        if (alone) {
          store_out(a, start, kv_head * group, row, group, e, D, o, total);
        } else {
          const int64_t at = slot * (MT * kTile) + mt * kTile + row_t;
          store16_coherent(buffer_rsrc(a.partial + at * D, D * 4), e * 4,
                           __builtin_bit_cast(u32x4, o));
          if (e == 0)
            __builtin_amdgcn_raw_buffer_store_b64(
                u32x2{__float_as_uint(top), __float_as_uint(total)}, buffer_rsrc(ml + at * 2, 8), 0,
                0, kCachePolicyCoherent);
        }
      }
    }
    if (alone) return;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this thread's parts have been written
    __syncthreads();
    if (tid == 0)
      is_last = __hip_atomic_fetch_add(a.arrivals + unit, 1, __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT) == active - 1;
    __syncthreads();
    if (!is_last) return;
    if (tid == 0) __hip_atomic_store(a.arrivals + unit, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // the unit's rows in turn, MT * 16 of them
    for (int row_t = row_0; row_t < MT * kTile && row0 + row_t < rows; row_t += kRowsAtOnce) {
      const int64_t at0 = static_cast<int64_t>(unit) * a.parts * (MT * kTile) + row_t;
      float top = kNoScore, total = 0.f;
      f32x4 o = {0.f, 0.f, 0.f, 0.f};
      for (int p = 0; p < active; ++p) {
        const int64_t at = at0 + static_cast<int64_t>(p) * (MT * kTile);
        const u32x2 w = load8_coherent(buffer_rsrc(ml + at * 2, 8), 0);
        const f32x4 part_o = __builtin_bit_cast(
            f32x4, load16_coherent(buffer_rsrc(a.partial + at * D, D * 4), e * 4));
        const float m = __uint_as_float(w[0]);
        const float now = fmaxf(top, m);
        const float fa = __builtin_amdgcn_exp2f(top - now), fb = __builtin_amdgcn_exp2f(m - now);
        top = now;
        total = total * fa + __uint_as_float(w[1]) * fb;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = o[i] * fa + part_o[i] * fb;
      }
      store_out(a, start, kv_head * group, row0 + row_t, group, e, D, o, total);
    }
  }
}

// How a call is cut up: a function of the sizes alone.
struct AttentionPlan {
  int mt;          // row tiles of 16 a wave
  bool split;      // the waves share out the tokens (see the kernel)
  int row_tiles, parts, part_chunks;
  int64_t units;   // (sequence, key head, row tile)
  int64_t most_parts;  // no fewer than the parts of any smaller max_len
};

static AttentionPlan attention_plan(int num_seqs, int max_query_len, int64_t max_len, int q_heads,
                                    int kv_heads) {
  AttentionPlan p;
  const int64_t rows = static_cast<int64_t>(max_query_len) * (q_heads / kv_heads);
  p.mt = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4);
  p.split = rows < 256;
  p.row_tiles = static_cast<int>((rows + kTile * p.mt - 1) / (kTile * p.mt));
  p.units = static_cast<int64_t>(num_seqs) * kv_heads * p.row_tiles;
  p.parts = 1;
  p.most_parts = 1;
  const int64_t chunks = (max_len + kChunk - 1) / kChunk;
  p.part_chunks = static_cast<int>(chunks);
  if (!p.split) return p;
  // About two workgroups a CU; a part is whole rounds of the waves.
  const int waves = waves_of(p.mt, true);
  const int64_t most = (chunks + waves - 1) / waves;
  p.most_parts = (2 * kCus + p.units - 1) / p.units;
  p.most_parts = p.most_parts < most ? p.most_parts : most;
  const int64_t rounds = (most + p.most_parts - 1) / p.most_parts;
  p.part_chunks = static_cast<int>(rounds * waves);
  p.parts = static_cast<int>((most + rounds - 1) / rounds);
  return p;
}

static int64_t counter_bytes(const AttentionPlan& p) { return (p.units * 4 + 255) / 256 * 256; }

int64_t kv_attention_workspace_bytes(int num_seqs, int max_query_len, int max_seq_len, int q_heads,
                                     int kv_heads, int head_dim) {
  if (num_seqs < 1) return 0;
  const AttentionPlan p = attention_plan(num_seqs, max_query_len, max_seq_len, q_heads, kv_heads);
  if (p.most_parts <= 1) return 0;
  return counter_bytes(p) + p.units * p.most_parts * p.mt * kTile * (head_dim + 2) * 4;
}

template <int D, int MT, bool kSplit>
static void launch(const AttentionArgs& a, int heads, hipStream_t stream) {
  constexpr int kWaves = waves_of(MT, kSplit);
  const int groups = kSplit ? a.row_tiles * a.parts : (a.row_tiles + kWaves - 1) / kWaves;
  hipLaunchKernelGGL((kv_attention_kernel<D, MT, kSplit>), dim3(heads, groups),
                     dim3(kWaves * kWave), 0, stream, a);
}

template <int D>
static void launch_for(const AttentionArgs& a, const AttentionPlan& p, int heads, hipStream_t stream) {
  if (!p.split) launch<D, 4, false>(a, heads, stream);
  else if (p.mt == 1) launch<D, 1, true>(a, heads, stream);
  else if (p.mt == 2) launch<D, 2, true>(a, heads, stream);
  else launch<D, 4, true>(a, heads, stream);
}

hipError_t launch_kv_attention(const uint16_t* q, int64_t ldq, const int32_t* query_start,
                               const int32_t* seq_lens, const int32_t* page_table,
                               int64_t ld_table, const uint8_t* cache, int num_pages,
                               int page_shift, int num_tokens, int num_seqs, int max_query_len,
                               int max_seq_len, int q_heads, int kv_heads, int head_dim,
                               float scale, int window, uint16_t* out, int64_t ldo,
                               void* workspace, hipStream_t stream) {
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
                     p.row_tiles, p.parts, p.part_chunks, nullptr, nullptr};
  if (p.parts > 1) {
    a.arrivals = static_cast<int*>(workspace);
    a.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + counter_bytes(p));
  }
  const int heads = num_seqs * kv_heads;
  if (head_dim == 64) launch_for<64>(a, p, heads, stream);
  else launch_for<128>(a, p, heads, stream);
  return hipGetLastError();
}

}  // namespace lora
