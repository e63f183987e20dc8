// lora_kv_attention_mass: how much attention each cached token drew in a step, by key
// head, from the queries, the cached keys and the logarithms of the rows' sums that
// attention left:
//   drawn[t] = sum over the rows that see t of exp(scale * q . k_t - lse)
// added to what earlier steps left for the tokens before the queries, and put in the
// place of whatever was there for the queries' own.
//
// A wave takes 64 tokens of a key head and keeps their keys in registers as operands
// of the matrix unit; the rows come by in tiles of 16.  Lane (g, c) of a tile's scores
// has those of the tokens [16 g, 16 g + 16) for row c, so each lane adds up its
// sixteen tokens over the tiles, and the sixteen lanes of a group are joined once, at
// the end.  Every token has one writer: the sums are always taken in the same order.

#include "kv_attention.hpp"

namespace lora {

constexpr int kMassWaves = 4;

struct MassArgs {
  SumArgs a;
  float* mass;
};

// This lane's sixteen sums joined with those of its group's other lanes: lane (g, c)
// is left with the sum of token 16 g + c.  Each step halves the tokens a lane holds.
__device__ __forceinline__ float join_group(float (&v)[16]) {
  const int c = lane_id() & 15;
#pragma unroll
  for (int half = 8; half >= 1; half >>= 1) {
    const bool upper = (c & half) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float give = upper ? v[i] : v[i + half], keep = upper ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor(give, half);
    }
  }
  return v[0];
}

template <int D, int V>
__global__ __launch_bounds__(kMassWaves * kWave, 2) void kv_mass_kernel(MassArgs m) {
  const SumArgs& a = m.a;
  const int wave = wave_index(), lane = lane_id(), g = lane >> 4, c = lane & 15;
  const int kv_head = static_cast<int>(blockIdx.x);
  const int seq = sequence_at(a, static_cast<int>(blockIdx.z));
  RowTile t;
  if (!tile_of<V>(a, seq, 0, t, true)) return;
  const Reader<D> reader = reader_of<D>(a, seq, kv_head);
  const int length = t.before + t.queries;
  const int end = (length + kChunk - 1) / kChunk;

  __shared__ Draft drafts[V == kTree ? 64 * kDraftWords : 1];
  if constexpr (V == kTree) {
    stage_drafts(a, t, drafts, t.query1 + 1, kMassWaves * kWave);
    __syncthreads();
  }

  const int step = kMassWaves * static_cast<int>(gridDim.y);
  for (int chunk = t.first / kChunk + static_cast<int>(blockIdx.y) * kMassWaves + wave; chunk < end; chunk += step) {
    const int base = chunk * kChunk;
    const Pages pages = reader.pages(base);
    Keys<D> keys;
    reader.load(keys, pages, base);
    bf16x8 k[4][D / 32];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        k[j][i] = __builtin_bit_cast(bf16x8, word_to_bf16(keys.w[j][i], __uint_as_float(byte_scale(keys.scales, j))));

    // The rows that see some of the chunk.
    int from = 0, to = t.rows;
    if constexpr (V != kTree) {
      const int q0 = base - t.before;  // the first query that sees the chunk's first token
      from = q0 > t.query1 ? t.rows : (q0 > 0 ? q0 * a.group : 0);
      if (a.window) {
        const int64_t q1 = static_cast<int64_t>(base) + kChunk - 1 + a.window - t.before;  // and past the last
        to = q1 <= 0 ? 0 : (q1 * a.group < to ? static_cast<int>(q1 * a.group) : to);
      }
    }
    Span at;
    at.base = base;
    at.window = a.window;
    at.ok = pages.v >= 0;
    float sums[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) sums[i] = 0.f;
    for (int row0 = from & ~(kTile - 1); row0 < to; row0 += kTile) {
      const int query0 = row0 / a.group, head0 = row0 - query0 * a.group;
      const RowOf row = row_of(a, query0, head0, c);
      const bool there = row0 + c < t.rows;
      float lse = -INFINITY;
      bf16x8 q[D / 32];
      const int64_t token = t.start + (there ? row.query : 0);
      const int head = kv_head * a.group + (there ? row.head : 0);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        u32x4 w = load16(a.q + token * a.ldq + head * D + g * (D / 4) + 8 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] ^= a.sign;
        q[i] = __builtin_bit_cast(bf16x8, w);
      }
      lse = a.lse[token * a.ldl + head];
      f32x4 s[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < D / 32; ++i) s[j] = mfma(k[j][i], q[i], s[j]);
      }
      const bool counts = there && lse != -INFINITY;
      uint32_t seen = 0;
      if constexpr (V == kTree) seen = seen_bits(at, drafts[there ? row.query : 0], t.before);
      else seen = seen_bits(at, t.before + row.query);
      if (!counts) seen = 0;
      const float top = lse * 1.44269504f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = __builtin_amdgcn_exp2f(fmaf(s[j][i], a.scale_log2, -top));
          sums[4 * i + j] += seen >> (4 * i + j) & 1u ? p : 0.f;
        }
    }
    const float drawn = join_group(sums);
    const int token = base + lane;
    if (token < length && pages.v >= 0) {
      float* at_mass = m.mass + ((static_cast<int64_t>(pages.v) * a.cache.kv_heads + kv_head) << reader.shift) +
                       (token & ((1 << reader.shift) - 1));
      *at_mass = token >= t.before ? drawn : *at_mass + drawn;
    }
  }
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
                      fabsf(scale) * 1.44269504f, scale < 0.f ? 0x80008000u : 0u,
                      group, ((1 << 21) + group - 1) / group,
                      1, 1, 0, 0, nullptr, nullptr},
                      masks, words, const_cast<float*>(lse), ldl};
  m.mass = mass;
  const int64_t chunks = (static_cast<int64_t>(max_seq_len) + kChunk - 1) / kChunk;
  int64_t groups = (chunks + kMassWaves - 1) / kMassWaves;
  // enough workgroups to fill the device a few times over; beyond that each takes several chunks
  const int64_t most = (8 * kCus + static_cast<int64_t>(num_seqs) * kv_heads - 1) / (static_cast<int64_t>(num_seqs) * kv_heads);
  groups = groups < most ? groups : most;
  const dim3 grid(kv_heads, static_cast<unsigned>(groups), num_seqs), block(kMassWaves * kWave);
  if (masks) {
    if (head_dim == 64) hipLaunchKernelGGL((kv_mass_kernel<64, kTree>), grid, block, 0, stream, m);
    else hipLaunchKernelGGL((kv_mass_kernel<128, kTree>), grid, block, 0, stream, m);
  } else {
    if (head_dim == 64) hipLaunchKernelGGL((kv_mass_kernel<64, kPlain>), grid, block, 0, stream, m);
    else hipLaunchKernelGGL((kv_mass_kernel<128, kPlain>), grid, block, 0, stream, m);
  }
  return hipGetLastError();
}

}  // namespace lora
