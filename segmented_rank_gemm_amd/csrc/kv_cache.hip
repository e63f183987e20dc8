// lora_kv_append: rotate q and k by position, write q in bf16 and k and v into
// the 4-bit paged cache.  lora_kv_read: what the cache holds at given places.
//
// A thread takes 8 elements of a head (16 bytes of bf16, 4 bytes of codes); four
// neighbouring lanes share a 32-element block and its scale byte.
//
// Bound by: HBM and, for the rotation, the 64-bit conversions beside it (4096
// tokens of 32 and 32 heads of 128: append 39 us, 3.9 TB/s, read 18 us, 4.7 TB/s,
// where this library's copy reaches 5.5; 64 tokens of 64 and 8 heads 2.9 and 2.0 us,
// of which an empty launch is 1.9).

#include "kv_format.hpp"

namespace lora {

constexpr int kKvThreads = 256;

struct AppendArgs {
  const uint16_t* qkv;
  const int32_t* positions;
  const int64_t* slots;
  const float* rope;
  uint16_t* q_out;
  Cache<uint8_t> cache;
  int64_t ldqkv, ldq;
  int rope_rows, rot_dim, interleaved;
  int q_heads, kv_heads;
};

// The codes of v / scale, element 0 in the lowest bits: the nearest of 0, 0.5, 1,
// 1.5, 2, 3, 4, 6, ties to the even code, and 6 for more (the hardware's rounding).
__device__ __forceinline__ uint32_t to_codes(const float v[8], float scale) {
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0, v[0], v[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
}

// A thread's place in every head that it takes: the elements e .. e + 7.
struct Place {
  int e;
  bool turned;  // rotated: by the angles below, one an element (pairs rot_dim / 2
  int partner;  // apart: `partner` is where the others are) or, the first four,
  double cos[8], sin[8];  // one for two neighbours
};

// Eight rotated elements, in fp32; `other` are their partners, where those are
// not neighbours.  The products are exact in 64 bits (8 by 24 significant bits)
// and their sum is rounded there once, so the result is the formula's, rounded to
// fp32: what the codes are taken from lies on the right side of every border.
__device__ __forceinline__ void rotate(float out[8], u32x4 own, u32x4 other, const Place& p,
                                       bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const double a = bf16_at(own, 2 * k), b = bf16_at(own, 2 * k + 1);
      out[2 * k] = static_cast<float>(a * p.cos[k] - b * p.sin[k]);
      out[2 * k + 1] = static_cast<float>(b * p.cos[k] + a * p.sin[k]);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    // sin is negative where these are a pair's first elements
    const double a = bf16_at(own, k), b = bf16_at(other, k);
    out[k] = static_cast<float>(a * p.cos[k] + b * p.sin[k]);
  }
}

// One workgroup a token, or several where tokens are few.  A thread keeps its
// place in the head and takes every (threads / (D / 8))-th head, so that a
// position's angles are loaded and widened once; the next head is on its way
// while one is worked on.
template <int D>
__global__ __launch_bounds__(kKvThreads) void kv_append_kernel(AppendArgs a) {
  constexpr int kChunks = D / 8;  // of a head
  const int64_t token = blockIdx.x;
  const int64_t slot = a.slots[token];
  Place p;
  p.e = (static_cast<int>(threadIdx.x) % kChunks) * 8;
  p.turned = p.e < a.rot_dim;
  p.partner = p.e;
  if (a.rot_dim) {
    const int position = a.positions[token];
    if (position < 0 || position >= a.rope_rows) return;  // the whole workgroup
    if (p.turned) {
      const int half = a.rot_dim >> 1;
      const bool low = p.e < half;
      const int first = a.interleaved ? p.e >> 1 : (low ? p.e : p.e - half);
      if (!a.interleaved) p.partner = low ? p.e + half : p.e - half;
      const float* angles = a.rope + static_cast<int64_t>(position) * a.rot_dim + first;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (k == 1 && a.interleaved) break;
        const u32x4 c = load16(angles + 4 * k), s = load16(angles + half + 4 * k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p.cos[4 * k + i] = __uint_as_float(c[i]);
          const double sine = __uint_as_float(s[i]);
          p.sin[4 * k + i] = low && !a.interleaved ? -sine : sine;
        }
      }
    }
  }
  const bool kept = slot >= 0 && slot < (static_cast<int64_t>(a.cache.num_pages) << a.cache.page_shift);
  const int page = static_cast<int>(slot >> a.cache.page_shift);
  const int at = static_cast<int>(slot & (a.cache.page_size() - 1));
  const int heads = a.q_heads + (kept ? 2 * a.kv_heads : 0);
  const int step = static_cast<int>(gridDim.y) * (kKvThreads / kChunks);
  int head = (static_cast<int>(blockIdx.y) * kKvThreads + static_cast<int>(threadIdx.x)) / kChunks;
  const uint16_t* row = a.qkv + token * a.ldqkv;
  // (without conditions, so that a head's use waits for its own loads only; past
  // the last head, and for partners that are not needed, what is there is loaded)
  u32x4 own, other;
  auto load = [&](int h) {
    const uint16_t* src = row + (h < heads ? h : heads - 1) * D;
    own = load16(src + p.e);
    other = load16(src + p.partner);
  };
  load(head);
  for (; head < heads; head += step) {
    const u32x4 now = own, now_other = other;
    load(head + step);
    const bool value = head >= a.q_heads + a.kv_heads;
    float v[8];
    if (p.turned && !value) {
      rotate(v, now, now_other, p, a.interleaved);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = bf16_at(now, k);
    }
    if (head < a.q_heads) {
      u32x4 o;
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
      store16(a.q_out + token * a.ldq + head * D + p.e, o);
      continue;
    }
    // The four lanes of a block are all in this branch: a head has whole blocks.
    uint32_t bits = 0;  // of the largest magnitude; integer order, infinity and NaN on top
#pragma unroll
    for (int k = 0; k < 8; ++k) bits = max(bits, __float_as_uint(v[k]) & 0x7FFFFFFFu);
    bits = max(bits, static_cast<uint32_t>(__shfl_xor(static_cast<int>(bits), 1)));
    bits = max(bits, static_cast<uint32_t>(__shfl_xor(static_cast<int>(bits), 2)));
    const bool finite = bits < 0x7F800000u;
    const uint32_t sb = finite ? scale_byte(__uint_as_float(bits)) : kScaleNan;
    const uint32_t codes = finite ? to_codes(v, scale_value(sb)) : 0u;
    const int kv_head = head - a.q_heads - (value ? a.kv_heads : 0);
    uint8_t* block = a.cache.template block<D>(page, value ? 1 : 0, kv_head);
    *(LORA_GLOBAL uint32_t*)(block + at * (D / 2) + p.e / 2) = codes;
    if (p.e % kBlock == 0)
      block[a.cache.template scales_at<D>() + ((p.e / kBlock) << a.cache.page_shift) + at] =
          static_cast<uint8_t>(sb);
  }
}

template <int D>
__global__ __launch_bounds__(kKvThreads) void kv_read_kernel(const int64_t* slots,
                                                             Cache<const uint8_t> cache,
                                                             uint16_t* k_out, int64_t ldk,
                                                             uint16_t* v_out, int64_t ldv) {
  const int64_t token = blockIdx.x;
  const int64_t slot = slots[token];
  const bool held = slot >= 0 && slot < (static_cast<int64_t>(cache.num_pages) << cache.page_shift);
  const int page = held ? static_cast<int>(slot >> cache.page_shift) : 0;
  const int at = held ? static_cast<int>(slot & (cache.page_size() - 1)) : 0;
  constexpr int kChunks = D / 8;
  const int items = 2 * cache.kv_heads * kChunks;
  const int step = static_cast<int>(gridDim.y) * kKvThreads;
  for (int item = static_cast<int>(blockIdx.y) * kKvThreads + static_cast<int>(threadIdx.x);
       item < items; item += step) {
    const int head = item / kChunks;
    const int e = (item % kChunks) * 8;
    const int part = head >= cache.kv_heads ? 1 : 0;
    const int kv_head = head - part * cache.kv_heads;
    uint16_t* out = part ? v_out : k_out;
    if (!out) continue;
    u32x4 o = {0, 0, 0, 0};
    if (held) {
      const uint8_t* block = cache.template block<D>(page, part, kv_head);
      const uint32_t codes = *(const LORA_GLOBAL uint32_t*)(block + at * (D / 2) + e / 2);
      const uint32_t sb =
          block[cache.template scales_at<D>() + ((e / kBlock) << cache.page_shift) + at];
      o = word_to_bf16(codes, scale_value(sb));
    }
    store16(out + token * (part ? ldv : ldk) + kv_head * D + e, o);
  }
}

// Workgroups a token: one where the tokens alone fill the device, up to one
// pass over a token's items where they do not (1 token of 32 and 32 heads: append
// 4.5 -> 2.4 us, read 2.6 -> 1.9).
static int groups_of(int num_tokens, int items) {
  const int most = (items + kKvThreads - 1) / kKvThreads;
  const int want = (2 * kCus + num_tokens - 1) / num_tokens;
  return want < most ? want : most;
}

hipError_t launch_kv_append(const uint16_t* qkv, int64_t ldqkv, const int32_t* positions,
                            const int64_t* slots, const float* rope, int rope_rows, int rot_dim,
                            int interleaved, int num_tokens, int q_heads, int kv_heads,
                            int head_dim, uint16_t* q_out, int64_t ldq, uint8_t* cache,
                            int num_pages, int page_shift, hipStream_t stream) {
  const AppendArgs a = {qkv, positions, slots, rope, q_out,
                        {cache, num_pages, page_shift, kv_heads},
                        ldqkv, ldq, rope_rows, rot_dim, interleaved, q_heads, kv_heads};
  const dim3 grid(num_tokens, groups_of(num_tokens, (q_heads + 2 * kv_heads) * (head_dim / 8)));
  const dim3 block(kKvThreads);
  if (head_dim == 64) kv_append_kernel<64><<<grid, block, 0, stream>>>(a);
  else kv_append_kernel<128><<<grid, block, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv_read(const int64_t* slots, int num_tokens, int kv_heads, int head_dim,
                          const uint8_t* cache, int num_pages, int page_shift, uint16_t* k_out,
                          int64_t ldk, uint16_t* v_out, int64_t ldv, hipStream_t stream) {
  const Cache<const uint8_t> c = {cache, num_pages, page_shift, kv_heads};
  const dim3 grid(num_tokens, groups_of(num_tokens, 2 * kv_heads * (head_dim / 8)));
  const dim3 block(kKvThreads);
  if (head_dim == 64) kv_read_kernel<64><<<grid, block, 0, stream>>>(slots, c, k_out, ldk, v_out, ldv);
  else kv_read_kernel<128><<<grid, block, 0, stream>>>(slots, c, k_out, ldk, v_out, ldv);
  return hipGetLastError();
}

}  // namespace lora
