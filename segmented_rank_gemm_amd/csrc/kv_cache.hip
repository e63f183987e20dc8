// lora_kv_append: rotate q and k by position, write q in bf16 and k and v into
// the 4-bit paged cache.  lora_kv_read: what the cache holds at given places.
//
// A thread takes 8 elements of a head (16 bytes of bf16, 4 bytes of codes); four
// neighbouring lanes share a 32-element block and its scale byte.

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

// The element of the rotated head at position e + k (k < 8), in fp32.  The
// products are exact in 64 bits (8 by 24 significant bits) and their sum is
// rounded there once, so the result is the formula's, rounded to fp32: what
// the codes are taken from lies on the right side of every border.
template <int D>
__device__ __forceinline__ void rotate(float out[8], const uint16_t* head, int e, u32x4 own,
                                       const float* angles, int rot_dim, int interleaved) {
  const int half = rot_dim >> 1;
#pragma unroll
  for (int k = 0; k < 8; ++k) out[k] = bf16_at(own, k);
  if (e >= rot_dim) return;
  if (interleaved) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const double a = bf16_at(own, 2 * k), b = bf16_at(own, 2 * k + 1);
      const double c = angles[(e >> 1) + k], s = angles[half + (e >> 1) + k];
      out[2 * k] = static_cast<float>(a * c - b * s);
      out[2 * k + 1] = static_cast<float>(b * c + a * s);
    }
    return;
  }
  const bool low = e < half;
  const int i = low ? e : e - half;
  const u32x4 other = load16(head + (low ? e + half : i));
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const double x = bf16_at(own, k), y = bf16_at(other, k);
    const double c = angles[i + k], s = angles[half + i + k];
    out[k] = static_cast<float>(low ? x * c - y * s : x * c + y * s);
  }
}

template <int D>
__global__ __launch_bounds__(kKvThreads) void kv_append_kernel(AppendArgs a) {
  const int64_t token = blockIdx.x;
  int position = 0;
  if (a.rot_dim) {
    position = a.positions[token];
    if (position < 0 || position >= a.rope_rows) return;  // the whole workgroup
  }
  const int64_t slot = a.slots[token];
  const bool kept = slot >= 0 && slot < (static_cast<int64_t>(a.cache.num_pages) << a.cache.page_shift);
  const float* angles = a.rope + static_cast<int64_t>(position) * a.rot_dim;
  constexpr int kChunks = D / 8;  // of a head
  const int heads = a.q_heads + (kept ? 2 * a.kv_heads : 0);
  const int items = heads * kChunks;
  for (int item = static_cast<int>(threadIdx.x); item < items; item += kKvThreads) {
    const int head = item / kChunks;
    const int e = (item % kChunks) * 8;
    const uint16_t* src = a.qkv + token * a.ldqkv + head * D;
    const u32x4 own = load16(src + e);
    const bool value = head >= a.q_heads + a.kv_heads;
    float v[8];
    rotate<D>(v, src, e, own, angles, value ? 0 : a.rot_dim, a.interleaved);
    if (head < a.q_heads) {
      u32x4 o;
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
      store16(a.q_out + token * a.ldq + head * D + e, o);
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
    const int page = static_cast<int>(slot >> a.cache.page_shift);
    const int at = static_cast<int>(slot & (a.cache.page_size() - 1));
    uint8_t* block = a.cache.template block<D>(page, value ? 1 : 0, kv_head);
    *(LORA_GLOBAL uint32_t*)(block + at * (D / 2) + e / 2) = codes;
    if (e % kBlock == 0)
      block[a.cache.template scales_at<D>() + ((e / kBlock) << a.cache.page_shift) + at] =
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
  for (int item = static_cast<int>(threadIdx.x); item < items; item += kKvThreads) {
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

hipError_t launch_kv_append(const uint16_t* qkv, int64_t ldqkv, const int32_t* positions,
                            const int64_t* slots, const float* rope, int rope_rows, int rot_dim,
                            int interleaved, int num_tokens, int q_heads, int kv_heads,
                            int head_dim, uint16_t* q_out, int64_t ldq, uint8_t* cache,
                            int num_pages, int page_shift, hipStream_t stream) {
  const AppendArgs a = {qkv, positions, slots, rope, q_out,
                        {cache, num_pages, page_shift, kv_heads},
                        ldqkv, ldq, rope_rows, rot_dim, interleaved, q_heads, kv_heads};
  const dim3 grid(num_tokens), block(kKvThreads);
  if (head_dim == 64) kv_append_kernel<64><<<grid, block, 0, stream>>>(a);
  else kv_append_kernel<128><<<grid, block, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv_read(const int64_t* slots, int num_tokens, int kv_heads, int head_dim,
                          const uint8_t* cache, int num_pages, int page_shift, uint16_t* k_out,
                          int64_t ldk, uint16_t* v_out, int64_t ldv, hipStream_t stream) {
  const Cache<const uint8_t> c = {cache, num_pages, page_shift, kv_heads};
  const dim3 grid(num_tokens), block(kKvThreads);
  if (head_dim == 64) kv_read_kernel<64><<<grid, block, 0, stream>>>(slots, c, k_out, ldk, v_out, ldv);
  else kv_read_kernel<128><<<grid, block, 0, stream>>>(slots, c, k_out, ldk, v_out, ldv);
  return hipGetLastError();
}

}  // namespace lora
