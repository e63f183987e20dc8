// The 4-bit paged cache as the kernels see it: addresses of one page of one
// head, and the conversions between its codes and numbers (see lora_attention.h
// for the layout).
#pragma once

#include "device_common.hpp"
#include "lora_attention.h"

namespace lora {

constexpr int kBlock = 32;        // elements that share a scale byte
constexpr int kScaleBias = 127;   // scale byte b stands for 2^(b - 127)
constexpr int kScaleNan = 255;
// Scale exponents stay in [-125, 125], so that the smallest non-zero element
// (0.5 * 2^-125) is a normal bf16 number and the largest (6 * 2^125) a finite one.
constexpr int kMinExponent = -125;
constexpr int kMaxExponent = 125;

// One cache: page_size is a power of two.
template <typename Byte>
struct Cache {
  Byte* data;
  int num_pages;
  int page_shift;  // log2(page_size)
  int kv_heads;

  __device__ __forceinline__ int page_size() const { return 1 << page_shift; }
  // First byte of a page's keys (part 0) or values (part 1) of one head.
  template <int D>
  __device__ __forceinline__ Byte* block(int page, int part, int head) const {
    const int64_t bytes = static_cast<int64_t>(D / 2 + D / kBlock) << page_shift;
    return data + ((static_cast<int64_t>(page) * 2 + part) * kv_heads + head) * bytes;
  }
  // Offset of the scales inside such a block.
  template <int D>
  __device__ __forceinline__ int scales_at() const { return (D / 2) << page_shift; }
};

// A scale byte as the scale operand of the conversions below, which take its
// exponent: 2^(b - 127), and NaN for b = 255 (an infinity here).
__device__ __forceinline__ float scale_value(uint32_t b) { return __uint_as_float(b << 23); }

// Scale byte of a block whose largest magnitude is `largest` (fp32, not NaN or
// infinite): the smallest e in [-125, 125] with largest <= 7 * 2^e.  Magnitudes
// above 6 * 2^e then lose at most what the top step (4 to 6) loses anyway.
__device__ __forceinline__ uint32_t scale_byte(float largest) {
  const uint32_t bits = __float_as_uint(largest);
  // largest = 1.m * 2^E: e = E - 2, and one more where 1.m > 7/4
  int e = static_cast<int>(bits >> 23) - kScaleBias - 2 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < kMinExponent ? kMinExponent : (e > kMaxExponent ? kMaxExponent : e);
  return static_cast<uint32_t>(e + kScaleBias);
}

// Codes 2 S and 2 S + 1 of a word times a scale, as two bf16: exact (one
// significant bit after the first, times a power of two).
template <int S>
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, S));
}

// All eight of them.
__device__ __forceinline__ u32x4 word_to_bf16(uint32_t w, float scale) {
  return u32x4{codes_to_bf16<0>(w, scale), codes_to_bf16<1>(w, scale), codes_to_bf16<2>(w, scale),
               codes_to_bf16<3>(w, scale)};
}

}  // namespace lora
