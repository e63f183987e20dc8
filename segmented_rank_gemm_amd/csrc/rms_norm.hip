// lora_rms_norm: residual addition, root-mean-square norm, bf16 and 8-bit
// outputs, one workgroup a row.
//
//   h = bf16(x + residual), v = h w / sqrt(mean h^2 + eps), y = bf16(v),
//   s = max(fp32(max|v| / 448), 2^-126), y8 = e4m3(v / s)
//
// The row stays in registers between the sum and the outputs, so each input is
// read once.  Up to its one rounding to bf16 (through fp32) or 8 bits v carries
// about 46 bits: next to a border between two codes the result is then that of the
// formula.  h w is exact in fp32 (8 by 8 significant bits; rows with a product below
// the normal numbers take the other way); it is multiplied by a factor held as the
// sum of two fp32 numbers, which costs four operations where
// 64-bit arithmetic takes a multiplication and two conversions at a quarter of
// the rate (1001 rows of 11008: 20.4 us then, 14.8 now, the borders' care in it).
// Only the sum of squares is in 64 bits.
//
// Bound by: HBM for long batches (8192 rows of 8192 with residual, sum, bf16 and 8
// bits: 111 us, 5.4 TB/s, where this library's copy reaches 5.5); where one row a
// workgroup leaves each wave a few hundred elements, by the steps one after another
// (load, sum, scale, store).

#include "device_common.hpp"
#include "lora_attention.h"

namespace lora {

constexpr double kE4m3Max = 448.0;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126
constexpr uint32_t kInfinity = 0x7F800000u;
constexpr int kSubnormal = 0x90;  // of the classes of fp32 numbers: both signs' subnormal ones

struct NormArgs {
  const uint16_t* x;
  const uint16_t* residual;  // or nullptr
  const uint16_t* weight;
  uint16_t* sum;    // or nullptr
  uint16_t* y;      // or nullptr
  uint8_t* y8;      // or nullptr
  float* scales;    // with y8
  int64_t ldx, ldr, lds, ldy, ldy8;
  double eps, inv_hidden;
  int hidden;
  int group;        // elements a scale; hidden: one a row
  int group_shift;  // log2 of the chunks of 8 a group, where there are several groups
};

// Larger of two magnitudes; NaN if either is.
__device__ __forceinline__ double max_nan(double a, double b) { return a > b || a != a ? a : b; }

// A factor as the sum of two fp32 numbers, and a product with it to about 46
// bits.  Holds while neither part nor the product leaves fp32's normal range: for
// factors in [2^-60, 2^60].
struct Factor {
  float high, low;
};
__device__ __forceinline__ Factor factor(double f) {
  const float high = static_cast<float>(f);
  return Factor{high, static_cast<float>(f - static_cast<double>(high))};
}
// The product rounded to fp32.
__device__ __forceinline__ float times(float p, Factor f) {
#pragma clang fp contract(off)  // `high` has to be the same rounded number in all three places
  const float high = p * f.high;
  return high + fmaf(p, f.low, fmaf(p, f.high, -high));
}

// A number `high + low` (|low| at most half a step of high) as the fp32 number that
// rounds to 8 bits as the sum does: of the two neighbours, where it is neither, the
// odd one.  The nearest one will not do: h w and the row's largest are numbers of
// few bits, so their quotients lie on borders between codes (within 2^-24, the
// rounding of the scale) thousands of times as often as by chance, and a first
// rounding onto the border would send them to the even side.
__device__ __forceinline__ float odd(float high, float low) {
  const uint32_t bits = __float_as_uint(high);
  const bool away = (__float_as_uint(low) ^ bits) >> 31 == 0;  // low points away from zero
  const uint32_t moved = away ? bits + 1 : bits - 1;
  return __uint_as_float(low != 0.f && (bits & 1) == 0 ? moved : bits);
}
__device__ __forceinline__ float times_odd(float p, Factor f) {
#pragma clang fp contract(off)
  const float first = p * f.high;
  const float rest = fmaf(p, f.low, fmaf(p, f.high, -first));
  const float high = first + rest;
  return odd(high, rest - (high - first));
}
__device__ __forceinline__ float to_odd(double v) {
  const float high = static_cast<float>(v);
  // past fp32, infinite or NaN there is no rest
  return fabsf(high) < INFINITY ? odd(high, static_cast<float>(v - high)) : high;
}

// Largest of the magnitudes' bits over 1 << shift (2 to 5) neighbouring lanes, on
// data-parallel moves inside 16 lanes.  All lanes of the wave take part.
template <int kCtrl>
__device__ __forceinline__ uint32_t max_with(uint32_t v) {
  const int other = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), kCtrl, 0xF, 0xF, false);
  return max(v, static_cast<uint32_t>(other));
}
__device__ __forceinline__ uint32_t group_max(uint32_t v, int shift) {
  v = max_with<0xB1>(v);                   // the other of each two lanes
  v = max_with<0x4E>(v);                   // the other two of each four
  if (shift > 2) v = max_with<0x141>(v);   // eight, mirrored
  if (shift > 3) v = max_with<0x140>(v);   // sixteen, mirrored
  if (shift > 4) v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), 16)));
  return v;
}

// 1 / sqrt(x) to about 50 bits: the hardware's estimate and two Newton steps, a
// third of what a division and a root cost every thread.  0, infinity and NaN
// give what the estimate gives.
__device__ __forceinline__ double inverse_root(double x) {
  const double first = __builtin_amdgcn_rsq(x);
  double r = first;
#pragma unroll
  for (int i = 0; i < 2; ++i) r = fma(0.5 * r, fma(-x * r, r, 1.0), r);
  return r == r ? r : first;
}

// 1 / s for a normal fp32 number s in [2^-126, 2^125], to about 45 bits.
__device__ __forceinline__ double inverse(float s) {
  const double x = __builtin_amdgcn_rcpf(s);
  return fma(x, fma(-x, s, 1.0), x);
}

__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  int q = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  q = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, q, true);
  return static_cast<uint32_t>(q);
}

// A thread's part of a row: C chunks of 8 elements, T (threads of the row) apart.
template <int T, int C>
struct NormRow {
  u32x4 h[C];
  int chunks;     // of the row
  bool per_row;   // one scale
  double r;       // 1 / sqrt(mean h^2 + eps)

  __device__ __forceinline__ static int at(int c) {
    return c * T + static_cast<int>(threadIdx.x);
  }
  // Past the row's end, its last chunk: loads need no condition.
  __device__ __forceinline__ int load_at(int c) const { return at(c) < chunks ? at(c) : chunks - 1; }
  // No lane of this wave has a chunk c.
  __device__ __forceinline__ bool past(int c) const { return at(c) - lane_id() >= chunks; }
};

// The outputs where h w, its factors and v stay well inside fp32's range; top: the
// largest |h w| of the row.
template <int T, int C>
__device__ __forceinline__ void emit(const NormArgs& a, const NormRow<T, C>& n, int64_t row, double top) {
  // The weights again (from the L1 cache), all of them before the first output: a
  // load's wait counts the stores before it.
  u32x4 w[C];
#pragma unroll
  for (int c = 0; c < C; ++c) w[c] = load16(a.weight + 8 * n.load_at(c));
  const Factor to_v = factor(n.r);
  const double per_scale = n.r * (1.0 / kE4m3Max);
  float s = static_cast<float>(top * per_scale);
  s = s < kMinScale ? kMinScale : s;
  double code = n.r * inverse(s);  // what turns h w into the number that is coded
  if (a.y8 && n.per_row && threadIdx.x == 0) a.scales[row] = s;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (n.past(c)) break;
    const int i = n.at(c);
    const bool in = i < n.chunks;
    float p[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = bf16_at(n.h[c], k) * bf16_at(w[c], k);
    if (a.y && in) {
      u32x4 o;
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = pack_bf16x2(times(p[2 * k], to_v), times(p[2 * k + 1], to_v));
      store16(a.y + row * a.ldy + 8 * i, o);
    }
    if (!a.y8) continue;
    if (!n.per_row) {
      // a group is 4 to 32 neighbouring lanes, all inside the row or none
      uint32_t bits = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) bits = max(bits, __float_as_uint(p[k]) & 0x7FFFFFFFu);
      bits = group_max(bits, a.group_shift);
      s = static_cast<float>(__uint_as_float(bits) * per_scale);
      s = s < kMinScale ? kMinScale : s;
      code = n.r * inverse(s);
      if (in && (i & ((1 << a.group_shift) - 1)) == 0)
        a.scales[row * (n.chunks >> a.group_shift) + (i >> a.group_shift)] = s;
    }
    if (!in) continue;
    // Only where the nearest fp32 number is itself a border between two codes (its
    // last 20 bits, a one and zeros; or something below 2^-6, where they are others)
    // does it matter on which side of it the product is.
    const Factor f = factor(code);
    float u[8];
    uint32_t border = ~0u, least = ~0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      u[k] = times(p[k], f);
      const uint32_t bits = __float_as_uint(u[k]);
      border = min(border, (bits & 0xFFFFFu) ^ 0x80000u);
      least = min(least, bits & 0x7FFFFFFFu);
    }
    if (!(code >= 0x1p-60 && code <= 0x1p60)) {
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = to_odd(p[k] * code);
    } else if (border == 0 || least < __float_as_uint(0x1p-6f)) {
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = times_odd(p[k], f);
    }
    *(LORA_GLOBAL u32x2*)(a.y8 + row * a.ldy8 + 8 * i) =
        u32x2{pack_e4m3x4(u[0], u[1], u[2], u[3]), pack_e4m3x4(u[4], u[5], u[6], u[7])};
  }
}

// The outputs of any other row (very large or very small ones, infinities, NaN):
// everything in 64 bits, nothing for speed.  shared: (T / kWave) numbers that all
// threads are done with.
template <int T, int C>
__device__ __forceinline__ void emit_wide(const NormArgs& a, const NormRow<T, C>& n, int64_t row,
                                       double* shared) {
  auto v = [&](u32x4 h, u32x4 w, int k) {
    return static_cast<double>(bf16_at(h, k)) * bf16_at(w, k) * n.r;
  };
  auto largest = [&](int c) {
    double big = 0.0;
    const int i = n.at(c);
    if (i < n.chunks) {
      const u32x4 w = load16(a.weight + 8 * i);
#pragma unroll
      for (int k = 0; k < 8; ++k) big = max_nan(fabs(v(n.h[c], w, k)), big);
    }
    return big;
  };
  double row_top = 0.0;
  if (n.per_row) {
#pragma unroll
    for (int c = 0; c < C; ++c) row_top = max_nan(largest(c), row_top);
    for (int m = 1; m < kWave; m <<= 1) row_top = max_nan(__shfl_xor(row_top, m), row_top);
    if (lane_id() == 0) shared[threadIdx.x / kWave] = row_top;
    __syncthreads();
    row_top = 0.0;
    for (int i = 0; i < (T / kWave); ++i) row_top = max_nan(shared[i], row_top);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = n.at(c);
    const bool in = i < n.chunks;
    double top = row_top;
    if (!n.per_row) {
      top = largest(c);
      for (int m = 1; m < 1 << a.group_shift; m <<= 1) top = max_nan(__shfl_xor(top, m), top);
    }
    if (!in) continue;
    float s = static_cast<float>(top / kE4m3Max);
    s = s < kMinScale ? kMinScale : s;
    const u32x4 w = load16(a.weight + 8 * i);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const double e = v(n.h[c], w, k);
      const float u = to_odd(e / s);
      if (a.y)
        a.y[row * a.ldy + 8 * i + k] = static_cast<uint16_t>(pack_bf16x2(static_cast<float>(e), 0.f));
      if (a.y8) a.y8[row * a.ldy8 + 8 * i + k] = static_cast<uint8_t>(pack_e4m3x4(u, u, u, u));
    }
    if (!a.y8) continue;
    if (n.per_row ? i == 0 : (i & ((1 << a.group_shift) - 1)) == 0)
      a.scales[n.per_row ? row : row * (n.chunks >> a.group_shift) + (i >> a.group_shift)] = s;
  }
}

template <int T, int C>
__global__ __launch_bounds__(T) void rms_norm_kernel(NormArgs a) {
  const int64_t row = blockIdx.x;
  const int tid = static_cast<int>(threadIdx.x);
  NormRow<T, C> n;
  n.chunks = a.hidden >> 3;
  n.per_row = a.group == a.hidden;
  // All of the row's loads go out before the first is waited for.
  u32x4 res[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = n.at(c);
    n.h[c] = u32x4{0, 0, 0, 0};
    res[c] = u32x4{0, 0, 0, 0};
    if (i >= n.chunks) continue;
    n.h[c] = load16(a.x + row * a.ldx + 8 * i);
    if (a.residual) res[c] = load16(a.residual + row * a.ldr + 8 * i);
  }
  double sum = 0.0;
  float top = 0.f;  // the largest |h w|, NaN if one is
  bool subnormal = false;  // some h w has lost bits
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = n.at(c);
    if (i >= n.chunks) continue;
    const u32x4 w = load16(a.weight + 8 * i);
    if (a.residual) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        n.h[c][k] = pack_bf16x2(bf16_lo(n.h[c][k]) + bf16_lo(res[c][k]),
                                bf16_hi(n.h[c][k]) + bf16_hi(res[c][k]));
      if (a.sum) store16(a.sum + row * a.lds + 8 * i, n.h[c]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float e = bf16_at(n.h[c], k);
      const double e64 = e;
      sum = fma(e64, e64, sum);
      const float p = e * bf16_at(w, k);
      top = __builtin_elementwise_maximum(top, fabsf(p));
      subnormal |= __builtin_amdgcn_classf(p, kSubnormal);
    }
  }
  // its bits: integer order, infinity and NaN on top
  uint32_t top_bits = subnormal ? kInfinity : __float_as_uint(top) & 0x7FFFFFFFu;
  __shared__ double part_sum[(T / kWave)];
  __shared__ uint32_t part_top[(T / kWave)];
  __shared__ double spare[(T / kWave)];
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) {
    sum += __shfl_xor(sum, m);
    top_bits = max(top_bits, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top_bits), m)));
  }
  if (lane_id() == 0) {
    part_sum[tid / kWave] = sum;
    part_top[tid / kWave] = top_bits;
  }
  __syncthreads();
  sum = 0.0;
  top_bits = 0;
#pragma unroll
  for (int i = 0; i < (T / kWave); ++i) {
    sum += part_sum[i];
    top_bits = max(top_bits, part_top[i]);
  }
  if (!a.y && !a.y8) return;
  n.r = inverse_root(fma(sum, a.inv_hidden, a.eps));
  // The same for all threads of the row.  The last bound keeps v, and the scales with
  // their inverses, inside fp32's normal numbers, however large the weights.
  if (top_bits < kInfinity && n.r >= 0x1p-60 && n.r <= 0x1p10 &&
      __uint_as_float(top_bits) * n.r <= 0x1p120)
    emit<T, C>(a, n, row, __uint_as_float(top_bits));
  else
    emit_wide<T, C>(a, n, row, spare);
}

// T threads a row, the first of C, More... that holds a thread's chunks.
template <int T, int C, int... More>
static void launch(const NormArgs& a, int chunks, int rows, hipStream_t stream) {
  if constexpr (sizeof...(More) > 0) {
    if (chunks > C) return launch<T, More...>(a, chunks, rows, stream);
  }
  hipLaunchKernelGGL((rms_norm_kernel<T, C>), dim3(rows), dim3(T), 0, stream, a);
}

hipError_t launch_rms_norm(const uint16_t* x, int64_t ldx, const uint16_t* residual, int64_t ldr,
                           const uint16_t* weight, double eps, int num_tokens, int hidden,
                           uint16_t* sum, int64_t lds, uint16_t* y, int64_t ldy, uint8_t* y8,
                           int64_t ldy8, float* scales, int group, hipStream_t stream) {
  const NormArgs a = {x, residual, weight, sum, y, y8, scales, ldx, ldr, lds, ldy, ldy8,
                      eps, 1.0 / hidden, hidden, group, group < hidden ? __builtin_ctz(group / 8) : 0};
  const int chunks = hidden / 8;
  // Threads a row: enough that a thread has few chunks, and no more, since idle
  // waves cost their launch (us, 64 / 256 / 512 / 1024 threads: 8192 rows of 512
  // 10.9 / 16.7 / 27.3 / 52.9; 2048 of 4096 - / 15.9 / 16.9 / 21.5; 16 of 8192
  // - / 6.5 / 5.1 / 5.2; 8192 of 8192 - / 116 / 111 / 117).
  if (hidden <= 1024) launch<64, 1, 2>(a, (chunks + 63) / 64, num_tokens, stream);
  else if (hidden <= 4096) launch<256, 1, 2>(a, (chunks + 255) / 256, num_tokens, stream);
  else if (hidden <= 32768) launch<512, 2, 4, 8>(a, (chunks + 511) / 512, num_tokens, stream);
  else launch<1024, 8>(a, (chunks + 1023) / 1024, num_tokens, stream);
  return hipGetLastError();
}

}  // namespace lora
