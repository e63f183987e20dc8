// lora_rms_norm: residual addition, root-mean-square norm, bf16 and 8-bit
// outputs, one workgroup a row.
//
//   h = bf16(x + residual), v = h w / sqrt(mean h^2 + eps), y = bf16(v),
//   s = max(fp32(max|v| / 448), 2^-126), y8 = e4m3(v / s)
//
// The row stays in registers between the sum and the outputs, so each input is
// read once.  v is kept in 64 bits up to its one rounding to bf16 or (through
// fp32) to 8 bits: next to a border between two codes the result is then that
// of the formula.

#include "device_common.hpp"
#include "lora_attention.h"

namespace lora {

constexpr int kNormThreads = 256;
constexpr int kNormWaves = kNormThreads / kWave;
constexpr double kE4m3Max = 448.0;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126

struct NormArgs {
  const uint16_t* x;
  const uint16_t* residual;  // or nullptr
  const uint16_t* weight;
  uint16_t* sum;    // or nullptr
  uint16_t* y;      // or nullptr
  uint8_t* y8;      // or nullptr
  float* scales;    // with y8
  int64_t ldx, ldr, lds, ldy, ldy8;
  double eps;
  int hidden;
  int group;        // elements a scale; hidden: one a row
};

// Larger of two magnitudes; NaN if either is.
__device__ __forceinline__ double max_nan(double a, double b) { return a > b || a != a ? a : b; }

// C: chunks of 8 elements a thread.
template <int C>
__global__ __launch_bounds__(kNormThreads) void rms_norm_kernel(NormArgs a) {
  const int64_t row = blockIdx.x;
  const int tid = static_cast<int>(threadIdx.x);
  const int chunks = a.hidden >> 3;
  const bool per_row = a.group == a.hidden;
  u32x4 h[C];
  double sum = 0.0, top = 0.0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * kNormThreads + tid;
    if (i >= chunks) continue;
    h[c] = load16(a.x + row * a.ldx + 8 * i);
    if (a.residual) {
      const u32x4 r = load16(a.residual + row * a.ldr + 8 * i);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        h[c][k] = pack_bf16x2(bf16_lo(h[c][k]) + bf16_lo(r[k]), bf16_hi(h[c][k]) + bf16_hi(r[k]));
      if (a.sum) store16(a.sum + row * a.lds + 8 * i, h[c]);
    }
    const u32x4 w = load16(a.weight + 8 * i);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const double e = bf16_at(h[c], k);
      sum += e * e;
      top = max_nan(fabs(e * bf16_at(w, k)), top);
    }
  }
  __shared__ double part_sum[kNormWaves], part_top[kNormWaves];
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) {
    sum += __shfl_xor(sum, m);
    top = max_nan(__shfl_xor(top, m), top);
  }
  if (lane_id() == 0) {
    part_sum[tid / kWave] = sum;
    part_top[tid / kWave] = top;
  }
  __syncthreads();
  sum = 0.0;
  top = 0.0;
#pragma unroll
  for (int i = 0; i < kNormWaves; ++i) {
    sum += part_sum[i];
    top = max_nan(part_top[i], top);
  }
  const double r = 1.0 / sqrt(sum / a.hidden + a.eps);
  if (!a.y && !a.y8) return;

  float scale = static_cast<float>(top * r / kE4m3Max);
  scale = scale < kMinScale ? kMinScale : scale;
  if (a.y8 && per_row && tid == 0) a.scales[row] = scale;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * kNormThreads + tid;
    const bool in = i < chunks;
    double v[8];
    double big = 0.0;
    if (in) {
      const u32x4 w = load16(a.weight + 8 * i);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k] = static_cast<double>(bf16_at(h[c], k)) * bf16_at(w, k) * r;
        big = max_nan(fabs(v[k]), big);
      }
      if (a.y) {
        u32x4 o;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          o[k] = pack_bf16x2(static_cast<float>(v[2 * k]), static_cast<float>(v[2 * k + 1]));
        store16(a.y + row * a.ldy + 8 * i, o);
      }
    }
    if (!a.y8) continue;
    float s = scale;
    if (!per_row) {
      // a group is group / 8 neighbouring lanes (4 to 32), all inside the row or none
      for (int m = 1; m < (a.group >> 3); m <<= 1) big = max_nan(__shfl_xor(big, m), big);
      s = static_cast<float>(big / kE4m3Max);
      s = s < kMinScale ? kMinScale : s;
      if (in && (8 * i) % a.group == 0)
        a.scales[row * (a.hidden / a.group) + 8 * i / a.group] = s;
    }
    if (in) {
      const double inv = 1.0 / static_cast<double>(s);
      u32x2 o;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        int p = __builtin_amdgcn_cvt_pk_fp8_f32(static_cast<float>(v[4 * k] * inv),
                                                static_cast<float>(v[4 * k + 1] * inv), 0, false);
        p = __builtin_amdgcn_cvt_pk_fp8_f32(static_cast<float>(v[4 * k + 2] * inv),
                                            static_cast<float>(v[4 * k + 3] * inv), p, true);
        o[k] = static_cast<uint32_t>(p);
      }
      *(LORA_GLOBAL u32x2*)(a.y8 + row * a.ldy8 + 8 * i) = o;
    }
  }
}

hipError_t launch_rms_norm(const uint16_t* x, int64_t ldx, const uint16_t* residual, int64_t ldr,
                           const uint16_t* weight, double eps, int num_tokens, int hidden,
                           uint16_t* sum, int64_t lds, uint16_t* y, int64_t ldy, uint8_t* y8,
                           int64_t ldy8, float* scales, int group, hipStream_t stream) {
  const NormArgs a = {x, residual, weight, sum, y, y8, scales, ldx, ldr, lds, ldy, ldy8,
                      eps, hidden, group};
  const int need = (hidden / 8 + kNormThreads - 1) / kNormThreads;
  const dim3 grid(num_tokens), block(kNormThreads);
  if (need <= 1) rms_norm_kernel<1><<<grid, block, 0, stream>>>(a);
  else if (need <= 2) rms_norm_kernel<2><<<grid, block, 0, stream>>>(a);
  else if (need <= 4) rms_norm_kernel<4><<<grid, block, 0, stream>>>(a);
  else if (need <= 8) rms_norm_kernel<8><<<grid, block, 0, stream>>>(a);
  else if (need <= 16) rms_norm_kernel<16><<<grid, block, 0, stream>>>(a);
  else rms_norm_kernel<32><<<grid, block, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace lora
