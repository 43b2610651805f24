// Bias, activation and residual in the epilogue of a product:
//   y = bf16_RNE( act(v + bias[n]) + residual[m, n] ),   v the product in FP32.
// Everything between the FP32 accumulator and the one rounding to BF16 is FP32.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

namespace nvq {

enum : uint32_t { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

struct EpiParams {
  const __nv_bfloat16* bias;       // [N] or NULL
  const __nv_bfloat16* residual;   // [M, N] with row stride ldr, or NULL
  size_t ldr, ldy;                 // row strides in elements
  uint32_t act;
};

// v / (1 + 2^t) = v * sigmoid(-t ln 2), by the hardware's approximate power of two and
// reciprocal (two units in the last place together).  Rounding t costs |t| 2^-24: about
// 1e-5 relative where the result has not vanished next to 1e-36, far inside the 2^-9 of
// the BF16 rounding that follows.  2^t = inf gives 0, the limit.
__device__ __forceinline__ float over_one_plus_exp2(float v, float t) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return v * r;
}
constexpr float kNegLog2E = -1.4426950408889634f;
// v * sigmoid(s)
__device__ __forceinline__ float times_sigmoid(float v, float s) { return over_one_plus_exp2(v, s * kNegLog2E); }

template <uint32_t ACT>
__device__ __forceinline__ float activate_as(float v) {
  if constexpr (ACT == kActRelu) return v < 0.f ? 0.f : v;                        // NaN stays NaN
  if constexpr (ACT == kActGelu) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
  // 0.5 (1 + tanh(z)) = sigmoid(2 z), z = sqrt(2 / pi) (v + 0.044715 v^3)
  if constexpr (ACT == kActGeluTanh) {
    constexpr float a = kNegLog2E * 1.5957691216057308f, b = a * 0.044715f;
    return over_one_plus_exp2(v, v * __fmaf_rn(b, v * v, a));
  }
  if constexpr (ACT == kActSilu) return times_sigmoid(v, v);
  return v;
}

// N values with one branch (the same for every thread of the launch).
template <int N>
__device__ __forceinline__ void activate(float (&v)[N], uint32_t act) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate_as<kActRelu>(v[i]);
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate_as<kActGelu>(v[i]);
      break;
    case kActGeluTanh:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate_as<kActGeluTanh>(v[i]);
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate_as<kActSilu>(v[i]);
      break;
    default: break;
  }
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace nvq
