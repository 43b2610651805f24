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

// Two FP32 numbers in one 64-bit register, and operations on both.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// v Phi(v) = max(v, 0) - |v| Phi(-|v|), which keeps the digits of the negative tail that
// v (1 + erf) / 2 loses in FP32 (5 % at v = -5, all from -5.5 on).  Phi(-s) = exp(-s^2 / 2) R(s),
// R(s) = u (c0 + c1 u + .. + c7 u^7), u = 1 / (1 + 0.305 s): the form of Hastings'
// approximations, its coefficients fitted here to half the scaled complementary error
// function of s / sqrt 2 over s = 0 .. 13.5, to 9.4e-8 relative.  The whole is good to
// (v^2 + 1) 2^-23 + 2^-20 relative: the exponent's rounding, and all else.  A positive
// infinity has no tail (16 gives 2^-184); -inf and NaN give NaN, as the formula does.
__device__ __forceinline__ float2 gelu(float2 v) {
  const float2 s = make_float2(v.x < 0.f ? -v.x : fminf(v.x, 16.f), v.y < 0.f ? -v.y : fminf(v.y, 16.f));
  auto both = [](float c) { return pair(c, c); };
  const uint64_t ss = pair(s.x, s.y), vv = pair(v.x, v.y);
  float2 u = unpair(fma2(ss, both(0.305f), both(1.0f)));
  float2 e = unpair(mul2(mul2(vv, vv), both(0.5f * kNegLog2E)));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(u.x));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(u.y));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
  const uint64_t uu = pair(u.x, u.y);
  uint64_t q = fma2(uu, both(0.0366991609f), both(-0.152988181f));
  q = fma2(uu, q, both(0.185716659f));
  q = fma2(uu, q, both(-0.0379766114f));
  q = fma2(uu, q, both(0.121021569f));
  q = fma2(uu, q, both(0.103420898f));
  q = fma2(uu, q, both(0.122466817f));
  q = fma2(uu, q, both(0.121639736f));
  const float2 tail = unpair(mul2(mul2(ss, uu), mul2(pair(e.x, e.y), q)));
  return make_float2((v.x < 0.f ? 0.f : v.x) - tail.x, (v.y < 0.f ? 0.f : v.y) - tail.y);
}

// The same out of line, for kernels whose epilogue is copied many times over: code that long
// shows in their every activation.  8192 x 4096 x 4096 (the persistent W4A4 kernel, 64 values
// a thread) without an activation and with gelu: 93.6 and 108.1 us called, 96.5 and 105.9
// inlined; by erfcf, inlined, gelu takes 148.  W4A16, 31 x 24576 x 4096, residual and gelu: 27.0 and 27.7
// called, 27.3 and 27.8 inlined.  Inlined for few values a thread: W4A16, 1 x 4096 x 4096,
// gelu: 5.7 us (5.9 called); W4A4, 777 x 5128 x 1088: 14.1 (15.8).
__device__ __noinline__ float2 gelu_called(float2 v) { return gelu(v); }

template <uint32_t ACT>
__device__ __forceinline__ float activate_as(float v) {
  if constexpr (ACT == kActRelu) return v < 0.f ? 0.f : v;                        // NaN stays NaN
  // 0.5 (1 + tanh(z)) = sigmoid(2 z), z = sqrt(2 / pi) (v + 0.044715 v^3)
  if constexpr (ACT == kActGeluTanh) {
    constexpr float a = kNegLog2E * 1.5957691216057308f, b = a * 0.044715f;
    return over_one_plus_exp2(v, v * __fmaf_rn(b, v * v, a));
  }
  if constexpr (ACT == kActSilu) return times_sigmoid(v, v);
  return v;
}

// N values with one branch (the same for every thread of the launch).
template <bool CALL, int N>
__device__ __forceinline__ void activate(float (&v)[N], uint32_t act) {
  static_assert(N % 2 == 0, "gelu takes two");
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate_as<kActRelu>(v[i]);
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float2 z = make_float2(v[i], v[i + 1]), r = CALL ? gelu_called(z) : gelu(z);
        v[i] = r.x;
        v[i + 1] = r.y;
      }
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
