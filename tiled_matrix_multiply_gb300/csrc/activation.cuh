// activation.cuh -- the activations of a linear layer's epilogue and their derivatives, on pairs of FP32
// values (fma.rn.f32x2 and the like: two results an instruction).
//
//   relu       max(z, 0)                        (derivative at 0: 0)
//   silu       z s(z),                          s(z) = 1 / (1 + e^-z)
//   gelu       z Phi(z) = max(z, 0) - |z| Phi(-|z|)
//   gelu_tanh  z/2 (1 + tanh u) = z s(2 u),     u = sqrt(2/pi) (z + 0.044715 z^3)
//   Phi(-a) = erfc(a / sqrt 2) / 2,  erfc(x) = e^(-x^2) t q(t),  t = 1 / (1 + c x):  x e^(x^2) erfc(x) tends
//   to a constant, so that t q(t) stands for e^(x^2) erfc(x) with a bounded relative error everywhere.
//   q is a polynomial whose largest relative error on [0, 10] is as small as FP32 coefficients let it be (a
//   linear program over 4001 points; its coefficients rounded one after another, the rest fitted again
//   each time; c the best of a few): of degree 7 and c = 0.432, 2^-23.2; of degree 8 and c = 0.4875,
//   2^-25.4.  CUDA's erfcf has three times as many instructions and held the result warps up beyond the
//   products: 8192 x 4096 x 4096 in bf16 190 us, without activation 154.
// FAST, for results of 16 bits: exponentials by the hardware's power of two with a rounded argument
// (relative error 2^-22 and |z| 2^-24, far below 2^-12).  Else the argument's rounding is made up for.
// Infinities and NaN are the formulas', those of the derivatives at infinities their limits.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "tmm_gemm.h"

namespace tmm {

__device__ __forceinline__ uint64_t pair_of(float x, float y) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  return v;
}
__device__ __forceinline__ float2 of_pair(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t both(float x) { return pair_of(x, x); }
__device__ __forceinline__ uint64_t reciprocal2(uint64_t v) {
  float2 f = of_pair(v);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(f.x));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(f.y));
  return pair_of(f.x, f.y);
}
__device__ __forceinline__ uint64_t power2(uint64_t v) {
  float2 f = of_pair(v);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(f.x));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(f.y));
  return pair_of(f.x, f.y);
}
// Between lo and hi; NaN stays.
__device__ __forceinline__ float within(float v, float lo, float hi) {
  float y;
  asm("{\n .reg .f32 t;\n max.NaN.f32 t, %1, %2;\n min.NaN.f32 %0, t, %3;\n}\n"
      : "=f"(y)
      : "f"(v), "f"(lo), "f"(hi));
  return y;
}
__device__ __forceinline__ float positive_part(float z) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(z));
  return y;
}

// e^v
template <bool FAST>
__device__ __forceinline__ uint64_t exp_pair(uint64_t v) {
  if (FAST) return power2(mul2(v, both(1.44269504f)));
  const float2 f = of_pair(v);
  v = pair_of(within(f.x, -88.0f, 88.0f), within(f.y, -88.0f, 88.0f));      // (finite, 0 in 1 / e)
  // v log2(e) = h + l, and e^v = 2^h (1 + l ln 2).
  const uint64_t h = mul2(v, both(1.44269504f));
  const uint64_t l = fma2(v, both(1.9259630e-8f), fma2(v, both(1.44269504f), mul2(h, both(-1.0f))));
  const uint64_t e = power2(h);
  return fma2(mul2(e, l), both(0.69314718f), e);
}
// 1 / (1 + e^v)
template <bool FAST>
__device__ __forceinline__ uint64_t logistic(uint64_t v) {
  return reciprocal2(add2(exp_pair<FAST>(v), both(1.0f)));
}
// Phi(-a), and e = e^(-a^2 / 2); a >= 0.
template <bool FAST>
__device__ __forceinline__ uint64_t normal_tail(uint64_t a, uint64_t &e) {
  // The coefficients of q / 2, the highest first.
  constexpr float few[8] = {0.0366231166f, -0.151907831f, 0.182719693f, -0.0356251895f,
                            0.119878531f, 0.103872582f,  0.12260922f,  0.121829927f};
  constexpr float more[9] = {-0.028188616f, 0.144669294f, -0.270742476f, 0.187449187f, -0.0376035161f,
                             0.111842997f, 0.117160685f, 0.137906998f,  0.137505442f};
  // (c / sqrt 2)
  const uint64_t t = reciprocal2(fma2(a, both(FAST ? 0.305470139f : 0.34471455f), both(1.0f)));
  uint64_t q = both(FAST ? few[0] : more[0]);
#pragma unroll
  for (int i = 1; i < (FAST ? 8 : 9); ++i) q = fma2(q, t, both(FAST ? few[i] : more[i]));
  e = FAST ? power2(mul2(mul2(a, both(-0.72134752f)), a))
           : exp_pair<false>(mul2(mul2(a, both(-0.5f)), a));
  return mul2(mul2(t, q), e);
}
constexpr float kTanhSlope = 1.5957691216057308f, kTanhCube = 0.044715f;      // 2 sqrt(2/pi)

template <bool FAST>
__device__ __forceinline__ uint64_t activate2(int act, uint64_t z) {
  const float2 f = of_pair(z);
  switch (act) {
    case TMM_ACT_RELU: return pair_of(positive_part(f.x), positive_part(f.y));
    case TMM_ACT_SILU: return mul2(z, logistic<FAST>(mul2(z, both(-1.0f))));
    case TMM_ACT_GELU: {
      // (|z| no more than 64, whose tail is 0.)
      const uint64_t a = pair_of(fminf(fabsf(f.x), 64.0f), fminf(fabsf(f.y), 64.0f));
      uint64_t e;
      return fma2(mul2(a, both(-1.0f)), normal_tail<FAST>(a, e),
                  pair_of(positive_part(f.x), positive_part(f.y)));
    }
    case TMM_ACT_GELU_TANH: {
      const uint64_t w = fma2(mul2(z, z), both(-kTanhSlope * kTanhCube), both(-kTanhSlope));
      return mul2(z, logistic<FAST>(mul2(z, w)));
    }
    default: return z;
  }
}
// The derivatives at z.  They are 0 and 1 but for less than any FP32 value beyond 200 (gelu 64), and so at
// infinities, which a kept z of FP16 is from 65520 on.
template <bool FAST>
__device__ __forceinline__ uint64_t slope2(int act, uint64_t z) {
  float2 f = of_pair(z);
  const uint64_t one = both(1.0f), minus = both(-1.0f);
  switch (act) {
    case TMM_ACT_RELU:      // (of NaN NaN)
      return pair_of(f.x > 0.0f ? 1.0f : positive_part(f.x),
                     f.y > 0.0f ? 1.0f : positive_part(f.y));
    case TMM_ACT_SILU: {
      z = pair_of(within(f.x, -200.0f, 200.0f), within(f.y, -200.0f, 200.0f));
      const uint64_t s = logistic<FAST>(mul2(z, minus));
      return mul2(s, fma2(z, fma2(s, minus, one), one));
    }
    case TMM_ACT_GELU: {
      f = make_float2(within(f.x, -64.0f, 64.0f), within(f.y, -64.0f, 64.0f));
      z = pair_of(f.x, f.y);
      uint64_t e;
      const float2 tail = of_pair(normal_tail<FAST>(pair_of(fabsf(f.x), fabsf(f.y)), e));
      return fma2(mul2(z, both(0.39894228f)), e,
                  pair_of(f.x > 0.0f ? 1.0f - tail.x : tail.x,
                          f.y > 0.0f ? 1.0f - tail.y : tail.y));
    }
    case TMM_ACT_GELU_TANH: {
      // (Constant beyond 10^4, and z^3 finite.)
      z = pair_of(within(f.x, -1e4f, 1e4f), within(f.y, -1e4f, 1e4f));
      const uint64_t square = mul2(z, z);
      const uint64_t w = fma2(square, both(-kTanhSlope * kTanhCube), both(-kTanhSlope));
      const uint64_t s = logistic<FAST>(mul2(z, w));
      const uint64_t d = fma2(square, both(3.0f * kTanhSlope * kTanhCube), both(kTanhSlope));
      return mul2(s, fma2(mul2(z, fma2(s, minus, one)), d, one));
    }
    default: return one;
  }
}

// f of every pair, with one choice for all.  (A chain of comparisons: a jump table's first use in a block
// costs more than a thousand cycles.)
template <int N, typename F>
__device__ __forceinline__ void for_activation(int act, uint64_t (&z)[N], F f) {
#pragma unroll
  for (int code = TMM_ACT_RELU; code <= TMM_ACT_GELU_TANH; ++code)
    if (act == code) {
#pragma unroll
      for (int k = 0; k < N; ++k) z[k] = f(code, z[k]);
      return;
    }
}
template <bool FAST, int N>
__device__ __forceinline__ void activate_pairs(int act, uint64_t (&z)[N]) {
  if (act == TMM_ACT_NONE) return;
  for_activation(act, z, [](int code, uint64_t v) { return activate2<FAST>(code, v); });
}
template <bool FAST, int N>
__device__ __forceinline__ void slope_pairs(int act, uint64_t (&z)[N]) {
  for_activation(act, z, [](int code, uint64_t v) { return slope2<FAST>(code, v); });
}

}  // namespace tmm
