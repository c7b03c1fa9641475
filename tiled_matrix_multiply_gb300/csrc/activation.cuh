// activation.cuh -- the activations of a linear layer's epilogue and their derivatives.
//
//   relu       max(z, 0)                        (derivative at 0: 0)
//   silu       z s(z),                          s(z) = 1 / (1 + e^-z)
//   gelu       z Phi(z) = z/2 erfc(-z / sqrt 2)
//   gelu_tanh  z/2 (1 + tanh u) = z s(2 u),     u = sqrt(2/pi) (z + 0.044715 z^3)
// FAST, for results of 16 bits: the exponential and the quotient are the hardware's approximations
// (relative errors of a few 2^-22, far below 2^-12), and e^-z may overflow, which gives s = 0.
// There erfc(x) = e^(-x^2) t q(t), t = 1 / (1 + 0.45 x), x >= 0: x e^(x^2) erfc(x) tends to a constant,
// so that t q(t) stands for e^(x^2) erfc(x) with a relative error below 2^-21 everywhere.  q is the
// polynomial of degree 7 whose largest relative error on [0, 10] is the smallest (a linear program
// over 4001 points).  CUDA's erfcf, right to a few 2^-24 and three times as many instructions, held
// the result warps up beyond the products: 8192 x 4096 x 4096 in bf16 190 us, without activation 154.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "tmm_gemm.h"

namespace tmm {

template <bool FAST>
__device__ __forceinline__ float logistic(float z) {
  if (FAST) return __fdividef(1.0f, 1.0f + __expf(-z));
  return 1.0f / (1.0f + expf(-z));
}
__device__ __forceinline__ float tanh_argument(float z) {      // 2 u
  return 1.5957691216057308f * z * fmaf(0.044715f * z, z, 1.0f);
}

// Phi(-|z|), and e^(-z^2 / 2).
__device__ __forceinline__ float normal_tail(float z, float &e) {
  const float t = __fdividef(1.0f, fmaf(0.31819805f, fabsf(z), 1.0f));
  float q = 0.0668829f;
  q = fmaf(q, t, -0.24035851f);
  q = fmaf(q, t, 0.2090319f);
  q = fmaf(q, t, 0.04007119f);
  q = fmaf(q, t, 0.18879604f);
  q = fmaf(q, t, 0.22802131f);
  q = fmaf(q, t, 0.25364735f);
  q = fmaf(q, t, 0.25390811f);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-0.72134752f * z * z));
  return 0.5f * t * q * e;
}

template <bool FAST>
__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case TMM_ACT_RELU: return z < 0.0f ? 0.0f : z;
    case TMM_ACT_SILU: return z * logistic<FAST>(z);
    case TMM_ACT_GELU: {
      if (!FAST) return 0.5f * z * erfcf(-0.70710678118654752f * z);
      // z Phi(-|z|), less z where z > 0; (a tail of 0 times an infinity is 0).
      float e;
      const float r = copysignf(fminf(fabsf(z), 64.0f), z) * normal_tail(z, e);
      return z > 0.0f ? z - r : r;
    }
    case TMM_ACT_GELU_TANH: return z * logistic<FAST>(tanh_argument(z));
    default: return z;
  }
}

// The derivative at z.
template <bool FAST>
__device__ __forceinline__ float activation_slope(int act, float z) {
  switch (act) {
    case TMM_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case TMM_ACT_SILU: {
      const float s = logistic<FAST>(z), r = logistic<FAST>(-z);
      return s * fmaf(z, r, 1.0f);
    }
    case TMM_ACT_GELU: {
      if (!FAST)
        return fmaf(0.5f, erfcf(-0.70710678118654752f * z),
                    0.39894228040143268f * z * expf(-0.5f * z * z));
      float e;
      const float tail = normal_tail(z, e);
      return fmaf(0.39894228040143268f * z, e, z > 0.0f ? 1.0f - tail : tail);
    }
    case TMM_ACT_GELU_TANH: {
      z = z > 1e4f ? 1e4f : z < -1e4f ? -1e4f : z;      // constant beyond, and z^3 finite
      const float v = tanh_argument(z), s = logistic<FAST>(v), r = logistic<FAST>(-v);
      return s * fmaf(z * r, 1.5957691216057308f * fmaf(0.134145f * z, z, 1.0f), 1.0f);
    }
    default: return 1.0f;
  }
}

// ---- pairs, for results of 16 bits ---------------------------------------------------------

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
__device__ __forceinline__ uint64_t exp2_pair(uint64_t v) {
  float2 f = of_pair(v);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(f.x));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(f.y));
  return pair_of(f.x, f.y);
}
__device__ __forceinline__ float positive_part(float z) {      // (NaN stays)
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(z));
  return y;
}
// z / (1 + 2^u)
__device__ __forceinline__ uint64_t times_logistic2(uint64_t z, uint64_t u) {
  return mul2(z, reciprocal2(add2(exp2_pair(u), both(1.0f))));
}

// Two values at once, half the instructions; the same formulas as `activate`.
__device__ __forceinline__ uint64_t activate2(int act, uint64_t z) {
  const float2 f = of_pair(z);
  switch (act) {
    case TMM_ACT_RELU: return pair_of(positive_part(f.x), positive_part(f.y));
    case TMM_ACT_SILU: return times_logistic2(z, mul2(z, both(-1.44269504f)));
    case TMM_ACT_GELU: {
      // max(z, 0) - a Phi(-a), a = |z| (no more than 64, whose tail is 0).
      const uint64_t a = pair_of(fminf(fabsf(f.x), 64.0f), fminf(fabsf(f.y), 64.0f));
      const uint64_t t = reciprocal2(fma2(a, both(0.31819805f), both(1.0f)));
      uint64_t q = both(0.5f * 0.0668829f);
      q = fma2(q, t, both(0.5f * -0.24035851f));
      q = fma2(q, t, both(0.5f * 0.2090319f));
      q = fma2(q, t, both(0.5f * 0.04007119f));
      q = fma2(q, t, both(0.5f * 0.18879604f));
      q = fma2(q, t, both(0.5f * 0.22802131f));
      q = fma2(q, t, both(0.5f * 0.25364735f));
      q = fma2(q, t, both(0.5f * 0.25390811f));
      const uint64_t e = exp2_pair(mul2(mul2(a, both(-0.72134752f)), a));
      const uint64_t tail = mul2(mul2(t, q), mul2(e, both(-1.0f)));
      return fma2(a, tail, pair_of(positive_part(f.x), positive_part(f.y)));
    }
    case TMM_ACT_GELU_TANH: {
      // z s(2 u): the exponent -2 u log2(e) = z (c0 + c1 z^2).
      const uint64_t square = mul2(z, z);
      return times_logistic2(
          z, mul2(z, fma2(square, both(-2.3022082f * 0.044715f), both(-2.3022082f))));
    }
    default: return z;
  }
}
template <int N>
__device__ __forceinline__ void activate_pairs(int act, uint64_t (&z)[N]) {
  if (act == TMM_ACT_NONE) return;
#pragma unroll
  for (int code = TMM_ACT_RELU; code <= TMM_ACT_GELU_TANH; ++code)
    if (act == code) {
#pragma unroll
      for (int k = 0; k < N; ++k) z[k] = activate2(code, z[k]);
      return;
    }
}
// N values, with one choice for all.
template <int N>
__device__ __forceinline__ void activate_all(int act, float (&z)[N]) {
  if (act == TMM_ACT_NONE) return;
  uint64_t v[N / 2];
#pragma unroll
  for (int k = 0; k < N / 2; ++k) v[k] = pair_of(z[2 * k], z[2 * k + 1]);
  activate_pairs(act, v);
#pragma unroll
  for (int k = 0; k < N / 2; ++k) {
    const float2 f = of_pair(v[k]);
    z[2 * k] = f.x;
    z[2 * k + 1] = f.y;
  }
}

}  // namespace tmm
