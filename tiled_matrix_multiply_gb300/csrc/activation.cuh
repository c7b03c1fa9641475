// activation.cuh -- the activations of a linear layer's epilogue and their derivatives.
//
//   relu       max(z, 0)                        (derivative at 0: 0)
//   silu       z s(z),                          s(z) = 1 / (1 + e^-z)
//   gelu       z Phi(z) = z/2 erfc(-z / sqrt 2)
//   gelu_tanh  z/2 (1 + tanh u) = z s(2 u),     u = sqrt(2/pi) (z + 0.044715 z^3)
// FAST, for results of 16 bits: the exponential and the quotient are the hardware's approximations
// (relative errors of a few 2^-22, far below 2^-12), and e^-z may overflow, which gives s = 0.
#pragma once

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

template <bool FAST>
__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case TMM_ACT_RELU: return z < 0.0f ? 0.0f : z;
    case TMM_ACT_SILU: return z * logistic<FAST>(z);
    case TMM_ACT_GELU: return 0.5f * z * erfcf(-0.70710678118654752f * z);
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
      const float e = FAST ? __expf(-0.5f * z * z) : expf(-0.5f * z * z);
      return fmaf(0.5f, erfcf(-0.70710678118654752f * z), 0.39894228040143268f * z * e);
    }
    case TMM_ACT_GELU_TANH: {
      z = z > 1e4f ? 1e4f : z < -1e4f ? -1e4f : z;      // constant beyond, and z^3 finite
      const float v = tanh_argument(z), s = logistic<FAST>(v), r = logistic<FAST>(-v);
      return s * fmaf(z * r, 1.5957691216057308f * fmaf(0.134145f * z, z, 1.0f), 1.0f);
    }
    default: return 1.0f;
  }
}

// N values, with one switch for all.
template <int N>
__device__ __forceinline__ void activate_all(int act, float (&z)[N]) {
  switch (act) {
#define TMM_EACH(code)                                              \
  case code:                                                        \
    _Pragma("unroll") for (int k = 0; k < N; ++k) z[k] = activate<true>(code, z[k]); \
    break;
    TMM_EACH(TMM_ACT_RELU)
    TMM_EACH(TMM_ACT_SILU)
    TMM_EACH(TMM_ACT_GELU)
    TMM_EACH(TMM_ACT_GELU_TANH)
#undef TMM_EACH
    default: break;
  }
}

}  // namespace tmm
