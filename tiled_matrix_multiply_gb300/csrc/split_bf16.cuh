// split_bf16.cuh -- FP32 values as three bf16 parts, x = x0 + x1 + x2 exactly (from 2^-102 up).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace tmm {

// The bf16 nearest an FP32 value (ties away from zero), as its bits; in the top binade, where
// rounding could reach infinity, the value truncated.
__device__ __forceinline__ uint32_t nearest_bf16(uint32_t b) {
  return (b & 0x7F800000u) == 0x7F000000u ? b & 0xFFFF0000u : (b + 0x8000u) & 0xFFFF0000u;
}
// The three bf16 parts of an FP32 value: each the nearest to what the ones before leave, so
// |x1| <= 2^-8 |x| and |x2| <= 2^-16 |x|, and x = x0 + x1 + x2 exactly (for |x| >= 2^-102;
// below, what falls under the smallest subnormal is dropped).  An infinity or a NaN is its own
// first part.
__device__ __forceinline__ void split3(float x, uint16_t (&h)[3]) {
  const uint32_t b = __float_as_uint(x);
  if ((b & 0x7F800000u) == 0x7F800000u) {
    h[0] = uint16_t((b >> 16) | ((b & 0x007FFFFFu) ? 0x0040u : 0u));
    h[1] = h[2] = 0;
    return;
  }
  const uint32_t b0 = nearest_bf16(b);
  const float r = x - __uint_as_float(b0);
  const uint32_t b1 = nearest_bf16(__float_as_uint(r));
  const float s = r - __uint_as_float(b1);
  h[0] = uint16_t(b0 >> 16);
  h[1] = uint16_t(b1 >> 16);
  h[2] = uint16_t(nearest_bf16(__float_as_uint(s)) >> 16);
}

// split3 of eight values: the parts of value i in 16 bits of h[part], as they are stored.  Values
// below 2^127 take the conversion instruction, two at a time (5.5 instructions a value against
// split3's 20).
__device__ __forceinline__ uint32_t pair_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void split8(const float (&x)[8], uint32_t (&h)[3][4]) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));      // (a NaN is not seen)
  const float sum = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
  if (top < 0x1p127f && sum == sum) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = x[2 * i], b = x[2 * i + 1];
#pragma unroll
      for (int pl = 0; pl < 3; ++pl) {
        h[pl][i] = pair_bf16(a, b);
        a -= __uint_as_float(h[pl][i] << 16);
        b -= __uint_as_float(h[pl][i] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint16_t a[3], b[3];
      split3(x[2 * i], a);
      split3(x[2 * i + 1], b);
#pragma unroll
      for (int pl = 0; pl < 3; ++pl) h[pl][i] = a[pl] | (uint32_t(b[pl]) << 16);
    }
  }
}

// The same of two values.
__device__ __forceinline__ void split2(float a, float b, uint32_t (&h)[3]) {
  if (fmaxf(fabsf(a), fabsf(b)) < 0x1p127f && a == a && b == b) {
#pragma unroll
    for (int pl = 0; pl < 3; ++pl) {
      h[pl] = pair_bf16(a, b);
      a -= __uint_as_float(h[pl] << 16);
      b -= __uint_as_float(h[pl] & 0xFFFF0000u);
    }
  } else {
    uint16_t x[3], y[3];
    split3(a, x);
    split3(b, y);
#pragma unroll
    for (int pl = 0; pl < 3; ++pl) h[pl] = x[pl] | (uint32_t(y[pl]) << 16);
  }
}

}  // namespace tmm
