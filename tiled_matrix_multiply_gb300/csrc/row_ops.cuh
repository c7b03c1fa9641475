// row_ops.cuh -- what the kernels over rows of scores (routing, log probabilities) and the products'
// epilogues share: element types, wide loads and stores, and the order of launches.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace tmm {

template <typename T>
__device__ __forceinline__ float as_float(T v) {
  return float(v);
}
template <typename T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half rounded<__half>(float v) {
  return __float2half_rn(v);
}

// 16 bytes of values.
template <typename T>
struct Vec {
  static constexpr int kCount = 16 / int(sizeof(T));
  uint4 w;
  __device__ __forceinline__ float get(int i) const {
    return float(reinterpret_cast<const T *>(&w)[i]);
  }
  __device__ __forceinline__ void set(int i, float v) {
    reinterpret_cast<T *>(&w)[i] = rounded<T>(v);
  }
};
template <>
__device__ __forceinline__ float Vec<__nv_bfloat16>::get(int i) const {
  const uint32_t two = reinterpret_cast<const uint32_t *>(&w)[i >> 1];
  return __uint_as_float(i & 1 ? two & 0xFFFF0000u : two << 16);
}

// Programmatic dependent launch: the launches before are complete and visible after it, and the
// next one may start as soon as there is room (it waits in turn).  What the launches before wrote is no
// constant of the kernel, which runs already while they do: its inputs are read by plain loads, not
// by __ldg or through pointers to const that are __restrict__, which may take the read-only path.
__device__ __forceinline__ void wait_then_start_next() {
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}

// 2^x, relative error below 2^-22; 0 below 2^-126.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

}  // namespace tmm
