// linear_epilogue.cuh -- what becomes of a product's sums in a linear layer:
//   z = sum + bias (kept as it is rounded, where asked for),  y = act(z) + residual.
// Results are D[n, q], n on the lanes of tensor memory; `Params` are those of either product kernel, by
// their fields: out, ld_out, out_type, vec_out, N, bias, bias_f32, act, residual, ld_residual, pre,
// ld_pre.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "activation.cuh"

namespace tmm {

constexpr int kOutF32 = 0, kOutBF16 = 1, kOutF16 = 2;      // types of results

// Element `at` of a matrix of the operands' type, in FP32.
template <int PLANES, typename Params>
__device__ __forceinline__ float linear_value(const Params &p, const void *m, int64_t at) {
  if constexpr (PLANES == 3) return static_cast<const float *>(m)[at];
  if (p.out_type == kOutBF16) return float(static_cast<const __nv_bfloat16 *>(m)[at]);
  return float(static_cast<const __half *>(m)[at]);
}
template <int PLANES, typename Params>
__device__ __forceinline__ float linear_bias(const Params &p, int n) {
  if (p.bias == nullptr || n >= p.N) return 0.0f;
  if (p.bias_f32) return static_cast<const float *>(p.bias)[n];
  return linear_value<PLANES>(p, p.bias, n);
}
template <int PLANES, typename Params>
__device__ __forceinline__ void linear_store(const Params &p, void *m, int64_t at, float v) {
  if constexpr (PLANES == 3)
    static_cast<float *>(m)[at] = v;
  else if (p.out_type == kOutBF16)
    static_cast<__nv_bfloat16 *>(m)[at] = __float2bfloat16_rn(v);
  else
    static_cast<__half *>(m)[at] = __float2half_rn(v);
}
// One result: z = the sum and the bias.
template <int PLANES, typename Params>
__device__ __forceinline__ void linear_one(const Params &p, int64_t row, int n, float z) {
  if (p.pre) linear_store<PLANES>(p, p.pre, row * p.ld_pre + n, z);
  float y = activate<PLANES == 1>(p.act, z);
  if (p.residual) y += linear_value<PLANES>(p, p.residual, row * p.ld_residual + n);
  linear_store<PLANES>(p, p.out, row * p.ld_out + n, y);
}
template <typename Params>
__device__ __forceinline__ uint32_t pack_results(const Params &p, float lo, float hi) {
  uint32_t w;
  if (p.out_type == kOutBF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
template <typename Params>
__device__ __forceinline__ float2 unpack_values(const Params &p, uint32_t w) {
  if (p.out_type == kOutBF16)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// 16 columns of the tile, the rows of the result from `first` on, `left` of them at most, for the
// warp's 32 n from nw on.  In FP32 a lane has its n in all of
// them, 128 bytes of a row a warp.  16-bit results go through 2 KiB of shared memory a warp as FP32,
// 16 rows of 32 n, of which a lane then has two pieces of 8 n: everything read and written is 16
// bytes a lane.  The bias of those 8 n (or of the lane's one) is in `bias`.
template <int PLANES, typename Params>
__device__ __forceinline__ void linear_columns(const Params &p, int64_t first, int left, int nw,
                                               const float (&v)[16], const float (&bias)[8],
                                               uint32_t stage) {
  const int lane = threadIdx.x & 31;
  const int count = min(16, left);
  if (PLANES == 3 || !p.vec_out) {
    const int n = nw + lane;
    if (n < p.N)
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (j < count) linear_one<PLANES>(p, first + j, n, v[j] + bias[0]);
    return;
  }
  // Chunk c of four n of row r is at r * 128 + 16 (c ^ r % 8): free of bank conflicts both ways.
  __syncwarp();      // the reads of the block before are done
#pragma unroll
  for (int j = 0; j < 16; ++j)
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(stage + j * 128 + (((lane >> 2) ^ (j & 7)) << 4) +
                                                 (lane & 3) * 4),
                 "f"(v[j])
                 : "memory");
  __syncwarp();
  const int piece = lane & 3, n8 = nw + piece * 8;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = (lane >> 2) + 8 * i;
    float z[8];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(z[4 * h]), "=f"(z[4 * h + 1]), "=f"(z[4 * h + 2]), "=f"(z[4 * h + 3])
                   : "r"(stage + row * 128 + (((2 * piece + h) ^ (row & 7)) << 4))
                   : "memory");
    if (row >= count || n8 >= p.N) continue;
    const int64_t r = first + row;
#pragma unroll
    for (int k = 0; k < 8; ++k) z[k] += bias[k];
    if (n8 + 8 > p.N) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (n8 + k < p.N) linear_one<PLANES>(p, r, n8 + k, z[k]);
      continue;
    }
    uint4 res = make_uint4(0, 0, 0, 0);
    if (p.residual)
      res = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.residual) +
                                             r * p.ld_residual + n8);
    if (p.pre)
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.pre) + r * p.ld_pre + n8) =
          make_uint4(pack_results(p, z[0], z[1]), pack_results(p, z[2], z[3]),
                     pack_results(p, z[4], z[5]), pack_results(p, z[6], z[7]));
    activate_all<8>(p.act, z);
    if (p.residual) {
      const uint32_t w[4] = {res.x, res.y, res.z, res.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 a = unpack_values(p, w[k]);
        z[2 * k] += a.x;
        z[2 * k + 1] += a.y;
      }
    }
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + r * p.ld_out + n8) =
        make_uint4(pack_results(p, z[0], z[1]), pack_results(p, z[2], z[3]),
                   pack_results(p, z[4], z[5]), pack_results(p, z[6], z[7]));
  }
}

}  // namespace tmm
