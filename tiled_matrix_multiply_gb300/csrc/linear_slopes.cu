// linear_slopes.cu -- what the gradients of a linear layer y = act(z) + residual start with:
//   dz = dy act'(z),  dbias[n] = sum over the rows of dz[., n].
//
// One pass over dy and z (and one write of dz) is the bound.  A block does a run of rows of 32 lanes'
// vectors of columns, eight warps a row each in turn; a thread's columns are its own, so that the
// sums stay in registers (FP32, of dz before it is rounded) until the eight warps' are added in
// shared memory.  The runs' sums are added by a second launch: no atomics, a fixed order.
#include <algorithm>
#include <cstdint>

#include "activation.cuh"
#include "grouped.h"
#include "row_ops.cuh"
#include "split_bf16.cuh"
#include "tmm_gemm.h"

namespace tmm {
namespace {

constexpr int kWarps = 8;
constexpr int kAhead = 4;        // rows of a warp in flight

struct SlopeParams {
  const void *dy, *pre;
  void *dz;
  float *sums;          // runs x N, or NULL
  int64_t rows, N, lddy, ld_pre, ldz, run;
  int act;
  int planes;           // FP32: dz as its three bf16 parts, planes rows * ldz apart
};

// Lane l has columns first + l W .. + W, 16 bytes' worth, read as vectors (VEC) or one by one; dz's rows
// are vectors in any case, whose last may have values past N that nothing reads (4096 x 4095, bf16, with
// the sums: 34 us where values are read and written one by one with 32 lanes side by side, 26 so).
template <typename T, bool VEC>
__global__ void __launch_bounds__(32 * kWarps)
slopes_kernel(const __grid_constant__ SlopeParams p) {
  constexpr int W = Vec<T>::kCount;
  __shared__ float part[kWarps][32 * W];
  wait_then_start_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t first = int64_t(blockIdx.x) * 32 * W;
  const int64_t r0 = blockIdx.y * p.run, r1 = min(r0 + p.run, p.rows);
  const auto column = [&](int k) { return first + lane * W + k; };
  const auto load = [&](const void *m, int64_t ld, int64_t row, Vec<T> &v) {
    const T *const from = static_cast<const T *>(m) + row * ld;
    if (VEC) {
      if (column(0) < p.N) v.w = *reinterpret_cast<const uint4 *>(from + column(0));
    } else {
#pragma unroll
      for (int k = 0; k < W; ++k)
        if (column(k) < p.N) reinterpret_cast<T *>(&v.w)[k] = from[column(k)];
    }
  };
  uint64_t sum[W / 2] = {};      // pairs of zeros
  for (int64_t r = r0 + warp; r < r1; r += kWarps * kAhead) {
    Vec<T> dy[kAhead], z[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t row = r + u * kWarps;
      dy[u].w = z[u].w = make_uint4(0, 0, 0, 0);
      if (row < r1) {
        load(p.dy, p.lddy, row, dy[u]);
        if (p.pre) load(p.pre, p.ld_pre, row, z[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t row = r + u * kWarps;
      if (row >= r1) break;
      uint64_t d[W / 2];
#pragma unroll
      for (int k = 0; k < W / 2; ++k) d[k] = pair_of(z[u].get(2 * k), z[u].get(2 * k + 1));
      if (p.pre) slope_pairs<sizeof(T) == 2>(p.act, d);
#pragma unroll
      for (int k = 0; k < W / 2; ++k) {
        const uint64_t g = pair_of(dy[u].get(2 * k), dy[u].get(2 * k + 1));
        d[k] = p.pre ? mul2(g, d[k]) : g;
        sum[k] = add2(sum[k], d[k]);
      }
      if (p.dz == nullptr) continue;
      if constexpr (sizeof(T) == 4)
        if (p.planes) {
          uint16_t *const to = static_cast<uint16_t *>(p.dz) + row * p.ldz;
          uint32_t h[W / 2][3];
#pragma unroll
          for (int k = 0; k < W / 2; ++k) split2(of_pair(d[k]).x, of_pair(d[k]).y, h[k]);
#pragma unroll
          for (int pl = 0; pl < 3; ++pl)
            if (column(0) < p.N)
              *reinterpret_cast<uint2 *>(to + pl * p.rows * p.ldz + column(0)) =
                  make_uint2(h[0][pl], h[1][pl]);
          continue;
        }
      Vec<T> out;
#pragma unroll
      for (int k = 0; k < W / 2; ++k) {
        out.set(2 * k, of_pair(d[k]).x);
        out.set(2 * k + 1, of_pair(d[k]).y);
      }
      T *const to = static_cast<T *>(p.dz) + row * p.ldz;
      if (column(0) < p.N) *reinterpret_cast<uint4 *>(to + column(0)) = out.w;
    }
  }
  if (p.sums == nullptr) return;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    const float2 f = of_pair(sum[k >> 1]);
    part[warp][lane * W + k] = k & 1 ? f.y : f.x;
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 32 * W; c += 32 * kWarps) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += part[w][c];
    if (first + c < p.N) p.sums[blockIdx.y * p.N + first + c] = s;
  }
}

// dbias[n] = the runs' sums, 32 columns a block and eight threads a column.
__global__ void __launch_bounds__(256)
runs_kernel(const float *__restrict__ sums, int64_t runs, int64_t N, float *__restrict__ dbias) {
  __shared__ float part[8][32];
  wait_then_start_next();
  const int c = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t n = int64_t(blockIdx.x) * 32 + c;
  float s = 0.0f;
  if (n < N)
    for (int64_t i = w; i < runs; i += 8) s += sums[i * N + n];
  part[w][c] = s;
  __syncthreads();
  if (w == 0 && n < N) {
    for (int i = 1; i < 8; ++i) s += part[i][c];
    dbias[n] = s;
  }
}

// Runs of rows: three blocks an SM, as many as fit at once, of 32 rows at least (4096 x 4096, gelu, bf16,
// sums alone: 21 us, by four blocks 23; reading takes the memory 10 us, the erf bounds the rest).
int64_t runs_of(int64_t rows, int64_t N, int dtype) {
  const int64_t strip = dtype == TMM_F32 ? 128 : 256, strips = (N + strip - 1) / strip;
  const int64_t want = std::max<int64_t>(1, 3 * 152 / strips);
  return std::max<int64_t>(1, std::min(want, (rows + 31) / 32));
}

bool aligned(const void *p, int64_t ld, int64_t size) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * size % 16 == 0;
}

template <typename T>
cudaError_t launch_as(const LinearGradProblem &g, void *dz, int64_t ldz, bool planes,
                      float *partial, cudaStream_t stream) {
  const int64_t size = sizeof(T), runs = runs_of(g.rows, g.N, g.dtype);
  SlopeParams p = {};
  p.dy = g.dy.data;
  p.lddy = g.dy.ld;
  p.pre = g.act == TMM_ACT_NONE ? nullptr : g.pre;
  p.ld_pre = g.ld_pre;
  p.dz = dz;
  p.ldz = ldz;
  p.planes = planes;
  p.rows = g.rows;
  p.N = g.N;
  p.act = g.act;
  p.run = (g.rows + runs - 1) / runs;
  p.sums = g.dbias == nullptr ? nullptr : runs > 1 ? partial : g.dbias;
  const bool vec = g.N * size % 16 == 0 && aligned(p.dy, p.lddy, size) &&
                   (p.pre == nullptr || aligned(p.pre, p.ld_pre, size));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  const int64_t strip = 32 * Vec<T>::kCount;
  cfg.gridDim = dim3(unsigned((g.N + strip - 1) / strip), unsigned(runs), 1);
  cfg.blockDim = dim3(32 * kWarps, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e =
      cudaLaunchKernelEx(&cfg, vec ? slopes_kernel<T, true> : slopes_kernel<T, false>, p);
  if (e != cudaSuccess || g.dbias == nullptr || runs == 1) return e;
  cfg.gridDim = dim3(unsigned((g.N + 31) / 32), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  return cudaLaunchKernelEx(&cfg, runs_kernel, static_cast<const float *>(partial), runs, g.N,
                            g.dbias);
}

}  // namespace

size_t linear_bias_bytes(int64_t rows, int64_t N, int dtype) {
  const int64_t runs = runs_of(rows, N, dtype);
  return runs > 1 ? size_t(runs) * size_t(N) * sizeof(float) : 0;
}

cudaError_t launch_linear_slopes(const LinearGradProblem &p, void *dz, int64_t ldz, bool planes,
                                 float *partial, const DeviceInfo &, cudaStream_t stream) {
  if (p.dtype == TMM_BF16) return launch_as<__nv_bfloat16>(p, dz, ldz, planes, partial, stream);
  if (p.dtype == TMM_F16) return launch_as<__half>(p, dz, ldz, planes, partial, stream);
  return launch_as<float>(p, dz, ldz, planes, partial, stream);
}

}  // namespace tmm
