// linear_slopes.cu -- what the gradients of a linear layer y = act(z) + residual start with:
//   dz = dy act'(z),  dbias[n] = sum over the rows of dz[., n].
//
// One pass over dy and z (and one write of dz) is the bound.  A block does a run of rows of 32 lanes'
// vectors of columns, eight warps a row each in turn; a thread's columns are its own, so that the
// sums stay in registers (FP32, of dz before it is rounded) until the eight warps' are added in
// shared memory.  The runs' sums are added by a second launch: no atomics, a fixed order.
//
// dz goes to the products in the operands' type, as the tensor cores take two operands of one type, and a
// second part for the rest of its bits would double the products' time.  That rounding adds to a result's
// error about as much as the result's own does (bf16, of the norm: 2.3e-3 in all, 1.7e-3 without).
// In FP16 slopes of up to 1.13 take dy past 65504, and small dy past 2^-14 downwards, where dx and dw may
// be neither.  So dz is kept times a power of two that brings the largest finite |dy| to between 2^14
// and 2^15, found by a pass over dy before (peaks_kernel), and the products take it out again: dz is
// rounded to eleven bits, and to 2^-39 of the largest |dy|.  (relu's dz is dy or 0.)
#include <algorithm>
#include <cstdint>
#include <type_traits>

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
  const uint32_t *peaks;      // SCALED: the blocks' largest |dy|, as bits
  int peak_count;
  float *unscale;             // and what dz is to be multiplied by, written here
};

// Blocks of the pass over dy at most: two an SM, and no more than a block of slopes_kernel can read soon.
constexpr int kMaxPeaks = 304;
constexpr int kPeakStrip = 256;        // columns of a warp's load
constexpr int kPeakAhead = 8;          // loads of a warp in flight

// The largest finite |dy| of a block's strips of rows, by turns a warp each: a pass that memory bounds
// (4096 x 4096 8 us; with loads of four rows of one strip in flight, of which there are only two, 40).  VEC:
// rows start on 16-byte boundaries (a matrix without gaps is one row).
template <bool VEC>
__global__ void __launch_bounds__(32 * kWarps)
peaks_kernel(const uint16_t *dy, int64_t rows, int64_t N, int64_t ld, int64_t strips,
             int64_t down, int64_t across, uint32_t *peaks) {
  constexpr int W = kPeakStrip / 32;
  __shared__ uint32_t part[kWarps];
  wait_then_start_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // Strip s of row r; the warp's next is `down` rows and `across` strips on.
  const int64_t start = int64_t(blockIdx.x) * kWarps + warp;
  int64_t r = start < strips ? 0 : start / strips, s = start - r * strips;
  uint32_t most = 0;      // of the even and the odd columns
  while (r < rows) {
    uint4 v[kPeakAhead];
#pragma unroll
    for (int u = 0; u < kPeakAhead; ++u) {
      // (Single values are read with the lanes side by side.)
      const int64_t c = s * kPeakStrip + (VEC ? lane * W : lane);
      const uint16_t *const from = dy + r * ld + c;
      v[u] = make_uint4(0, 0, 0, 0);
      if (VEC && r < rows && c + W <= N) {
        v[u] = *reinterpret_cast<const uint4 *>(from);
      } else {
        constexpr int kNext = VEC ? 1 : 32;
#pragma unroll
        for (int k = 0; k < W; ++k)
          if (r < rows && c + kNext * k < N)
            reinterpret_cast<uint16_t *>(&v[u])[k] = from[kNext * k];
      }
      r += down;
      if ((s += across) >= strips) {
        s -= strips;
        ++r;
      }
    }
#pragma unroll
    for (int u = 0; u < kPeakAhead; ++u) {
      const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // Infinities and NaN, 0x7C00 and more without their signs, are left out.
        const uint32_t size = w[k] & 0x7FFF7FFFu, out = (size + 0x04000400u) & 0x80008000u;
        most = __vmaxu2(most, size & ~(out | (out - (out >> 15))));
      }
    }
  }
  most = __reduce_max_sync(~0u, max(most & 0xFFFFu, most >> 16));
  if (lane == 0) part[warp] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWarps; ++w) most = max(most, part[w]);
    peaks[blockIdx.x] = most;
  }
}

// The power of two that brings the FP16 value of these bits to between 2^14 and 2^15 (1 for 0): 2^-1 to
// 2^38.
__device__ __forceinline__ float scale_of(uint32_t bits) {
  const int power = bits >> 10 ? int(bits >> 10) - 15 : 31 - __clz(int(bits)) - 24;
  return bits == 0 ? 1.0f : __int_as_float((14 - power + 127) << 23);
}

// Lane l has columns first + l W .. + W, 16 bytes' worth, read as vectors (VEC) or one by one; dz's rows
// are vectors in any case, whose last may have values past N that nothing reads (4096 x 4095, bf16, with
// the sums: 34 us where values are read and written one by one with 32 lanes side by side, 26 so).
// SCALED: dz times a power of two (FP16).
template <typename T, bool VEC, bool SCALED>
__global__ void __launch_bounds__(32 * kWarps)
slopes_kernel(const __grid_constant__ SlopeParams p) {
  constexpr int W = Vec<T>::kCount;
  __shared__ float part[kWarps][32 * W];
  wait_then_start_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t scale = 0;
  if constexpr (SCALED) {
    __shared__ uint32_t peak[kWarps];
    uint32_t most = 0;
    for (int i = threadIdx.x; i < p.peak_count; i += 32 * kWarps) most = max(most, p.peaks[i]);
    most = __reduce_max_sync(~0u, most);
    if (lane == 0) peak[warp] = most;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) most = max(most, peak[w]);
    const float f = scale_of(most);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.unscale = 1.0f / f;
    scale = both(f);
  }
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
        if constexpr (SCALED) d[k] = mul2(d[k], scale);
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
runs_kernel(const float *sums, int64_t runs, int64_t N, float *dbias) {
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
// sums alone: 19 us, by four blocks 23; reading takes the memory 10 us, and a warp asks for its next rows
// only after the slopes of these).  Of 4096 rows at most, however wide the matrix: a thread adds an eighth
// of a run one after another (65536 FP32 rows of 29312 in one run: off by up to 2046 half steps of the
// sum, in runs by at most 530).  The number of SMs is that of the GPU this is built for and not asked:
// workspaces and results then depend on the sizes alone.
constexpr int kSMs = 152, kLongestRun = 4096, kMostRuns = 65535;      // (of a grid's second dimension)
int64_t runs_of(int64_t rows, int64_t N, int dtype) {
  const int64_t strip = dtype == TMM_F32 ? 128 : 256, strips = (N + strip - 1) / strip;
  const int64_t want = std::max<int64_t>(3 * kSMs / strips, (rows + kLongestRun - 1) / kLongestRun);
  return std::max<int64_t>(1, std::min({want, (rows + 31) / 32, int64_t(kMostRuns)}));
}

bool aligned(const void *p, int64_t ld, int64_t size) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * size % 16 == 0;
}

template <typename T>
cudaError_t launch_as(const LinearGradProblem &g, void *dz, int64_t ldz, bool planes,
                      float *unscale, float *partial, cudaStream_t stream) {
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
  cfg.blockDim = dim3(32 * kWarps, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (unscale) {
    uint32_t *const peaks = reinterpret_cast<uint32_t *>(unscale) + 1;
    const bool flat = p.lddy == g.N || g.rows == 1;
    const int64_t rows = flat ? 1 : g.rows, N = flat ? g.rows * g.N : g.N;
    const int64_t strips = (N + kPeakStrip - 1) / kPeakStrip;
    p.peaks = peaks;
    p.peak_count = int(std::min<int64_t>(kMaxPeaks, (rows * strips + kWarps - 1) / kWarps));
    p.unscale = unscale;
    const int64_t step = int64_t(p.peak_count) * kWarps, down = step / strips;
    cfg.gridDim = dim3(unsigned(p.peak_count), 1, 1);
    const auto kernel = aligned(p.dy, flat ? 0 : p.lddy, 2) ? peaks_kernel<true> : peaks_kernel<false>;
    if ((e = cudaLaunchKernelEx(&cfg, kernel, static_cast<const uint16_t *>(p.dy), rows, N, p.lddy,
                                strips, down, step - down * strips, peaks)) != cudaSuccess)
      return e;
  }
  cfg.gridDim = dim3(unsigned((g.N + strip - 1) / strip), unsigned(runs), 1);
  auto kernel = vec ? slopes_kernel<T, true, false> : slopes_kernel<T, false, false>;
  if constexpr (std::is_same_v<T, __half>)
    if (unscale) kernel = vec ? slopes_kernel<T, true, true> : slopes_kernel<T, false, true>;
  e = cudaLaunchKernelEx(&cfg, kernel, p);
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

size_t linear_unscale_bytes() { return sizeof(uint32_t) * (1 + kMaxPeaks); }

cudaError_t launch_linear_slopes(const LinearGradProblem &p, void *dz, int64_t ldz, bool planes,
                                 float *unscale, float *partial, cudaStream_t stream) {
  if (p.dtype == TMM_BF16)
    return launch_as<__nv_bfloat16>(p, dz, ldz, planes, nullptr, partial, stream);
  if (p.dtype == TMM_F16) return launch_as<__half>(p, dz, ldz, planes, unscale, partial, stream);
  return launch_as<float>(p, dz, ldz, planes, nullptr, partial, stream);
}

}  // namespace tmm
