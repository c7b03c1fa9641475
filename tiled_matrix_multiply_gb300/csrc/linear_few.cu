// linear_few.cu -- linear layers of few rows in FP32: y = act(x w + bias) + residual on the FP32 units.
//
// Reading w is the bound, 4 bytes a value once; the tensor cores' way (gemm_linear.cu) reads and writes
// 16 for the bf16 parts of each.  Sixteen rows take the FP32 units 0.7 of the time that w takes the
// memory (256 operations a cycle and SM).
//
// A block does 128 columns and 16 rows at most over a run of k, a cluster of up to eight blocks all of k.
// Each of its eight warps takes its own k and sums for all the rows, pairs of rows an instruction
// (fma.rn.f32x2: x is in shared memory as [k][row], so that pairs come as they are).  w stored K x N is
// read as it is used, four columns a lane; stored N x K it passes through shared memory in tiles of 128
// columns x 32 k, whose rows of 36 values are free of bank conflicts.  The warps' sums, then the
// blocks', are added in order.
// Measured (4096 x 4096 stored K x N, gelu and residual; w takes the memory 10 us): 1 row 18 us, 8
// rows 22, 16 rows 29 (stored N x K 22, 24, 30); by way of the parts 44.  Seventeen to 32 rows in two
// runs of sixteen took 48 us, no less than the parts' 47.
#include <cstdint>

#include "activation.cuh"
#include "grouped.h"
#include "row_ops.cuh"
#include "tensor_core.cuh"
#include "tmm_gemm.h"

namespace tmm {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kColumns = 128;
constexpr int kRun = 256;        // k whose x is in shared memory at a time
constexpr int kTile = 32;        // k of a tile of w stored N x K
constexpr int kPitch = kTile + 4;

struct FewParams {
  int M, N, K;
  const float *x, *w;
  int64_t ldx, ldw;
  const float *bias;
  int act;
  const float *residual;
  int64_t ld_residual;
  float *y;
  int64_t ldy;
  float *pre;
  int64_t ld_pre;
  int vec;               // w's rows on 16-byte boundaries, and whole vectors of them
};

// Shared memory: x and a tile of w, then over them the warps' sums; and the block's.
template <int ROWS>
struct Shared {
  static constexpr int kOperands = kRun * ROWS + kColumns * kPitch, kSums = kWarps * ROWS * kColumns;
  static constexpr int kPart = kOperands > kSums ? kOperands : kSums;
  static constexpr int kBytes = int(sizeof(float)) * (kPart + ROWS * kColumns);
};

// MN: w is stored K x N.  Of a lane's four columns, the i-th.
template <bool MN>
__device__ __forceinline__ int column(const FewParams &p, int lane, int i) {
  return MN && p.vec ? 4 * lane + i : lane + 32 * i;
}

// acc += the products of one k: x of all rows with four values of w.
template <int ROWS>
__device__ __forceinline__ void add_products(uint64_t (&acc)[ROWS / 2][4], const float *x,
                                             const float (&w)[4]) {
  uint64_t two[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) two[i] = both(w[i]);
#pragma unroll
  for (int r = 0; r < ROWS / 2; ++r) {
    const uint64_t v = *reinterpret_cast<const uint64_t *>(x + 2 * r);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[r][i] = fma2(v, two[i], acc[r][i]);
  }
}

template <int ROWS, bool MN>
__global__ void __launch_bounds__(kThreads, 2)
few_kernel(const __grid_constant__ FewParams p, int split) {
  extern __shared__ __align__(16) float shared[];
  float *const xs = shared, *const ws = shared + kRun * ROWS, *const sums = shared;
  float *const part = shared + Shared<ROWS>::kPart;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int panel = int(blockIdx.x) / split, rank = int(blockIdx.x) - panel * split;
  const int n0 = panel * kColumns;
  // This block's k, in whole tiles.
  const int tiles = (p.K + kTile - 1) / kTile;
  const int k0 = tiles * rank / split * kTile, k1 = min(p.K, tiles * (rank + 1) / split * kTile);
  wait_then_start_next();

  uint64_t acc[ROWS / 2][4];
#pragma unroll
  for (int r = 0; r < ROWS / 2; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[r][i] = 0;
  for (int begin = k0; begin < k1; begin += kRun) {
    const int run = min(kRun, k1 - begin);
    __syncthreads();      // the run before has been used
    for (int i = tid; i < kRun * ROWS; i += kThreads) {
      const int r = i / kRun, k = i - r * kRun;
      xs[k * ROWS + r] = r < p.M && k < run ? p.x[r * p.ldx + begin + k] : 0.0f;
    }
    __syncthreads();
    if constexpr (MN) {
      constexpr int kAhead = 8;
      for (int k = warp; k < run; k += kWarps * kAhead) {
        float w[kAhead][4];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int at = k + u * kWarps;
          const float *const from = p.w + int64_t(begin + at) * p.ldw + n0;
          if (p.vec) {
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (at < run && n0 + 4 * lane < p.N) v = reinterpret_cast<const float4 *>(from)[lane];
            w[u][0] = v.x;
            w[u][1] = v.y;
            w[u][2] = v.z;
            w[u][3] = v.w;
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[u][i] = at < run && n0 + lane + 32 * i < p.N ? from[lane + 32 * i] : 0.0f;
          }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (k + u * kWarps < run)      // (0 times what is not there might be NaN)
            add_products<ROWS>(acc, xs + (k + u * kWarps) * ROWS, w[u]);
      }
    } else {
      // Eight threads a row of a tile, four k each, four rows a thread; the next tile on its way.
      const int row = tid >> 3, at = (tid & 7) * 4;
      float4 next[4];
      const auto fetch = [&](int k) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = n0 + row + 32 * j;
          const float *const from = p.w + int64_t(n) * p.ldw + begin + k + at;
          next[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (n >= p.N || k >= run) continue;
          if (p.vec && k + at + 4 <= run) {
            next[j] = *reinterpret_cast<const float4 *>(from);
          } else {
            if (k + at < run) next[j].x = from[0];
            if (k + at + 1 < run) next[j].y = from[1];
            if (k + at + 2 < run) next[j].z = from[2];
            if (k + at + 3 < run) next[j].w = from[3];
          }
        }
      };
      fetch(0);
      for (int k = 0; k < run; k += kTile) {
        if (k > 0) __syncthreads();      // the tile before has been used
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float4 *>(ws + (row + 32 * j) * kPitch + at) = next[j];
        __syncthreads();
        fetch(k + kTile);
        float4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = *reinterpret_cast<const float4 *>(ws + (lane + 32 * i) * kPitch + 4 * warp);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float w[4] = {(&v[0].x)[j], (&v[1].x)[j], (&v[2].x)[j], (&v[3].x)[j]};
          if (k + 4 * warp + j < run) add_products<ROWS>(acc, xs + (k + 4 * warp + j) * ROWS, w);
        }
      }
    }
  }
  // The warps' sums, over the operands.
  __syncthreads();
#pragma unroll
  for (int r = 0; r < ROWS / 2; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = of_pair(acc[r][i]);
      float *const to = sums + (warp * ROWS + 2 * r) * kColumns + column<MN>(p, lane, i);
      to[0] = f.x;
      to[kColumns] = f.y;
    }
  __syncthreads();
  for (int i = tid; i < ROWS * kColumns; i += kThreads) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sums[w * ROWS * kColumns + i];
    part[i] = s;
  }
  if (split > 1) cluster_sync();
  else __syncthreads();
  // This block's share of the results, pairs of neighbouring columns.
  constexpr int kPairs = ROWS * kColumns / 2, kMine = (kPairs + kThreads - 1) / kThreads;
  const int i0 = kPairs * rank / split, i1 = kPairs * (rank + 1) / split;
  uint64_t z[kMine];
  const uint32_t here = smem_u32(part);
#pragma unroll
  for (int j = 0; j < kMine; ++j) z[j] = 0;
  for (int r = 0; r < split; ++r) {
    const uint32_t from = split > 1 ? map_rank(here, uint32_t(r)) : here;
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int i = i0 + tid + j * kThreads;
      if (i >= i1) continue;
      uint64_t v;
      asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(from + i * 8) : "memory");
      z[j] = r == 0 ? v : add2(z[j], v);
    }
  }
  // The others may leave once their sums have been read.
  if (split > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int i = i0 + tid + j * kThreads;
    const int row = i / (kColumns / 2), n = n0 + 2 * (i - row * (kColumns / 2));
    if (i >= i1 || row >= p.M || n >= p.N) continue;
    const bool two = n + 1 < p.N;
    const int64_t at = row;
    if (p.bias) z[j] = add2(z[j], pair_of(p.bias[n], two ? p.bias[n + 1] : 0.0f));
    if (p.pre) {
      const float2 f = of_pair(z[j]);
      p.pre[at * p.ld_pre + n] = f.x;
      if (two) p.pre[at * p.ld_pre + n + 1] = f.y;
    }
    uint64_t v[1] = {z[j]};
    activate_pairs<false>(p.act, v);
    float2 f = of_pair(v[0]);
    if (p.residual) {
      f.x += p.residual[at * p.ld_residual + n];
      if (two) f.y += p.residual[at * p.ld_residual + n + 1];
    }
    p.y[at * p.ldy + n] = f.x;
    if (two) p.y[at * p.ldy + n + 1] = f.y;
  }
  if (split > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

template <int ROWS, bool MN>
cudaError_t launch_as(const FewParams &p, const DeviceInfo &dev, cudaStream_t stream) {
  const auto kernel = few_kernel<ROWS, MN>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Shared<ROWS>::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t panels = (p.N + kColumns - 1) / kColumns;
  // Two blocks an SM, of eight tiles of k at least.
  int split = 1;
  while (split < 8 && panels * split * 2 <= 2 * dev.sm_count &&
         (p.K + kTile - 1) / kTile >= 16 * split)
    split *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(unsigned(panels * split), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Shared<ROWS>::kBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p, split);
}

}  // namespace

cudaError_t launch_linear_few(const LinearProblem &g, const DeviceInfo &dev, cudaStream_t stream) {
  FewParams p = {};
  p.M = int(g.rows);
  p.N = int(g.N);
  p.K = int(g.K);
  p.x = static_cast<const float *>(g.x.data);
  p.ldx = g.x.ld;
  p.w = static_cast<const float *>(g.w.data);
  p.ldw = g.w.ld;
  p.bias = static_cast<const float *>(g.bias);
  p.act = g.act;
  p.residual = static_cast<const float *>(g.residual);
  p.ld_residual = g.ld_residual;
  p.y = static_cast<float *>(g.y);
  p.ldy = g.ldy;
  p.pre = static_cast<float *>(g.pre);
  p.ld_pre = g.ld_pre;
  p.vec = (reinterpret_cast<uintptr_t>(p.w) & 15u) == 0 && p.ldw % 4 == 0 &&
          (g.trans_w || g.N % 4 == 0);
  const auto launch = [&](auto mn) {
    constexpr bool MN = decltype(mn)::value;
    if (g.rows <= 2) return launch_as<2, MN>(p, dev, stream);
    if (g.rows <= 4) return launch_as<4, MN>(p, dev, stream);
    if (g.rows <= 8) return launch_as<8, MN>(p, dev, stream);
    return launch_as<16, MN>(p, dev, stream);
  };
  return g.trans_w ? launch(std::false_type()) : launch(std::true_type());
}

}  // namespace tmm
