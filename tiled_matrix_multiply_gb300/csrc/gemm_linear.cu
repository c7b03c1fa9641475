// gemm_linear.cu -- the product of a linear layer and of its gradients, 16-bit operands, on the tcgen05
// tensor cores, with the layer's epilogue (linear_epilogue.cuh).
//
//   D[n, q] = sum_k P[n, k] Q[q, k]:  the result's contiguous dimension n on the tensor-memory lanes, its
//   rows q on the columns.
//   forward   P = w^T, Q = x;     dx: P = w, Q = dz;     dw: P = dz^T, Q = x^T.
// Either operand may be stored with k or with its own dimension contiguous: both are read in place
// (K-major and MN-major tiles in 128-byte swizzle).
//
// Two shapes, chosen by an estimate of their cycles (dense_shape):
//   pairs  (CG = 2): 256 lanes x up to 256 columns on two SMs (cta_group::2), each staging half of
//          the columns.  Tensor memory holds two tiles, so that one's results leave it while the next
//          is summed.  For large products.
//   single (CG = 1): 128 lanes x up to 256 columns; where tiles are few, up to eight blocks of a
//          cluster share a tile's sum, leave their parts in their shared memory (where the ring was)
//          and each finish a share of the columns.  Reading the weights is the bound then, and more
//          blocks read faster.
// A warp copies (one thread: tensor copies into a ring of stages), one issues the products (one
// thread), eight take results out.  Every wait is bounded (globaltimer); on timeout bit 1 of the
// status word is set and the kernel runs to its end.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "grouped.h"
#include "linear_epilogue.cuh"
#include "tensor_core.cuh"
#include "tmm_gemm.h"

namespace tmm {

__device__ unsigned int g_linear_status;

namespace {

constexpr int kBK = 64;                  // values of a K slice: one 128-byte swizzle row
constexpr int kEpiWarps = 8, kEpi0 = 2;  // result warps, the first of them
constexpr int kThreads = 32 * (kEpi0 + kEpiWarps);
constexpr uint32_t kPTile = 128 * 128;   // 128 lanes x 64 values: 16 KiB
constexpr int kWidest = 256;             // columns of a tile, and of one of the two sums
constexpr int kMaxStages = 10;
constexpr int kOutStage = 2048;          // bytes of a result warp
constexpr uint32_t kMaxSmem = 232448;    // 227 KiB
constexpr uint32_t kFixed = 1024 + kEpiWarps * kOutStage + 8 * (2 * kMaxStages + 5) + 16;
// Slices of one tensor-memory sum at most: its additions do not round to nearest (2^-24 of the partial
// sum each, 512 of them here: 2^-15, a sixteenth of FP16's rounding).
constexpr int kLong = 128;

template <bool BF16>
struct DenseParams {
  static constexpr int out_type = BF16 ? kOutBF16 : kOutF16;
  int M, N, K;             // rows of the result (columns of a tile), its columns (lanes), the sum
  int bn;                  // columns of a tile
  int panels, q_tiles;     // tiles along N and along M
  int stages, ksplit;
  int p_mn, q_mn;          // operands stored with their own dimension contiguous
  uint32_t idesc;
  void *out;
  int64_t ld_out;
  int vec_out;             // everything of the result's shape on 16-byte rows
  const void *bias;
  int bias_f32, act;
  const void *residual;
  int64_t ld_residual;
  void *pre;
  int64_t ld_pre;
  int64_t wait_limit_ns;
  int drop_block;          // testing hook: this block waits for bytes that never come (-1: none)
};

struct DenseTile {
  int n0, q0;
};
// Tiles in bands of eight along M, so that those in flight share their operands.
template <typename Params>
__device__ __forceinline__ DenseTile tile_at(const Params &p, int t, int lanes) {
  const int band = 8 * p.panels, b = t / band;
  const int wide = min(8, p.q_tiles - 8 * b), i = t - b * band;
  const int panel = i / wide;
  return {panel * lanes, (8 * b + i - panel * wide) * p.bn};
}

// Four results of one row: n to n + 3.
template <typename Params>
__device__ __forceinline__ void finish_four(const Params &p, int64_t row, int n, float (&z)[4]) {
  if (!p.vec_out || n + 4 > p.N) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (n + k < p.N) linear_one<1>(p, row, n + k, z[k]);
    return;
  }
  if (p.pre)
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.pre) + row * p.ld_pre + n) =
        make_uint2(pack_results(p, z[0], z[1]), pack_results(p, z[2], z[3]));
  activate_all<4>(p.act, z);
  if (p.residual) {
    const uint2 r = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.residual) +
                                                     row * p.ld_residual + n);
    const float2 a = unpack_values(p, r.x), b = unpack_values(p, r.y);
    z[0] += a.x;
    z[1] += a.y;
    z[2] += b.x;
    z[3] += b.y;
  }
  *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + row * p.ld_out + n) =
      make_uint2(pack_results(p, z[0], z[1]), pack_results(p, z[2], z[3]));
}

template <int CG, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
dense_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
             const __grid_constant__ DenseParams<BF16> p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;    // the same offset in every block
  const int mine = p.bn / CG;                      // columns that this block stages
  const uint32_t stage_bytes = kPTile + uint32_t(mine) * 128;
  const uint32_t out_stage = base + p.stages * stage_bytes;
  const uint32_t bar_full = out_stage + kEpiWarps * kOutStage;
  const uint32_t bar_empty = bar_full + 8 * kMaxStages;
  const uint32_t bar_tfull = bar_empty + 8 * kMaxStages;
  const uint32_t bar_tempty = bar_tfull + 16;      // pairs: used in the leader
  const uint32_t bar_drain = bar_tempty + 16;
  const uint32_t slot = bar_drain + 8;             // tensor memory address
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = CG == 1 || rank == 0;
  const int half = CG == 2 ? int(rank) : 0;        // which 128 lanes, which half of the columns

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_tfull + 8 * b, 1);
      mbar_init(bar_tempty + 8 * b, CG * kEpiWarps);
    }
    mbar_init(bar_drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_map(&map_p);
    prefetch_map(&map_q);
  }
  if (warp == 1) {
    if constexpr (CG == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(slot)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(slot)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();   // barriers exist before any remote arrival
  tc_fence_after();
  const uint32_t tmem =
      *reinterpret_cast<volatile uint32_t *>(smem_raw + (slot - raw));
  grid_wait();
  grid_start_next();

  const int share = CG == 2 ? 2 : p.ksplit;        // blocks of a tile
  const int first = int(blockIdx.x) / share, step = int(gridDim.x) / share;
  const int tiles = p.panels * p.q_tiles;
  const int all = (p.K + kBK - 1) / kBK;           // slices, [s0, s1) of them this block's
  const int s0 = CG == 2 ? 0 : int(int64_t(all) * rank / p.ksplit);
  const int s1 = CG == 2 ? all : int(int64_t(all) * (rank + 1) / p.ksplit);
  bool timed_out = false;
  uint32_t q = 0;                                  // tiles so far

  if (warp == 0) {
    // ---- copies ----
    if (elect_one()) {
      bool dropped = int(blockIdx.x) == p.drop_block;
      int stage = 0;
      uint32_t parity = 1;
      for (int t = first; t < tiles && !timed_out; t += step) {
        const DenseTile tile = tile_at(p, t, 128 * CG);
        const int n0 = tile.n0 + 128 * half, q0 = tile.q0 + mine * half;
        for (int s = s0; s < s1; ++s) {
          if (!mbar_wait(bar_empty + 8 * stage, parity, p.wait_limit_ns)) {
            timed_out = true;
            break;
          }
          const uint32_t to = base + stage * stage_bytes, k0 = s * kBK;
          uint32_t bar = bar_full + 8 * stage;
          if (leader) {
            mbar_expect(bar, CG * stage_bytes + (dropped ? 16 : 0));
            dropped = false;
          }
          if (CG == 2) bar = map_rank(bar, 0);
          if (p.p_mn) {
            tma_2d<CG>(to, &map_p, n0, k0, bar);
            tma_2d<CG>(to + 8192, &map_p, n0 + 64, k0, bar);
          } else {
            tma_2d<CG>(to, &map_p, k0, n0, bar);
          }
          if (p.q_mn) {
            for (int c = 0; c < mine; c += 64)
              tma_2d<CG>(to + kPTile + c * 128, &map_q, q0 + c, k0, bar);
          } else {
            tma_2d<CG>(to + kPTile, &map_q, k0, q0, bar);
          }
          if (++stage == p.stages) {
            stage = 0;
            parity ^= 1;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- products ----
    if (leader && elect_one()) {
      const uint32_t idesc = p.idesc | (uint32_t(p.bn >> 3) << 17) |
                             (uint32_t(128 * CG >> 4) << 24) | (p.p_mn ? 1u << 15 : 0u) |
                             (p.q_mn ? 1u << 16 : 0u);
      const uint32_t pstep = p.p_mn ? 128 : 2, qstep = p.q_mn ? 128 : 2;   // 16 k, in 16 bytes
      int stage = 0;
      uint32_t parity = 0;
      for (int t = first; t < tiles && !timed_out; t += step, ++q) {
        const uint32_t d = tmem + (q & 1) * kWidest;
        if (q >= 2 &&
            !mbar_wait(bar_tempty + 8 * (q & 1), ((q >> 1) - 1) & 1u, p.wait_limit_ns)) {
          timed_out = true;
          break;
        }
        tc_fence_after();
        for (int s = s0; s < s1; ++s) {
          if (!mbar_wait(bar_full + 8 * stage, parity, p.wait_limit_ns)) {
            timed_out = true;
            break;
          }
          tc_fence_after();
          const uint32_t at = base + stage * stage_bytes;
          const uint64_t a = tile_desc(at, p.p_mn), b = tile_desc(at + kPTile, p.q_mn);
          const int steps = min(4, (p.K - s * kBK + 15) / 16);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < steps) mma<CG>(d, a + k * pstep, b + k * qstep, idesc, s > s0 || k > 0);
          mma_commit<CG>(bar_empty + 8 * stage, true);
          if (++stage == p.stages) {
            stage = 0;
            parity ^= 1;
          }
        }
        if (!timed_out) mma_commit<CG>(bar_tfull + 8 * (q & 1), true);
      }
      mma_commit<CG>(bar_drain, false);
      if (!mbar_wait(bar_drain, 0u, p.wait_limit_ns)) timed_out = true;
    }
    __syncwarp();
  } else {
    // ---- results ----
    const int quarter = warp & 3, odd = (warp - kEpi0) >> 2;
    const uint32_t lanes = tmem + (uint32_t(32 * quarter) << 16);
    const uint32_t tempty = CG == 2 ? map_rank(bar_tempty, 0) : bar_tempty;
    const uint32_t stage = out_stage + uint32_t(warp - kEpi0) * kOutStage;
    float *const parts = reinterpret_cast<float *>(smem_raw + (base - raw));
    for (int t = first; t < tiles; t += step, ++q) {
      const DenseTile tile = tile_at(p, t, 128 * CG);
      const int nw = tile.n0 + 128 * half + 32 * quarter, left = p.M - tile.q0;
      const bool split = CG == 1 && p.ksplit > 1;
      float bias[8] = {};
      if (p.bias && !split) {
        if (p.vec_out) {
#pragma unroll
          for (int k = 0; k < 8; ++k) bias[k] = linear_bias<1>(p, nw + (lane & 3) * 8 + k);
        } else {
          bias[0] = linear_bias<1>(p, nw + lane);
        }
      }
      const bool ready = mbar_wait(bar_tfull + 8 * (q & 1), (q >> 1) & 1u, p.wait_limit_ns);
      if (!__all_sync(~0u, ready)) {
        timed_out = true;
        break;
      }
      tc_fence_after();
      for (int c0 = 16 * odd; c0 < p.bn && c0 < left; c0 += 32) {
        float v[16];
        __syncwarp();
        tmem_load_16(lanes + (q & 1) * kWidest + c0, v);
        if (split) {
#pragma unroll
          for (int j = 0; j < 16; ++j) parts[(c0 + j) * 128 + 32 * quarter + lane] = v[j];
        } else {
          linear_columns<1>(p, tile.q0 + c0, left - c0, nw, v, bias, stage);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed(tempty + 8 * (q & 1));
    }
  }

  if (CG == 1 && p.ksplit > 1) {
    // One tile, in parts of the sum: each block adds a share of its columns, in block order.
    __syncwarp();
    cluster_sync();
    if (warp >= kEpi0) {
      const DenseTile tile = tile_at(p, first, 128);
      const int qn = min(p.bn, p.M - tile.q0);
      const int c0 = qn * int(rank) / p.ksplit, c1 = qn * int(rank + 1) / p.ksplit;
      const int tid = int(threadIdx.x) - 32 * kEpi0, n = tile.n0 + (tid & 31) * 4;
      float bias[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) bias[k] = linear_bias<1>(p, n + k);
      for (int c = c0 + (tid >> 5); c < c1; c += kEpiWarps) {
        float z[4] = {};
#pragma unroll 4
        for (int r = 0; r < p.ksplit; ++r) {
          const float4 v =
              ld_cluster4(map_rank(base, uint32_t(r)) + uint32_t(c * 512 + (tid & 31) * 16));
          z[0] += v.x;
          z[1] += v.y;
          z[2] += v.z;
          z[3] += v.w;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) z[k] += bias[k];
        finish_four(p, tile.q0 + c, n, z);
      }
    }
    __syncwarp();
    cluster_sync();
  }
  if (timed_out && lane == 0) atomicOr(&g_linear_status, 2u);
  tc_fence_before();
  if (__syncthreads_or(timed_out)) {
    // Let the copies in flight land before the block goes away: one that was issued does within
    // microseconds.
    const uint64_t t0 = timer_ns();
    while (timer_ns() - t0 < 1000 * 1000) {
    }
  }
  if (CG == 2) cluster_sync();   // remote arrivals have landed; neither block uses tensor memory
  tc_fence_after();
  if (warp == 1) {
    if constexpr (CG == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// ---- host -------------------------------------------------------------------------------

std::atomic<int64_t> g_wait_limit_ns{int64_t(10) * 1000 * 1000 * 1000};
std::atomic<int> g_drop_block{-1};

struct DenseShape {
  int cg = 0;              // 0: none will do
  int bn = 0, split = 1;
};

// The shape of the fewest cycles, by an estimate: rounds of tiles times what a slice of 64 takes in
// one -- products at 4096 multiply-adds a cycle and SM, copies at 64 bytes -- and what comes before
// and after.
DenseShape dense_shape(const DenseProblem &p, int sms) {
  const int64_t slices = (p.K + kBK - 1) / kBK;
  DenseShape best;
  double least = 0;
  const auto consider = [&](int cg, int64_t bn, int split) {
    if ((slices + split - 1) / split > kLong || (split > 1 && slices < 2 * split)) return;
    const int64_t tiles = (p.N + 128 * cg - 1) / (128 * cg) * ((p.M + bn - 1) / bn);
    const int64_t slots = cg == 2 ? sms / 2 : sms / split;
    if (split > 1 && tiles > slots) return;
    const int64_t rounds = (tiles + slots - 1) / slots;
    const double slice = cg == 2 ? std::max(2 * bn, 256 + bn) : 256 + 2 * bn;
    const double cycles = double(rounds) * double((slices + split - 1) / split) * slice +
                          8.0 * double(bn) + (split > 1 ? 2500 + 6.0 * double(bn) : 0);
    if (best.cg == 0 || cycles < least) {
      best = {cg, int(bn), split};
      least = cycles;
    }
  };
  for (int cg = 1; cg <= 2; ++cg) {
    const int64_t unit = (p.q.mn ? 64 : 16) * cg;
    for (int64_t bn = unit; bn <= kWidest && bn < p.M + unit; bn += unit)
      for (int split = 1; split <= (cg == 1 ? 8 : 1); split *= 2) consider(cg, bn, split);
  }
  return best;
}

template <int CG, bool BF16>
cudaError_t launch_as(const DenseProblem &g, const DenseShape &s, const DeviceInfo &dev,
                      cudaStream_t stream) {
  auto kernel = dense_kernel<CG, BF16>;
  static std::atomic<uint64_t> configured{0};
  const uint64_t bit = uint64_t(1) << (dev.id & 63);
  cudaError_t e;
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMaxSmem));
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_release);
  }
  DenseParams<BF16> p = {};
  p.M = int(g.M);
  p.N = int(g.N);
  p.K = int(g.K);
  p.bn = s.bn;
  p.panels = int((g.N + 128 * CG - 1) / (128 * CG));
  p.q_tiles = int((g.M + s.bn - 1) / s.bn);
  p.ksplit = s.split;
  const uint32_t stage = kPTile + uint32_t(s.bn / CG) * 128;
  p.stages = int(std::min<uint32_t>(kMaxStages, (kMaxSmem - kFixed) / stage));
  p.p_mn = g.p.mn;
  p.q_mn = g.q.mn;
  // Instruction descriptor of kind::f16: D FP32 (bit 4), A and B bf16 (1 in bits 7-9 and 10-12) or
  // FP16 (0); majors and sizes are added in the kernel.
  p.idesc = (1u << 4) | (BF16 ? (1u << 7) | (1u << 10) : 0u);
  p.out = g.out;
  p.ld_out = g.ld_out;
  p.bias = g.bias;
  p.bias_f32 = g.bias_f32;
  p.act = g.act;
  p.residual = g.residual;
  p.ld_residual = g.residual ? g.ld_residual : 0;
  p.pre = g.pre;
  p.ld_pre = g.pre ? g.ld_pre : 0;
  p.vec_out = ((reinterpret_cast<uintptr_t>(p.out) | reinterpret_cast<uintptr_t>(p.residual) |
                reinterpret_cast<uintptr_t>(p.pre)) & 15u) == 0 &&
              p.ld_out % 8 == 0 && p.ld_residual % 8 == 0 && p.ld_pre % 8 == 0;
  p.wait_limit_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  p.drop_block = g_drop_block.load(std::memory_order_relaxed);
  CUtensorMap map_p, map_q;
  const auto encode = [&](CUtensorMap *m, const DenseOperand &o, uint32_t rows) {
    const uint64_t size[2] = {uint64_t(o.cols), uint64_t(o.rows)};
    const uint64_t stride[1] = {uint64_t(o.ld)};
    const uint32_t box[2] = {kBK, o.mn ? uint32_t(kBK) : rows};
    return encode_16bit(m, o.data, 2, size, stride, box);
  };
  if ((e = encode(&map_p, g.p, 128)) != cudaSuccess ||
      (e = encode(&map_q, g.q, uint32_t(s.bn / CG))) != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(CG == 2 ? 2 : s.split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kFixed + p.stages * stage;
  cfg.stream = stream;
  const int64_t tiles = int64_t(p.panels) * p.q_tiles, share = CG == 2 ? 2 : s.split;
  const int64_t slots = s.split > 1 ? tiles : dev.sm_count / share;
  cfg.gridDim = dim3(unsigned(share * std::max<int64_t>(1, std::min(tiles, slots))), 1, 1);
  return cudaLaunchKernelEx(&cfg, kernel, map_p, map_q, p);
}

}  // namespace

cudaError_t launch_dense(const DenseProblem &p, const DeviceInfo &dev, cudaStream_t stream) {
  if (p.dtype == TMM_F32 || p.K == 0 ||
      (p.N + 127) / 128 * ((p.M + 15) / 16) >= INT32_MAX / 16)
    return cudaErrorNotSupported;
  const DenseShape s = dense_shape(p, dev.sm_count);
  if (s.cg == 0) return cudaErrorNotSupported;
  if (p.dtype == TMM_BF16)
    return s.cg == 2 ? launch_as<2, true>(p, s, dev, stream) : launch_as<1, true>(p, s, dev, stream);
  return s.cg == 2 ? launch_as<2, false>(p, s, dev, stream) : launch_as<1, false>(p, s, dev, stream);
}

cudaError_t linear_device_status(unsigned int *status, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(status, g_linear_status, sizeof(unsigned int));
  if (e != cudaSuccess || !clear) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_linear_status, &zero, sizeof(unsigned int));
}

void linear_set_test_hooks(int drop_block, int64_t wait_limit_ns) {
  g_drop_block.store(drop_block, std::memory_order_relaxed);
  g_wait_limit_ns.store(wait_limit_ns > 0 ? wait_limit_ns : int64_t(10) * 1000 * 1000 * 1000,
                        std::memory_order_relaxed);
}

}  // namespace tmm
