// gemm_linear.cu -- linear layers: the product with one matrix for all rows and what follows it, and
// the products of its gradients, on the tcgen05 tensor cores.
//
//   D[n, q] = sum_k P[n, k] Q[q, k]:  the result's contiguous dimension n on the tensor-memory lanes, its
//   rows q on the columns.
//   forward   P = w^T, Q = x;     dx: P = w, Q = dz;     dw: P = dz^T, Q = x^T.
// Either operand may be stored with k or with its own dimension contiguous: both are read in place
// (K-major and MN-major tiles in 128-byte swizzle).
//
// FP32: every value is its three bf16 parts (split_bf16.cuh), made by a launch before; of the nine part
// products the three smallest (2^-24 of the term and less) are left out.  The leading one goes to one
// accumulator, the five others (2^-8 of it and less) to another; the tensor core's additions do not
// round to nearest, and a sum's error grows with the number of additions made in tensor memory (16
// values of K each), so that both are taken out every 128 values and added in FP32 registers.  For
// 16-bit operands a sum stays for 8192 values, 512 additions whose errors (2^-24 of the partial sum on
// the mean) come to 2^-15, a sixteenth of FP16's rounding; longer ones are taken out likewise.
//
// Two shapes, chosen by an estimate of their time (dense_shape):
//   pairs  (CG = 2): 256 lanes x up to 256 columns on two SMs (cta_group::2), each staging half of
//          the columns;
//   single (CG = 1): 128 lanes x up to 256 columns.
// Persistent where tiles are many: tensor memory holds two sums, so that one's results leave it while
// the next is made.  Where they are few, the blocks of a cluster of up to eight share a tile's sum: each
// leaves its part in its shared memory (where the ring was) and finishes a share of the columns.
// Reading the weights is the bound then, and more blocks read faster.
// A warp copies (one thread's tensor copies into a ring of stages), one issues the products (one
// thread's), sixteen take results out (with eight the results of a tile of one slice took 3.9 us, with
// sixteen 2.9).  Every wait is bounded (globaltimer); on timeout bit 1 of the status word is set and the
// kernel runs to its end.
// Measured (us, kernels alone, replayed from a graph): 8192 x 4096 x 4096 in bf16 plain 140 (1.96 PFLOP/s; a
// library's product 138), with gelu, residual and z kept 151 to 159 (called again and again, which the
// card's power slows down, 177 to 184); 512 x 4096 x 4096 16 to 17 (a library's 13.3); one row 8.3, where
// reading the weights takes 5.0; FP32 4096^3 with gelu and residual 492, six bf16 products at the library's
// rate 428.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "activation.cuh"
#include "grouped.h"
#include "row_ops.cuh"
#include "tensor_core.cuh"
#include "tmm_gemm.h"

namespace tmm {

__device__ unsigned int g_linear_status;

namespace {

constexpr int kBK = 64;                  // values of a K slice: one 128-byte swizzle row
constexpr int kEpiWarps = 16, kEpi0 = 2;  // result warps, the first of them
constexpr int kThreads = 32 * (kEpi0 + kEpiWarps);
constexpr uint32_t kPTile = 128 * 128;   // 128 lanes x 64 values: 16 KiB
constexpr int kWidest = 256;             // columns of a tile
constexpr int kWideSum = 128;            // of one whose sum is made of several (FP32: any)
constexpr int kMaxStages = 10;
constexpr int kShare = kWidest / 2 / kEpiWarps;      // columns of a thread in a shared sum, at most
constexpr uint32_t kMaxSmem = 232448;    // 227 KiB
// Slices of one tensor-memory sum at most.
constexpr int kLong = 128, kLongF32 = 2;

// What the operands and results are.
constexpr int kBF16 = 0, kF16 = 1, kF32 = 2;
template <int KIND>
struct Kind {
  static constexpr bool kSplit = KIND == kF32;
  static constexpr int kPlanes = kSplit ? 3 : 1;
  using T = std::conditional_t<KIND == kF32, float,
                               std::conditional_t<KIND == kF16, __half, __nv_bfloat16>>;
  // Bytes of a result warp: 16-bit results and residuals on their way.
  static constexpr uint32_t kOutStage = kSplit ? 0 : 2048;
  static constexpr uint32_t kFixed =
      1024 + kEpiWarps * kOutStage + 8 * (2 * kMaxStages + 5) + 16;
  __host__ __device__ static constexpr uint32_t stage(int columns) {      // of the block
    return kPlanes * (kPTile + uint32_t(columns) * 128);
  }
};

struct DenseParams {
  int M, N, K;             // rows of the result (columns of a tile), its columns (lanes), the sum
  int bn;                  // columns of a tile
  int panels, q_tiles;     // tiles along N and along M
  int stages, ksplit;
  int chunk;               // slices of a tensor-memory sum
  int p_mn, q_mn;          // operands stored with their own dimension contiguous
  uint32_t idesc;
  void *out;
  int64_t ld_out;
  int vec_out;             // everything of the result's shape on 16-byte rows
  const float *unscale;    // FP16: what the sums are multiplied by, or NULL
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
__device__ __forceinline__ DenseTile tile_at(const DenseParams &p, int t, int lanes) {
  const int band = 8 * p.panels, b = t / band;
  const int wide = min(8, p.q_tiles - 8 * b), i = t - b * band;
  const int panel = i / wide;
  return {panel * lanes, (8 * b + i - panel * wide) * p.bn};
}

// ---- results: z = sum + bias, y = act(z) + residual ------------------------------------------

// Sums of an operand that was kept times a power of two (see linear_slopes.cu).
template <int KIND>
__device__ __forceinline__ float unscale_of(const DenseParams &p) {
  return KIND == kF16 && p.unscale ? *p.unscale : 1.0f;
}
template <int KIND>
__device__ __forceinline__ uint64_t with_bias(uint64_t sum, float unscale, float bias) {
  if (KIND == kF16) return fma2(sum, both(unscale), both(bias));
  return add2(sum, both(bias));
}
template <int KIND>
__device__ __forceinline__ float bias_at(const DenseParams &p, int n) {
  if (p.bias == nullptr || n >= p.N) return 0.0f;
  if (p.bias_f32) return static_cast<const float *>(p.bias)[n];
  return float(static_cast<const typename Kind<KIND>::T *>(p.bias)[n]);
}
template <int KIND>
__device__ __forceinline__ uint32_t pack_results(float lo, float hi) {
  uint32_t w;
  if (KIND == kBF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
template <int KIND>
__device__ __forceinline__ float2 unpack_values(uint32_t w) {
  if (KIND == kBF16)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// Results n to n + 3 of one row, sum and bias in z.
template <int KIND>
__device__ __forceinline__ void finish_four(const DenseParams &p, int64_t row, int n,
                                            float (&z)[4]) {
  using T = typename Kind<KIND>::T;
  T *const out = static_cast<T *>(p.out) + row * p.ld_out + n;
  T *const pre = static_cast<T *>(p.pre) + row * p.ld_pre + n;
  const T *const residual = static_cast<const T *>(p.residual) + row * p.ld_residual + n;
  const bool whole = p.vec_out && n + 4 <= p.N;
  const auto store = [&](T *to) {
    if (!whole) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (n + k < p.N) to[k] = rounded<T>(z[k]);
    } else if constexpr (KIND == kF32) {
      *reinterpret_cast<float4 *>(to) = make_float4(z[0], z[1], z[2], z[3]);
    } else {
      *reinterpret_cast<uint2 *>(to) =
          make_uint2(pack_results<KIND>(z[0], z[1]), pack_results<KIND>(z[2], z[3]));
    }
  };
  float r[4] = {};
  if (p.residual && whole) {
    if constexpr (KIND == kF32) {
      const float4 v = *reinterpret_cast<const float4 *>(residual);
      r[0] = v.x;
      r[1] = v.y;
      r[2] = v.z;
      r[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2 *>(residual);
      const float2 a = unpack_values<KIND>(v.x), b = unpack_values<KIND>(v.y);
      r[0] = a.x;
      r[1] = a.y;
      r[2] = b.x;
      r[3] = b.y;
    }
  } else if (p.residual) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (n + k < p.N) r[k] = float(residual[k]);
  }
  if (p.pre) store(pre);
  uint64_t v[2] = {pair_of(z[0], z[1]), pair_of(z[2], z[3])};
  activate_pairs<KIND != kF32>(p.act, v);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float2 f = of_pair(v[k]);
    z[2 * k] = p.residual ? f.x + r[2 * k] : f.x;
    z[2 * k + 1] = p.residual ? f.y + r[2 * k + 1] : f.y;
  }
  store(out);
}

// 16 columns of a tile (rows of the result from row0 on, `count` of them), sums in v, for the one n of
// each lane: a warp writes 32 neighbours of a row.
template <int KIND>
__device__ __forceinline__ void finish_lanes(const DenseParams &p, int64_t row0, int count, int n,
                                             const float (&v)[16], float unscale, float bias) {
  using T = typename Kind<KIND>::T;
  if (n >= p.N) return;
  float r[16];
  const T *const residual = static_cast<const T *>(p.residual) + row0 * p.ld_residual + n;
  T *const out = static_cast<T *>(p.out) + row0 * p.ld_out + n;
  T *const pre = static_cast<T *>(p.pre) + row0 * p.ld_pre + n;
#pragma unroll
  for (int j = 0; j < 16; ++j)
    r[j] = p.residual && j < count ? float(residual[j * p.ld_residual]) : 0.0f;
  uint64_t z[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    z[j] = with_bias<KIND>(pair_of(v[2 * j], v[2 * j + 1]), unscale, bias);
  if (p.pre) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float2 f = of_pair(z[j >> 1]);
      if (j < count) pre[j * p.ld_pre] = rounded<T>(j & 1 ? f.y : f.x);
    }
  }
  activate_pairs<KIND != kF32>(p.act, z);
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float2 f = of_pair(z[j >> 1]);
    const float y = j & 1 ? f.y : f.x;
    if (j < count) out[j * p.ld_out] = rounded<T>(p.residual ? y + r[j] : y);
  }
}

// ---- one thread's instructions, issued by a whole warp ------------------------------------
//
// The copying and the multiplying warp run their loops as warps, and the one thread that acts is a
// predicate of the instruction: descriptors, addresses and counters then stay in the uniform registers
// that these instructions take.  (With the loops in a branch of one thread a product took 50 cycles to
// issue, 310 cycles a slice with its waits.)

template <int CG>
__device__ __forceinline__ void copy_if(uint32_t on, uint32_t dst, const CUtensorMap *map, int x,
                                        int y, int z, uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " @p cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];\n}\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(on)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " @p cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];\n}\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(on)
        : "memory");
}
__device__ __forceinline__ void expect_if(uint32_t on, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %2, 0;\n"
      " @p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}\n" ::"r"(bar),
      "r"(bytes), "r"(on)
      : "memory");
}
template <int CG>
__device__ __forceinline__ void mma_if(uint32_t on, uint32_t d, uint64_t a, uint64_t b,
                                       uint32_t idesc, uint32_t accumulate) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %3, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %4, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(accumulate), "r"(idesc), "r"(on)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %3, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %4, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(accumulate), "r"(idesc), "r"(on)
        : "memory");
}
// Arrive on `bar` of this block (of both blocks of the pair whose first has rank `head`) once the
// products issued so far by the thread have completed.
template <int CG>
__device__ __forceinline__ void commit_if(uint32_t on, uint32_t bar, uint32_t head) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %2, 0;\n"
        " @p tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
        ".multicast::cluster.b64 [%0], %1;\n}\n" ::"r"(bar),
        "h"(uint16_t(3u << head)), "r"(on)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %1, 0;\n"
        " @p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
            bar),
        "r"(on)
        : "memory");
}
// Whether the phase has passed already, for a look ahead.
__device__ __forceinline__ bool mbar_passed(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// A wait of a whole warp; the same answer in all lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int64_t limit_ns) {
  if (__all_sync(~0u, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = timer_ns();
  while (!__all_sync(~0u, mbar_try_wait(bar, parity)))
    if (__any_sync(~0u, int64_t(timer_ns() - t0) > limit_ns)) return false;
  return true;
}

// ---- results in 16 bits --------------------------------------------------------------------

// 16 columns of a tile (rows of the result) for the 32 n of a warp, all of them inside the result, as
// tmem_load_matrices leaves lanes 16 i to 16 i + 15 in f[i]: pairs of neighbouring columns of one n,
// which the bias, the activation and the residual are added to as they are.  Matrix instructions
// transpose 16-bit values on their way to shared memory (results) and from it (the residual), so that
// memory is read and written 16 bytes a lane: about 45 instructions and the activation's, where
// values staged in FP32 took 260.
template <int KIND>
__device__ __forceinline__ void finish_block(const DenseParams &p, int64_t row0, int nw,
                                             const uint32_t (&f)[2][8], float unscale,
                                             const float (&bias)[4], const uint4 (&residual)[2], uint32_t stage) {
  const int lane = threadIdx.x & 31;
  const auto piece = [&](uint32_t at, int row, int c) {      // free of bank conflicts
    return at + uint32_t(row * 64 + ((c ^ (row >> 1 & 3)) << 4));
  };
  uint64_t z[2][4];      // [8 columns][8 n]
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int m = 0; m < 4; ++m)
      z[c][m] = with_bias<KIND>(pair_of(__uint_as_float(f[m >> 1][4 * c + 2 * (m & 1)]),
                                        __uint_as_float(f[m >> 1][4 * c + 2 * (m & 1) + 1])),
                                unscale, bias[m]);
  __syncwarp();      // the reads of the block before are done
  if (p.residual) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                       piece(stage + 1024, (lane >> 2) + 8 * i, lane & 3)),
                   "r"(residual[i].x), "r"(residual[i].y), "r"(residual[i].z), "r"(residual[i].w)
                   : "memory");
    __syncwarp();
  }
  // The matrices' rows: 8 c + lane % 8, n from 8 (lane / 8) on.
  const auto put = [&](uint16_t *to, int64_t ld) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t h[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float2 v = of_pair(z[c][m]);
        h[m] = pack_results<KIND>(v.x, v.y);
      }
      asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                       piece(stage, 8 * c + (lane & 7), lane >> 3)),
                   "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                   : "memory");
    }
    __syncwarp();
    uint16_t *const dst = to + (row0 + (lane >> 2)) * ld + nw + (lane & 3) * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint4 w;
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                   : "r"(piece(stage, (lane >> 2) + 8 * i, lane & 3))
                   : "memory");
      *reinterpret_cast<uint4 *>(dst + i * 8 * ld) = w;
    }
  };
  if (p.pre) {
    put(static_cast<uint16_t *>(p.pre), p.ld_pre);
    __syncwarp();
  }
  activate_pairs<true>(p.act, z[0]);
  activate_pairs<true>(p.act, z[1]);
  if (p.residual) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t r[4];
      asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                   : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                   : "r"(piece(stage + 1024, 8 * c + (lane & 7), lane >> 3))
                   : "memory");
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float2 v = unpack_values<KIND>(r[m]);
        z[c][m] = add2(z[c][m], pair_of(v.x, v.y));
      }
    }
  }
  put(static_cast<uint16_t *>(p.out), p.ld_out);
}

template <int CG, int KIND>
__global__ void __launch_bounds__(kThreads, 1)
dense_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
             const __grid_constant__ DenseParams p) {
  using D = Kind<KIND>;
  constexpr int kWide = D::kSplit ? kWideSum : kWidest;      // columns from one sum to the next
  constexpr uint32_t kLower = 2 * kWide;                     // and to the lower parts' products
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;    // the same offset in every block
  const int mine = p.bn / CG;                      // columns that this block stages
  const uint32_t stage_bytes = D::stage(mine), q_tile = uint32_t(mine) * 128;
  const uint32_t out_stage = base + p.stages * stage_bytes;
  const uint32_t bar_full = out_stage + kEpiWarps * D::kOutStage;
  const uint32_t bar_empty = bar_full + 8 * kMaxStages;
  const uint32_t bar_tfull = bar_empty + 8 * kMaxStages;
  const uint32_t bar_tempty = bar_tfull + 16;      // pairs: used in the leader
  const uint32_t bar_drain = bar_tempty + 16;
  const uint32_t slot = bar_drain + 8;             // tensor memory address
  const int warp = __shfl_sync(~0u, int(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
  // Of a cluster's blocks, CG make a tile's part, ksplit parts its sum.
  const uint32_t rank = cluster_rank();
  const int half = CG == 2 ? int(rank & 1) : 0;    // which 128 lanes, which half of the columns
  const int part = int(rank) / CG;                 // of the sum
  const uint32_t head = rank - half;               // the pair's leader
  const bool leader = half == 0;
  const int share = CG * p.ksplit;                 // blocks of a tile
  const int first = int(blockIdx.x) / share, step = int(gridDim.x) / share;
  const int tiles = p.panels * p.q_tiles;
  const int all = (p.K + kBK - 1) / kBK;           // slices, [s0, s1) of them this block's
  const int s0 = all * part / p.ksplit, s1 = all * (part + 1) / p.ksplit;
  DenseTile tile = tile_at(p, first, 128 * CG);

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
    if (p.K > 0) {      // (no maps for an empty sum)
      prefetch_map(&map_p);
      prefetch_map(&map_q);
    }
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

  const int n = s1 - s0;
  const int sums = max(1, (n + p.chunk - 1) / p.chunk);      // tensor-memory sums of a tile
  const int total = first < tiles ? (tiles - first + step - 1) / step * sums : 0;      // of the block
  bool timed_out = false;
  int q = 0;                                       // sums so far

  if (warp == 0) {
    // ---- copies ----
    const uint32_t on = elect_one(), lead = on && leader;
    const uint32_t bytes = CG * stage_bytes;
    uint32_t extra = int(blockIdx.x) == p.drop_block ? 16 : 0;
    int stage = 0;
    uint32_t parity = 1;
    bool ahead = false;      // the next stage is known to be free
    for (int t = first; t < tiles && !timed_out;) {
      const int n0 = tile.n0 + 128 * half, q0 = tile.q0 + mine * half;
      for (int s = s0; s < s1; ++s) {
        if (!ahead && !warp_wait(bar_empty + 8 * stage, parity, p.wait_limit_ns)) {
          timed_out = true;
          break;
        }
        const uint32_t to = base + stage * stage_bytes;
        const int k0 = s * kBK;
        uint32_t bar = bar_full + 8 * stage;
        expect_if(lead, bar, bytes + extra);
        extra = 0;
        if (CG == 2) bar = map_rank(bar, head);
        if (++stage == p.stages) {
          stage = 0;
          parity ^= 1;
        }
        const bool next = mbar_passed(bar_empty + 8 * stage, parity);
#pragma unroll
        for (int pl = 0; pl < D::kPlanes; ++pl) {
          const uint32_t at = to + pl * kPTile, qt = to + D::kPlanes * kPTile + pl * q_tile;
          if (p.p_mn) {
            copy_if<CG>(on, at, &map_p, n0, k0, pl, bar);
            copy_if<CG>(on, at + 8192, &map_p, n0 + 64, k0, pl, bar);
          } else {
            copy_if<CG>(on, at, &map_p, k0, n0, pl, bar);
          }
          if (p.q_mn) {
            for (int c = 0; c < mine; c += 64)
              copy_if<CG>(on, qt + c * 128, &map_q, q0 + c, k0, pl, bar);
          } else {
            copy_if<CG>(on, qt, &map_q, k0, q0, pl, bar);
          }
        }
        ahead = __all_sync(~0u, next);
      }
      if ((t += step) < tiles) tile = tile_at(p, t, 128 * CG);
    }
  } else if (warp == 1) {
    // ---- products ----
    if (leader) {
      const uint32_t on = elect_one();
      const uint32_t idesc = p.idesc | (uint32_t(p.bn >> 3) << 17) |
                             (uint32_t(128 * CG >> 4) << 24) | (p.p_mn ? 1u << 15 : 0u) |
                             (p.q_mn ? 1u << 16 : 0u);
      const uint32_t pstep = p.p_mn ? 128 : 2, qstep = p.q_mn ? 128 : 2;   // 16 k, in 16 bytes
      int stage = 0;
      uint32_t parity = 0;
      bool ahead = false;    // the next stage is known to be full
      while (q < total && !timed_out) {
        for (int begin = s0; begin < s1 && !timed_out; begin += p.chunk, ++q) {
          const uint32_t d = tmem + (q & 1) * kWide;
          if (q >= 2 &&
              !warp_wait(bar_tempty + 8 * (q & 1), ((q >> 1) - 1) & 1u, p.wait_limit_ns)) {
            timed_out = true;
            break;
          }
          tc_fence_after();
          const int end = min(begin + p.chunk, s1);
          for (int s = begin; s < end; ++s) {
            if (!ahead && !warp_wait(bar_full + 8 * stage, parity, p.wait_limit_ns)) {
              timed_out = true;
              break;
            }
            tc_fence_after();
            const uint32_t at = base + stage * stage_bytes, empty = bar_empty + 8 * stage;
            const uint64_t a = tile_desc(at, p.p_mn);
            const uint64_t b = tile_desc(at + D::kPlanes * kPTile, p.q_mn);
            const int steps = min(4, (p.K - s * kBK + 15) / 16);
            if (++stage == p.stages) {
              stage = 0;
              parity ^= 1;
            }
            const bool next = mbar_passed(bar_full + 8 * stage, parity);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (k >= steps) break;
              const uint64_t x = a + k * pstep, y = b + k * qstep;
              const bool add = s > begin || k > 0;
              mma_if<CG>(on, d, x, y, idesc, add);
              if constexpr (D::kSplit) {
                constexpr uint64_t pa = kPTile >> 4;
                const uint64_t qa = q_tile >> 4;
                mma_if<CG>(on, d + kLower, x + 2 * pa, y, idesc, add);
                mma_if<CG>(on, d + kLower, x, y + 2 * qa, idesc, true);
                mma_if<CG>(on, d + kLower, x + pa, y + qa, idesc, true);
                mma_if<CG>(on, d + kLower, x + pa, y, idesc, true);
                mma_if<CG>(on, d + kLower, x, y + qa, idesc, true);
              }
            }
            commit_if<CG>(on, empty, head);
            ahead = __all_sync(~0u, next);
          }
          if (!timed_out) commit_if<CG>(on, bar_tfull + 8 * (q & 1), head);
        }
        if (n == 0) break;      // (an empty sum: K = 0)
      }
      commit_if<CG>(on, bar_drain, head);
      if (!warp_wait(bar_drain, 0u, p.wait_limit_ns)) timed_out = true;
    }
  } else {
    // ---- results ----
    const int quarter = warp & 3, turn = (warp - kEpi0) >> 2;
    const uint32_t lanes = tmem + (uint32_t(32 * quarter) << 16);
    const uint32_t tempty = CG == 2 ? map_rank(bar_tempty, head) : bar_tempty;
    const uint32_t stage = out_stage + uint32_t(warp - kEpi0) * D::kOutStage;
    float *const parts = reinterpret_cast<float *>(smem_raw + (base - raw));
    const bool split = p.ksplit > 1;
    const float unscale = unscale_of<KIND>(p);
    // Waits for the next sum, and hands it back.
    const auto ready = [&] {
      const bool ok = mbar_wait(bar_tfull + 8 * (q & 1), (q >> 1) & 1u, p.wait_limit_ns);
      if (!__all_sync(~0u, ok)) timed_out = true;
      tc_fence_after();
      return !timed_out;
    };
    const auto done = [&] {
      tc_fence_before();
      __syncwarp();
      // (Only where it is waited for: no arrival is under way when the pair's blocks end.)
      if (lane == 0 && q + 2 < total) mbar_arrive_relaxed(tempty + 8 * (q & 1));
      ++q;
    };
    for (int t = first; t < tiles;) {
      const int nw = tile.n0 + 128 * half + 32 * quarter, left = p.M - tile.q0;
      // 16-bit results in whole blocks of 16 columns and 32 n, all of it on 16-byte rows.
      const bool whole = !D::kSplit && !split && sums == 1 && n > 0 && p.vec_out && nw + 32 <= p.N;
      const auto one_n = [&](int c0, const float (&v)[16]) {
        if (split) {
#pragma unroll
          for (int j = 0; j < 16; ++j) parts[(c0 + j) * 128 + 32 * quarter + lane] = v[j];
        } else if (c0 < left) {
          finish_lanes<KIND>(p, tile.q0 + c0, min(16, left - c0), nw + lane, v,
                             unscale, bias_at<KIND>(p, nw + lane));
        }
      };
      if (!D::kSplit && sums == 1 && n > 0) {
        float bias[4] = {};
        if (p.bias && whole) {
#pragma unroll
          for (int k = 0; k < 4; ++k) bias[k] = bias_at<KIND>(p, nw + 8 * k + (lane >> 2));
        }
        const auto load_residual = [&](int c0, uint4 (&r)[2]) {
          if (p.residual == nullptr || !whole || c0 >= p.bn || left - c0 < 16) return;
          const uint16_t *const from = static_cast<const uint16_t *>(p.residual) +
                                       (tile.q0 + c0 + (lane >> 2)) * p.ld_residual + nw +
                                       (lane & 3) * 8;
          r[0] = *reinterpret_cast<const uint4 *>(from);
          r[1] = *reinterpret_cast<const uint4 *>(from + 8 * p.ld_residual);
        };
        uint4 residual[2];
        load_residual(16 * turn, residual);
        if (!ready()) break;
        const uint32_t at = lanes + (q & 1) * kWide;
        for (int c0 = 16 * turn; c0 < p.bn && c0 < left; c0 += 4 * kEpiWarps) {
          __syncwarp();
          if (whole && left - c0 >= 16) {
            uint32_t f[2][8];
            tmem_load_matrices(at + c0, f[0]);
            tmem_load_matrices(at + c0 + (16u << 16), f[1]);
            uint4 next[2];
            load_residual(c0 + 4 * kEpiWarps, next);
            tmem_wait(f[0], f[1]);
            if constexpr (!D::kSplit)
              finish_block<KIND>(p, tile.q0 + c0, nw, f, unscale, bias, residual, stage);
            residual[0] = next[0];
            residual[1] = next[1];
          } else {
            float v[16];
            tmem_load_16(at + c0, v);
            one_n(c0, v);
          }
        }
        done();
      } else {
        // Several sums, added in registers: tiles of up to kWideSum columns.
        constexpr int kMine = kWideSum / (4 * kEpiWarps);      // blocks of 16 columns of a warp
        float acc[kMine][16];
#pragma unroll
        for (int b = 0; b < kMine; ++b)
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[b][j] = 0.0f;
        for (int i = 0; i < sums && n > 0; ++i) {
          if (!ready()) break;
          const uint32_t at = lanes + (q & 1) * kWide;
#pragma unroll
          for (int b = 0; b < kMine; ++b) {
            const int c0 = 16 * turn + b * 4 * kEpiWarps;
            if (c0 >= p.bn) break;
            __syncwarp();
            if constexpr (D::kSplit) {
              // The two are added to each other first: the lower parts' sum is small, and rounded
              // alone to steps of the whole sum its errors need not be of either sign.  A leading sum
              // that is not finite stands alone: an infinity's lower parts are zeros, whose products
              // with another are NaN.
#pragma unroll
              for (int j0 = 0; j0 < 16; j0 += 8) {
                uint32_t v[8], low[8];
                tmem_load_8(at + c0 + j0, v);
                tmem_load_8(at + kLower + c0 + j0, low);
                tmem_wait(v, low);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const float top = __uint_as_float(v[j]);
                  acc[b][j0 + j] += isfinite(top) ? top + __uint_as_float(low[j]) : top;
                }
              }
            } else {
              float v[16];
              tmem_load_16(at + c0, v);
#pragma unroll
              for (int j = 0; j < 16; ++j) acc[b][j] += v[j];
            }
          }
          done();
        }
        if (timed_out) break;
#pragma unroll
        for (int b = 0; b < kMine; ++b) {
          const int c0 = 16 * turn + b * 4 * kEpiWarps;
          if (c0 < p.bn) one_n(c0, acc[b]);
        }
      }
      if ((t += step) < tiles) tile = tile_at(p, t, 128 * CG);
    }
  }

  if (p.ksplit > 1) {
    // One tile, in parts of the sum: each block adds up a share of its columns, in the parts' order,
    // from the memory of the blocks that have the same lanes.
    __syncwarp();
    cluster_sync();
    const int qn = min(p.bn, p.M - tile.q0);
    const int c0 = qn * part / p.ksplit, c1 = qn * (part + 1) / p.ksplit;
    const int tid = int(threadIdx.x) - 32 * kEpi0, n0 = tile.n0 + 128 * half + (tid & 31) * 4;
    float z[kShare][4];
    if (warp >= kEpi0) {
#pragma unroll
      for (int i = 0; i < kShare; ++i) z[i][0] = z[i][1] = z[i][2] = z[i][3] = 0.0f;
      const uint32_t mine = base + uint32_t((c0 + (tid >> 5)) * 512 + (tid & 31) * 16);
      for (int r = 0; r < p.ksplit; ++r) {
        const uint32_t from = map_rank(mine, uint32_t(CG * r + half));
#pragma unroll
        for (int i = 0; i < kShare; ++i)
          if (c0 + (tid >> 5) + i * kEpiWarps < c1) {
            const float4 v = ld_cluster4(from + i * kEpiWarps * 512);
            z[i][0] += v.x;
            z[i][1] += v.y;
            z[i][2] += v.z;
            z[i][3] += v.w;
          }
      }
    }
    // The others may leave once their parts have been read; what is left needs none of them (and a
    // barrier after the results would wait for them to reach memory, 1500 cycles).
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    if (warp >= kEpi0) {
      float bias[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) bias[k] = bias_at<KIND>(p, n0 + k);
      const float unscale = unscale_of<KIND>(p);
#pragma unroll
      for (int i = 0; i < kShare; ++i) {
        const int c = c0 + (tid >> 5) + i * kEpiWarps;
        if (c >= c1) break;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          z[i][k] = KIND == kF16 ? fmaf(z[i][k], unscale, bias[k]) : z[i][k] + bias[k];
        finish_four<KIND>(p, tile.q0 + c, n0, z[i]);
      }
    }
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
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
  if (CG == 2 && warp == 1 && !leader) {
    // The last arrival from the leader's products, which this block's result warps have all waited for by
    // now: with the loops above it would be a wait of the whole call.
    if (!warp_wait(bar_drain, 0u, p.wait_limit_ns) && lane == 0) atomicOr(&g_linear_status, 2u);
    __syncwarp();
  }
  // Neither block uses tensor memory or the other's barriers.  (Every remote arrival has been waited
  // for, so that the order of execution is enough; a release would wait for the results to reach memory.)
  if (CG == 2) {
    asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    asm volatile("barrier.cluster.wait;" ::: "memory");
  }
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

// One product: out[q, n] = sum_k P[n, k] Q[q, k] for n < N, q < M.
struct DenseOperand {
  Planes planes;
  int mn;                  // stored k x own dimension (else own dimension x k)
};
struct DenseProblem {
  int dtype;
  int64_t M, N, K;
  DenseOperand p, q;
  void *out;
  int64_t ld_out;
  const float *unscale;
  const void *bias;
  int bias_f32, act;
  const void *residual;
  int64_t ld_residual;
  void *pre;
  int64_t ld_pre;
};

// The shape of the least time, by an estimate in ns fitted to measured products (M, N, K from 1 x 1024
// x 1024 to 8192 x 4096 x 4096, all widths and splits; the shapes it takes are within 5 % of the best
// measured one, as a rule):
//   a slice of 64 takes a single block 120 + 0.9 a column (256 columns 350) and a pair 140 + 0.55 a
//   column (256 columns 281, the products' own rate), either 180 at least;
//   in FP32 490 + 5.3 and 430 + 3.7 a column (4096^3: pairs of 128 columns 470 us, blocks 558 us);
//   a tile takes 700 + 6 a column, however few its slices: its results have to leave;
//   memory gives a block 70 bytes at most, all of them 6500, partly beside the above;
//   a launch has 3400 before and after its slices, and sharing a sum costs 1000 + 18 a column (512 x
//   4096 x 4096: pairs of 128 columns 17.2 us, of 256 columns shared by two 20.0 us; 128 x 4096 x
//   4096: 64 columns shared by two 12.3 us, not shared 15.6 us).
// `clusters` gives how many clusters of a size fit.
template <typename Clusters>
DenseShape dense_shape(const DenseProblem &p, Clusters clusters) {
  const int planes = p.dtype == TMM_F32 ? 3 : 1;
  const int64_t slices = (p.K + kBK - 1) / kBK;
  const double bytes = 2.0 * (planes * (double(p.N) * p.K + double(p.M) * p.K) +
                              (planes == 3 ? 2 : 1) * double(p.M) * p.N);
  DenseShape best;
  double least = 0;
  for (int cg = 1; cg <= 2; ++cg) {
    const int64_t unit = (p.q.mn ? 64 : 16) * cg, panels = (p.N + 128 * cg - 1) / (128 * cg);
    for (int64_t bn = unit; bn <= kWidest && bn < p.M + unit; bn += unit) {
      const int64_t tiles = panels * ((p.M + bn - 1) / bn);
      const double wide = double(bn);
      double slice = cg == 2 ? std::max(180.0, 140.0 + 0.55 * wide)
                             : std::max(180.0, 120.0 + 0.9 * wide);
      if (planes == 3) slice = cg == 2 ? 430 + 3.7 * wide : 490 + 5.3 * wide;
      for (int split = 1; cg * split <= 8; split *= 2) {
        const int64_t each = (slices + split - 1) / split, slots = clusters(cg * split);
        if (split > 1 && (slices < 2 * split || tiles > slots)) break;
        if (bn > kWideSum && (planes == 3 || each > kLong || each == 0)) continue;
        const int64_t rounds = (tiles + slots - 1) / slots;
        const double work = double(rounds) * std::max(double(each) * slice, 700 + 6.0 * wide);
        const double blocks = double(std::min(tiles, slots) * cg * split);
        const double memory = bytes / std::min(6500.0, 70.0 * blocks);
        const double ns = std::max(work, memory) + 0.25 * std::min(work, memory) + 4.0 * cg * wide +
                          (split > 1 ? 1000 + 18.0 * wide : 0);
        if (best.cg == 0 || ns < least) {
          best = {cg, int(bn), split};
          least = ns;
        }
      }
    }
  }
  return best;
}

// Opts the kernels in to their shared memory, and finds how many clusters of 1, 2, 4 and 8 blocks the
// device holds at once, a block an SM (the same for all of them): once per device.
std::mutex g_ready_mutex;
bool g_ready[64] = {};
int g_clusters[64][4];

template <typename Kernel>
cudaError_t opt_in(Kernel kernel) {
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMaxSmem));
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                              cudaSharedmemCarveoutMaxShared);
}

cudaError_t make_ready(const DeviceInfo &dev) {
  std::lock_guard<std::mutex> lock(g_ready_mutex);
  if (g_ready[dev.id & 63]) return cudaSuccess;
  cudaError_t e;
  if ((e = opt_in(dense_kernel<1, kBF16>)) != cudaSuccess ||
      (e = opt_in(dense_kernel<1, kF16>)) != cudaSuccess ||
      (e = opt_in(dense_kernel<1, kF32>)) != cudaSuccess ||
      (e = opt_in(dense_kernel<2, kBF16>)) != cudaSuccess ||
      (e = opt_in(dense_kernel<2, kF16>)) != cudaSuccess ||
      (e = opt_in(dense_kernel<2, kF32>)) != cudaSuccess)
    return e;
  for (int i = 0; i < 4; ++i) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << i;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(8, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kMaxSmem;
    int count = 0;
    if (i > 0 && (e = cudaOccupancyMaxActiveClusters(&count, dense_kernel<1, kBF16>, &cfg)) !=
                     cudaSuccess)
      return e;
    g_clusters[dev.id & 63][i] = std::max(1, i > 0 ? count : dev.sm_count);
  }
  g_ready[dev.id & 63] = true;
  return cudaSuccess;
}

template <int CG, int KIND>
cudaError_t launch_as(const DenseProblem &g, const DenseShape &s, const DeviceInfo &dev,
                      cudaStream_t stream) {
  using D = Kind<KIND>;
  DenseParams p = {};
  p.M = int(g.M);
  p.N = int(g.N);
  p.K = int(g.K);
  p.bn = s.bn;
  p.panels = int((g.N + 128 * CG - 1) / (128 * CG));
  p.q_tiles = int((g.M + s.bn - 1) / s.bn);
  p.ksplit = s.split;
  const uint32_t stage = D::stage(s.bn / CG);
  p.stages = int(std::min<uint32_t>(kMaxStages, (kMaxSmem - D::kFixed) / stage));
  // Equal sums, so that the next has time to be made while one is taken out.
  const int most = ((p.K + kBK - 1) / kBK + s.split - 1) / s.split;
  const int sums = (most + kLong - 1) / kLong;
  p.chunk = D::kSplit ? kLongF32 : std::max(1, sums <= 1 ? most : (most + sums - 1) / sums);
  p.p_mn = g.p.mn;
  p.q_mn = g.q.mn;
  // Instruction descriptor of kind::f16: D FP32 (bit 4), A and B bf16 (1 in bits 7-9 and 10-12) or
  // FP16 (0); majors and sizes are added in the kernel.
  p.idesc = (1u << 4) | (KIND == kF16 ? 0u : (1u << 7) | (1u << 10));
  p.out = g.out;
  p.ld_out = g.ld_out;
  p.unscale = g.unscale;
  p.bias = g.bias;
  p.bias_f32 = g.bias_f32 || D::kSplit;
  p.act = g.act;
  p.residual = g.residual;
  p.ld_residual = g.residual ? g.ld_residual : 0;
  p.pre = g.pre;
  p.ld_pre = g.pre ? g.ld_pre : 0;
  constexpr int64_t kPer16 = 16 / sizeof(typename D::T);
  p.vec_out = ((reinterpret_cast<uintptr_t>(p.out) | reinterpret_cast<uintptr_t>(p.residual) |
                reinterpret_cast<uintptr_t>(p.pre)) & 15u) == 0 &&
              p.ld_out % kPer16 == 0 && p.ld_residual % kPer16 == 0 && p.ld_pre % kPer16 == 0;
  p.wait_limit_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  p.drop_block = g_drop_block.load(std::memory_order_relaxed);
  CUtensorMap map_p = {}, map_q = {};
  const auto encode = [&](CUtensorMap *m, const DenseOperand &o, uint32_t rows) {
    const Planes &l = o.planes;
    const uint64_t size[3] = {uint64_t(l.cols), uint64_t(l.rows), uint64_t(l.count)};
    const uint64_t stride[2] = {uint64_t(l.ld), uint64_t(l.stride)};
    const uint32_t box[3] = {kBK, o.mn ? uint32_t(kBK) : rows, 1};
    return encode_16bit(m, l.data, 3, size, stride, box);
  };
  cudaError_t e;
  if (g.K > 0 && ((e = encode(&map_p, g.p, 128)) != cudaSuccess ||
                  (e = encode(&map_q, g.q, uint32_t(s.bn / CG))) != cudaSuccess))
    return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(CG * s.split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = D::kFixed + p.stages * stage;
  cfg.stream = stream;
  const int64_t tiles = int64_t(p.panels) * p.q_tiles, share = CG * s.split;
  const int64_t slots = s.split > 1 ? tiles : dev.sm_count / share;
  cfg.gridDim = dim3(unsigned(share * std::max<int64_t>(1, std::min(tiles, slots))), 1, 1);
  return cudaLaunchKernelEx(&cfg, dense_kernel<CG, KIND>, map_p, map_q, p);
}

cudaError_t launch_dense(const DenseProblem &p, const DeviceInfo &dev, cudaStream_t stream) {
  cudaError_t e = make_ready(dev);
  if (e != cudaSuccess) return e;
  if ((p.N + 127) / 128 * ((p.M + 15) / 16) >= INT32_MAX / 16) return cudaErrorInvalidConfiguration;
  const int *const fit = g_clusters[dev.id & 63];
  const DenseShape s = dense_shape(
      p, [&](int size) { return fit[size == 1 ? 0 : size == 2 ? 1 : size == 4 ? 2 : 3]; });
  if (p.dtype == TMM_BF16)
    return s.cg == 2 ? launch_as<2, kBF16>(p, s, dev, stream)
                     : launch_as<1, kBF16>(p, s, dev, stream);
  if (p.dtype == TMM_F16)
    return s.cg == 2 ? launch_as<2, kF16>(p, s, dev, stream) : launch_as<1, kF16>(p, s, dev, stream);
  return s.cg == 2 ? launch_as<2, kF32>(p, s, dev, stream) : launch_as<1, kF32>(p, s, dev, stream);
}

// dz in the workspace: of the type, on 16-byte rows, or (FP32) as planes.  FP32 of few rows: dx from
// FP32 values, whose planes dw takes.  FP16: times a power of two, unless it is dy or 0 (relu).
struct GradPlan {
  bool make_dz, few, dz_planes, scaled;
  int64_t ldz;
  size_t dz_bytes, unscale_bytes, partial_bytes, bytes;
};
// dz as a matrix of the type: what has been made at `made`, or dy itself.
Stack dz_stack(const LinearGradProblem &p, const GradPlan &g, const void *made) {
  return g.make_dz ? Stack{made, 1, p.rows, p.N, g.ldz, 0} : p.dy;
}
GradPlan plan_grad(const LinearGradProblem &p) {
  GradPlan g = {};
  g.make_dz = p.act != TMM_ACT_NONE && (p.dx || p.dw);
  g.ldz = (p.N + 7) / 8 * 8;
  g.few = linear_is_few(p.dtype, p.rows);
  g.dz_planes = p.dtype == TMM_F32 && !g.few;
  if (g.make_dz) {
    const __int128 n = __int128(p.rows) * g.ldz * (g.dz_planes ? 6 : p.dtype == TMM_F32 ? 4 : 2);
    g.dz_bytes = n > __int128(INT64_MAX / 4) ? SIZE_MAX : round256(size_t(n));
  }
  g.scaled = g.make_dz && p.dtype == TMM_F16 && p.act != TMM_ACT_RELU;
  g.unscale_bytes = g.scaled ? round256(linear_unscale_bytes()) : 0;
  g.partial_bytes = p.dbias ? round256(linear_bias_bytes(p.rows, p.N, p.dtype)) : 0;
  const bool planes = p.dw || (p.dx && !g.few);
  g.bytes = add_sizes({g.dz_bytes, g.unscale_bytes, g.partial_bytes,
                       planes && !(g.make_dz && !g.few)
                           ? planes_bytes(dz_stack(p, g, nullptr), p.dtype)
                           : 0,
                       p.dx && !g.few ? planes_bytes(p.w, p.dtype) : 0,
                       p.dw ? planes_bytes(p.x, p.dtype) : 0});
  return g;
}

}  // namespace

// FP32 of up to 16 rows: making planes of the weights takes longer than the sums (4096 x 4096, gelu and
// residual, 16 rows: 30 us and 44).
bool linear_is_few(int dtype, int64_t rows) { return dtype == TMM_F32 && rows <= 16; }

size_t linear_workspace_bytes(const LinearProblem &p) {
  if (p.K == 0 || linear_is_few(p.dtype, p.rows)) return 0;
  return add_sizes({planes_bytes(p.x, p.dtype), planes_bytes(p.w, p.dtype)});
}

cudaError_t launch_linear(const LinearProblem &p, const DeviceInfo &dev, void *workspace,
                          cudaStream_t stream) {
  if (linear_is_few(p.dtype, p.rows) && p.K > 0) return launch_linear_few(p, dev, stream);
  char *ws = static_cast<char *>(workspace);
  DenseProblem d = {p.dtype, p.rows, p.N, p.K};
  if (p.K > 0) {
    const Stack *const from[2] = {&p.x, &p.w};
    Planes to[2];
    const cudaError_t e = make_operand_planes(from, to, 2, p.dtype, &ws, dev, stream);
    if (e != cudaSuccess) return e;
    d.p = {to[1], !p.trans_w};
    d.q = {to[0], 0};
  }
  d.out = p.y;
  d.ld_out = p.ldy;
  d.bias = p.bias;
  d.bias_f32 = p.bias_f32;
  d.act = p.act;
  d.residual = p.residual;
  d.ld_residual = p.ld_residual;
  d.pre = p.pre;
  d.ld_pre = p.ld_pre;
  return launch_dense(d, dev, stream);
}

size_t linear_grad_workspace_bytes(const LinearGradProblem &p) { return plan_grad(p).bytes; }

cudaError_t launch_linear_grad(const LinearGradProblem &p, const DeviceInfo &dev, void *workspace,
                               cudaStream_t stream) {
  const GradPlan g = plan_grad(p);
  char *ws = static_cast<char *>(workspace);
  cudaError_t e;
  Planes dz = {}, w = {}, x = {};
  void *const made = ws;
  if (g.make_dz) {
    dz = {made, g.dz_planes ? 3 : 1, p.rows, p.N, g.ldz, p.rows * g.ldz};
    ws += g.dz_bytes;
  }
  float *const unscale = g.scaled ? reinterpret_cast<float *>(ws) : nullptr;
  ws += g.unscale_bytes;
  if (g.make_dz || p.dbias) {
    e = launch_linear_slopes(p, g.make_dz ? made : nullptr, g.ldz, g.dz_planes, unscale,
                             reinterpret_cast<float *>(ws), stream);
    if (e != cudaSuccess) return e;
  }
  ws += g.partial_bytes;
  const Stack matrix = dz_stack(p, g, made);
  const Stack *from[3];
  Planes to[3], *at[3];
  int count = 0;
  const auto need = [&](const Stack &s, Planes *planes) {
    from[count] = &s;
    at[count++] = planes;
  };
  if ((p.dw || (p.dx && !g.few)) && !(g.make_dz && !g.few)) need(matrix, &dz);
  if (p.dx && !g.few) need(p.w, &w);
  if (p.dw) need(p.x, &x);
  if ((e = make_operand_planes(from, to, count, p.dtype, &ws, dev, stream)) != cudaSuccess) return e;
  for (int i = 0; i < count; ++i) *at[i] = to[i];
  if (p.dx && g.few) {
    LinearProblem f = {};
    f.dtype = p.dtype;
    f.rows = p.rows;
    f.N = p.K;
    f.K = p.N;
    f.x = matrix;
    f.w = p.w;
    f.trans_w = !p.trans_w;
    f.y = p.dx;
    f.ldy = p.lddx;
    if ((e = launch_linear_few(f, dev, stream)) != cudaSuccess) return e;
  }
  DenseProblem d = {};
  d.dtype = p.dtype;
  d.unscale = unscale;
  if (p.dx && !g.few) {
    d.M = p.rows;
    d.N = p.K;
    d.K = p.N;
    d.p = {w, p.trans_w};
    d.q = {dz, 0};
    d.out = p.dx;
    d.ld_out = p.lddx;
    if ((e = launch_dense(d, dev, stream)) != cudaSuccess) return e;
  }
  if (p.dw) {
    d.M = p.trans_dw ? p.N : p.K;
    d.N = p.trans_dw ? p.K : p.N;
    d.K = p.rows;
    d.p = {p.trans_dw ? x : dz, 1};
    d.q = {p.trans_dw ? dz : x, 1};
    d.out = p.dw;
    d.ld_out = p.lddw;
    if ((e = launch_dense(d, dev, stream)) != cudaSuccess) return e;
  }
  return cudaSuccess;
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
