// gemm_grouped.cu -- products whose right-hand matrix is chosen row by row, on the tcgen05
// tensor cores: the grouped product, its weight gradient, and adapters beside a shared product.
//
//   forward   y[p, n]  = sum_k x[r(p), k] w[g, k, n]           rows p of group g
//   gradient  dw[g, k, n] = sum_{p in g} x[r(p), k] dy[p, n]
//   adapters  y[r(p), n] = sum_k x[r(p), k] w[k, n] + sum_j u[p, j] b[g, j, n],
//             u[p, j] = scale[g] sum_k x[r(p), k] a[g, k, j]   (a forward product of its own)
//
// One kernel serves all three.  It computes tiles of D[n, q] = sum_k P[n, k] Q[q, k], with the
// dimension that is contiguous in the result (n) on the 128 tensor-memory lanes of a block and
// the result's rows (q) on its columns.  The columns of a tile are the ragged side: a
// tcgen05.mma takes any multiple of 16 of them, so a group of few rows costs few columns, not a
// whole tile, and the weights -- the larger operand when rows are few -- fill the lanes.
//   forward:  P = w[g] (stored K x N or N x K: both majors are read in place),  Q = rows of x
//   gradient: P = dy^T,  Q = x^T, the sum running over the group's rows
//   adapters: the forward product with one P = w for all.  On pairs an adapter's columns start
//             at a multiple of 32 of the tile's, and its part, P = b[g] and Q = u, is added to
//             those columns alone; on single blocks, whose rows are few, it is added on the CUDA
//             cores while w streams.  (On pairs u is read as parts: see store_u4.)
// No operand value of another group, not even a NaN, meets a group's sums: columns are summed
// apart, those past a group's end are not stored, and the gradient, whose sum runs over the rows,
// reads zeros in their place.  A row number outside the matrix reads as zeros.
//
// Single precision: every operand x is split into three bf16 parts, x = x0 + x1 + x2 exactly
// (split3): for pairs by a pre-pass (planes), on single blocks by the copy warps (split_tile).
// Of the nine part products the three smallest (2^-24 of the term and less) are dropped.  x0 y0
// goes to one accumulator, the five smaller ones (2^-8 of it and less) to another; the tensor core's
// additions do not round to nearest, and the error of a sum grows with the number of additions made
// in tensor memory (16 values of K each), so both are taken out every kChunk slices and added in
// FP32 registers.
// For 16-bit operands a sum stays in tensor memory for kLong slices, 512 additions whose errors
// (2^-24 of the partial sum on the mean, of one sign where the terms are) come to 2^-15, a
// sixteenth of FP16's rounding; longer sums are made of several, added in FP32.
//
// Two shapes:
//   pairs  (CG = 2): two blocks on two SMs share 256 lanes x up to 256 columns
//          (cta_group::2): each stages half of the columns, which halves their
//          shared-memory traffic.  For many rows per group.
//   single (CG = 1): 128 lanes x up to 64 columns, and for few tiles a cluster of up to eight
//          blocks that share the sum over K: each leaves its part in its shared memory, and the
//          blocks add the parts in block order through distributed shared memory (no global
//          scratch, no atomics: results are deterministic).  For few rows per group, where
//          reading w is the bound and more blocks read it faster.
// Both are persistent: the tile list is made in every block from the group offsets, which only
// the GPU knows.  Roles: four warps copy (16 where they split FP32 values), eight take results out,
// one issues the products.  Every wait is bounded (globaltimer); on timeout bit 1 of the status word
// is set and the kernel runs to its end.
//
// Measured (a call's kernels, three sets of inputs by turns; rates of the measured 6780 GB/s and 1936
// TFLOP/s; "product": that kernel alone, nothing in the caches):
//   16384 rows in 8 groups, 4096 x 4096, bf16: 381 us, 1.44 PFLOP/s (75 %); the product 312, a gather
//     of the rows before it 44.  Bound by the tensor cores (active 82 % of the product's cycles).
//   its gradient with 8192 rows: 210 us, 1.31 PFLOP/s (68 %), product 182: the tensor cores (67 %), and
//     268 MB of results, which no products cover where a group has few rows.
//   two rows of two groups, 4096 x 4096: 15.8 us, 63 % of the 9.9 us that 67 MB take: the first
//     bytes come 4 us after the start, and the blocks meet to add their parts.
//   one row with its adapter, 4096 x 4096: 12.0 us against 5.0 for 34 MB: as above.
//   4096 rows with 6 adapters of rank 64, 4096 x 4096, fp16: 128 us; the product 100 (tensor cores 65
//     %): four rounds of tiles on 76 pairs where 3.6 would do.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "grouped.h"
#include "tmm_gemm.h"

namespace tmm {

__device__ unsigned int g_grouped_status;

namespace {

constexpr int kForward = 0, kWgrad = 1, kLora = 2;
constexpr int kBK = 64;                  // 16-bit values per K slice: one 128-byte swizzle row
constexpr int kEpiWarps = 8;
constexpr int kListed = kMaxGroups + 3;            // entries of a list of groups, see Table
constexpr int kFewRows = 512;                      // rows of an adapters' call on single blocks
constexpr int kChunk = 2;                // slices per tensor-memory sum of split operands
// Slices per tensor-memory sum of 16-bit operands at most, 8192 values.  (A gradient over 524365 rows
// of positive values was 0.7 % too small in one sum.  Taking sums out costs up to 8 %, see below.)
constexpr int kLong = 128;
// Slices of each of the tensor-memory sums of `n` slices, but for the last: equal ones, so that the
// next has time to run while one is taken out.
__device__ __forceinline__ int long_sum(int n) {
  const int sums = (n + kLong - 1) / kLong;
  return sums <= 1 ? n : (n + sums - 1) / sums;
}
constexpr uint32_t kPTile = 128 * 128;   // 128 lanes x 64 values: 16 KiB
constexpr uint32_t kMaxSmem = 232448;    // 227 KiB

// How the results are written.
constexpr int kOutF32 = 0, kOutBF16 = 1, kOutF16 = 2;
constexpr int kOutU = 3;       // the adapters' u: its parts, in three planes or side by side


// Values of `rank` per slice of the adapters' part: as many as the parts of u leave of the 64 columns
// of a slice (store_u4), or FP32's planes.
__host__ __device__ constexpr int rank_slice(int planes, int b_parts) {
  return planes == 3 ? 64 : b_parts == 2 ? 16 : 32;
}

template <int CG, int PLANES>
struct Shape {
  // FP32 on single blocks: the copy warps read the operands as they are stored and split them
  // on the way (DIRECT); no planes.
  static constexpr bool kDirect = CG == 1 && PLANES == 3;
  static constexpr int kCopyWarps = kDirect ? 16 : 4;
  static constexpr int kEpi0 = kCopyWarps;           // first of the result warps
  static constexpr int kMmaWarp = kCopyWarps + kEpiWarps;
  static constexpr int kThreads = 32 * (kMmaWarp + 1);
  static constexpr int kBN = PLANES == 3 ? (CG == 2 ? 128 : 64) : (CG == 2 ? 256 : 64);
  static constexpr int kUnit = CG == 2 ? 32 : 16;    // columns are rounded up to this
  static constexpr int kBox = CG == 2 ? 32 : 16;     // rows of one copy of Q (the last one may
                                                     // bring more rows than the tile needs)
  static constexpr uint32_t kQTile = uint32_t(kBN / CG) * 128;
  static constexpr uint32_t kStage = PLANES * (kPTile + kQTile);
  static constexpr int kStages = PLANES == 3 ? (CG == 2 ? 3 : 2) : (CG == 2 ? 6 : 7);
  static constexpr uint32_t kTmemCols =
      PLANES == 3 ? 4 * kBN : 2 * kBN;               // two accumulators (of each kind)
  // The parts of a shared sum (single blocks), and 1 KiB a result warp for 16-bit results.
  static constexpr uint32_t kRed = CG == 1 ? 128 * kBN * 4 : 0;
  static constexpr uint32_t kOutStage = PLANES == 1 ? kEpiWarps * 1024 : 0;
  static constexpr uint32_t kTable =
      kListed * 4 * 3 + kCopyWarps * 128 + 116 + (CG == 1 ? kFewRows * 4 : 0);
  static constexpr uint32_t kBars = 8 * (2 * kStages + 5) + 32;
  static constexpr uint32_t kSmem = 1024 + kStages * kStage + kRed + kOutStage + kTable + kBars;
  static_assert(kSmem <= kMaxSmem, "one block's shared memory");
  static_assert(kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "tensor memory columns");
};

struct Params {
  int rows;              // p runs over [0, rows)
  int groups;
  const int *offsets;    // groups + 1
  const int *row_index;  // r(p) of the rows read (single blocks; pairs read gathered rows), or NULL
  const int *out_index;  // r(p) of the rows written (adapters), or NULL
  int q_rows;            // rows of the x that is read
  int out_rows;          // rows of y, by out_index
  int K;                 // forward, adapters: length of the sum
  int N;                 // extent of the lanes' dimension
  int q_cols;            // gradient: columns of x
  int rank;              // adapters
  int panels;            // tiles along N
  int tile_n;            // columns of a tile, at most kBN
  int p_mn, e_mn;        // P (and b) stored with n contiguous
  int p_shared, e_shared;   // one P (one b) for all groups
  uint32_t idesc;        // types; majors and sizes are added in the kernel
  uint32_t idesc_e;      // types of the adapters' part
  // FP32 operands as they are stored (single blocks): P and x.
  const float *fp, *fx;
  int64_t ldp, stride_p, ldx;
  int vec;               // whole 16-byte loads of both
  void *out;
  int64_t ld_out, stride_out;   // stride: of dw's matrices, or of the result's planes
  int out_type;
  int n_out;             // columns written (from N on: zeros)
  int vec_out;           // 16-bit results with rows (and matrices) on 16-byte boundaries
  const float *scale;    // per group, or NULL
  // Adapters on single blocks: u in FP32 by row of x, and b as it is stored.
  const float *u;
  const void *b;
  int64_t ldu, ldb, stride_b;
  int trans_b, vec_b;
  int zero_rows;         // forward: write zeros to the rows of no group
  int ksplit;            // blocks of a cluster that share a tile's sum (CG = 1)
  int64_t wait_limit_ns;
  int drop_block;        // testing hook: this block waits for bytes that never come (-1: none)
};

// A place in the ring of stages, and the parity of its round.
struct Ring {
  int stage;
  uint32_t parity;
  template <int STAGES>
  __device__ __forceinline__ void next() {
    if (++stage == STAGES) {
      stage = 0;
      parity ^= 1;
    }
  }
};

// ---- primitives -------------------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint64_t timer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
// On this block's own barrier (`bar`: its shared memory address).
__device__ __forceinline__ void mbar_arrive_local(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Of any block of the cluster, where no access to memory of this thread has to be ordered before
// it.  (A cluster-wide release takes about 1500 cycles and waits for the thread's stores: result
// warps handing tensor memory back, whose reads have completed, would wait for their results to
// reach memory.)
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, int64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (int64_t(timer_ns() - t0) > limit_ns) return false;
  return true;
}
// True in one thread of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// Every thread of every block of the cluster.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Tensor copies into this block's shared memory; `bar` counts their bytes (a shared::cluster
// address, in pairs the leader's).
template <int CG>
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                       uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
template <int CG>
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                       uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// Four rows y[0..3] of 64 values from column x.
template <int CG>
__device__ __forceinline__ void tma_rows4(uint32_t dst, const CUtensorMap *map, int x,
                                          const int (&y)[4], uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4"
        ".mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]),
        "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4"
        ".mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]),
        "r"(bar)
        : "memory");
}
// Orders ordinary accesses to shared memory before the copy engine's and the tensor core's.
__device__ __forceinline__ void proxy_fence() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// Programmatic dependent launch: wait for the grid before (its results, and those of the grids
// before it, are visible then), and let the next one start as soon as there is room.  Every grid
// starts the next one only after its own wait, so whatever is before the grid before is done
// when a grid starts.
__device__ __forceinline__ void grid_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void grid_start_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    bool accumulate) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %3, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %4, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(uint32_t(accumulate)), "r"(idesc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %3, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %4, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(uint32_t(accumulate)), "r"(idesc)
        : "memory");
}
// Arrive on `bar` (of both blocks of a pair, with `both`) once the products issued so far by
// this thread have completed.
template <int CG>
__device__ __forceinline__ void mma_commit(uint32_t bar, bool both) {
  if constexpr (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(bar),
        "h"(uint16_t(both ? 3 : 1))
        : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}
// Waits for this thread's tensor-memory loads.  The registers that they fill are operands, so that no
// use of them, which depends on nothing else, is moved before the wait.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[8], uint32_t (&s)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(s[0]), "+r"(s[1]), "+r"(s[2]), "+r"(s[3]),
                 "+r"(s[4]), "+r"(s[5]), "+r"(s[6]), "+r"(s[7])
               :
               : "memory");
}
// 8 consecutive FP32 columns of this thread's lane, there after tmem_wait.
__device__ __forceinline__ void tmem_load_8(uint32_t addr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(addr)
      : "memory");
}
// 16 of them, waited for.
__device__ __forceinline__ void tmem_load_16(uint32_t addr, float (&v)[16]) {
  uint32_t r[2][8];
  tmem_load_8(addr, r[0]);
  tmem_load_8(addr + 8, r[1]);
  tmem_wait(r[0], r[1]);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i >> 3][i & 7]);
}

// 16 lanes x 16 consecutive FP32 columns, in the order of an 8 x 8 matrix instruction: r[4 c + 2 h]
// and the one after it are columns 8 c + 2 (l % 4) and + 1 of lane 8 h + l / 4 (l: this thread).
// The values are there after tmem_wait.
__device__ __forceinline__ void tmem_load_matrices(uint32_t addr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(addr)
      : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle: start address >> 4 (bits 0-13), leading
// byte offset >> 4 (16-29), stride byte offset >> 4 (32-45), version 1 (46-47), swizzle 2
// (61-63).  A tile stored with K contiguous has rows of 64 values (128 bytes), eight of them
// 1024 bytes apart (stride); 16 values of K are 32 bytes on.  A tile stored with n contiguous
// is made of blocks of 64 n (128 bytes) x 64 k, 8 KiB apart (leading), eight k 1024 bytes
// apart (stride); 16 values of K are 2048 bytes on.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, bool mn) {
  return uint64_t((addr >> 4) & 0x3FFFu) | (uint64_t(mn ? 512 : 1) << 16) | (uint64_t(64) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// ---- tiles ------------------------------------------------------------------------------

// What a tile covers.  Forward, adapters: columns are rows p in [q0, q0 + qn); gradient: they
// are columns of x, and the sum runs over the rows [k0, k0 + klen).  Adapters on pairs: columns
// count places in which every entry of the list starts at a multiple of 32.
struct Tile {
  int g;          // group (adapters on pairs: the entry of the first column)
  int n0;         // first n
  int q0, qn;     // columns of the tile
  int bn;         // qn rounded up for the tensor core
  int k0, klen;
  int e0, en;     // adapters on pairs: entries [e0, e0 + en) are those of adapters
};

// The tables in shared memory: the groups that have rows: number, first row (one more entry: the
// end of the last), first tile.  Adapters on pairs: the rows of no adapter, before and after the
// others, are entries too, of number -1, and `tile` counts 32 columns (one more entry: the end).
// In the gradient: every group's first row, by its number, and the numbers in the order of the
// tiles.
struct Table {
  const int *gid, *row, *tile;
  int count, tiles;
};

// An entry's part of a tile: columns from c0 on, 32 n32 of them, and the row of the first.
struct Part {
  int c0, n32, row;
};
__device__ __forceinline__ Part part_of(const Params &p, const Table &tab, const Tile &t, int e) {
  const int u0 = t.q0 >> 5, u1 = u0 + (p.tile_n >> 5);
  const int a = max(tab.tile[e], u0), b = min(tab.tile[e + 1], u1);
  return {(a - u0) * 32, b - a, tab.row[e] + (a - tab.tile[e]) * 32};
}

template <int CG, int MODE, int PLANES>
__device__ __forceinline__ Tile tile_at(const Params &p, const Table &tab, int t) {
  using S = Shape<CG, PLANES>;
  Tile r;
  r.e0 = r.en = r.k0 = 0;
  if (MODE == kWgrad) {
    const int qt = (p.q_cols + p.tile_n - 1) / p.tile_n;
    const int per = qt * p.panels;
    r.g = t / per;
    const int i = t - r.g * per;
    r.g = tab.gid[r.g];
    const int panel = i / qt;
    r.n0 = panel * 128 * CG;
    r.q0 = (i - panel * qt) * p.tile_n;
    r.qn = min(p.tile_n, p.q_cols - r.q0);
    r.bn = (r.qn + 64 * CG - 1) / (64 * CG) * (64 * CG);
    r.k0 = tab.row[r.g];
    r.klen = tab.row[r.g + 1] - r.k0;
    return r;
  }
  int lo, hi, i;
  if (MODE == kLora) {
    r.g = 0;
    lo = 0;
    hi = CG == 2 ? tab.tile[tab.count] * 32 : p.rows;
    i = t;
  } else {
    int a = 0, b = tab.count;      // the last entry whose first tile is <= t
    while (b - a > 1) {
      const int m = (a + b) >> 1;
      if (tab.tile[m] <= t) a = m;
      else b = m;
    }
    r.g = tab.gid[a];
    lo = tab.row[a];
    hi = tab.row[a + 1];
    i = t - tab.tile[a];
  }
  const int qt = (hi - lo + p.tile_n - 1) / p.tile_n;
  const int panel = i / qt;
  r.n0 = panel * 128 * CG;
  r.q0 = lo + (i - panel * qt) * p.tile_n;
  r.qn = min(p.tile_n, hi - r.q0);
  r.bn = (r.qn + S::kUnit - 1) / S::kUnit * S::kUnit;
  r.klen = p.K;
  if (MODE == kLora && CG == 2) {
    // Halves of the tile are whole 32 columns.  The entries in it: the last that starts at or
    // before its first column, to the last that starts before its end.
    r.bn = (r.qn + 63) / 64 * 64;
    const auto last = [&](int unit) {
      int a = 0, b = tab.count;
      while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (tab.tile[m] <= unit) a = m;
        else b = m;
      }
      return a;
    };
    r.g = last(r.q0 >> 5);
    const int end = last((r.q0 + r.qn - 1) >> 5);
    r.e0 = r.g + (tab.gid[r.g] < 0);
    r.en = max(0, end + (tab.gid[end] >= 0) - r.e0);
  }
  return r;
}

// This block's K slices [s0, s1) of a tile: the slices of the base sum, then those of the
// adapters in the tile; blocks that share a tile take equal runs of them.
template <bool EXT, int RS>
__device__ __forceinline__ void slices_of(const Params &p, const Tile &t, int rank, int &base,
                                          int &s0, int &s1) {
  base = (t.klen + kBK - 1) / kBK;
  int n = base;
  if (EXT) n += t.en * ((p.rank + RS - 1) / RS);
  if (p.ksplit == 1) {
    s0 = 0;
    s1 = n;
  } else {
    s0 = int(int64_t(n) * rank / p.ksplit);
    s1 = int(int64_t(n) * (rank + 1) / p.ksplit);
  }
}

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

// The adapters' u beside 16-bit operands: BF16 parts of the FP32 value (split3) side by side in a
// row, in blocks of 64 columns.  BF16 operands: two parts of 32 values, 17 bits of u, far below the
// result's rounding (all three parts took 2 to 13 % longer).  FP16 operands: all three parts of 16
// values, u's 24 bits and FP32's range (a pair of FP16 values is infinite above 65504 and has fewer
// than 17 bits below 2^-8; the number of rows, which decides how u is made, would decide that).  The
// fourth part is the first with zero in place of an infinity, for the products with b's second
// part, which is zero as a rule.  Measured, 4096 x 4096, rank 64, FP16 and BF16: 4096 rows of 6
// adapters 130 us and 122 us, of 64 adapters 178 us and 154 us.
//
// Parts of columns n to n + 3 (n % 4 = 0) of a row from one thread.
__device__ __forceinline__ uint2 pack4(const uint16_t (&h)[4][4], int i) {
  return make_uint2(h[0][i] | (uint32_t(h[1][i]) << 16), h[2][i] | (uint32_t(h[3][i]) << 16));
}
__device__ __forceinline__ void store_u4(uint16_t *row, int n, const float (&v)[4], bool bf16) {
  uint16_t h[4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint16_t s[3];
    split3(v[j], s);
    h[j][0] = s[0];
    h[j][1] = s[1];
    h[j][2] = s[2];
    h[j][3] = (s[0] & 0x7FFFu) == 0x7F80u ? uint16_t(0) : s[0];
  }
  if (bf16) {
    uint16_t *const o = row + (n >> 5) * 64 + (n & 31);
#pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<uint2 *>(o + 32 * i) = pack4(h, i);
  } else {
    uint16_t *const o = row + (n >> 4) * 64 + (n & 15);
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint2 *>(o + 16 * i) = pack4(h, i);
  }
}
// Four rows' column n from every lane (n: its lane in the warp, on from a multiple of 32), `in` the
// same in four lanes: they exchange values, so that each stores four columns of one row.  (Stores of
// two bytes took the whole kernel 3 us longer.)
__device__ __forceinline__ void store_u(uint16_t *row, int64_t ld, int n, const float (&v)[4],
                                        bool in, int count, bool bf16) {
  const int q = n & 3;
  float f[4];      // columns n - q + 0..3 of row q
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // In turn i, lane q has its value of row q ^ i taken by lane q ^ i.
    const float mine = q == 0 ? v[i] : q == 1 ? v[i ^ 1] : q == 2 ? v[i ^ 2] : v[i ^ 3];
    const float got = __shfl_xor_sync(~0u, mine, i);
    // Column q ^ i of row q.
    if (q == 0) f[i] = got;
    else if (q == 1) f[i ^ 1] = got;
    else if (q == 2) f[i ^ 2] = got;
    else f[i ^ 3] = got;
  }
  if (in && q < count) store_u4(row + q * ld, n - q, f, bf16);
}

// Two FP16 values (low and high half) as two BF16 parts each, exactly: 8 of the 11 bits and what they
// leave (none of an infinity or a NaN).
__device__ __forceinline__ void half_parts(uint32_t two, uint32_t (&h)[2]) {
  const float a = __half2float(__ushort_as_half(uint16_t(two)));
  const float b = __half2float(__ushort_as_half(uint16_t(two >> 16)));
  h[0] = pair_bf16(a, b);
  const float ra = a - __uint_as_float(h[0] << 16), rb = b - __uint_as_float(h[0] & 0xFFFF0000u);
  h[1] = pair_bf16(ra == ra ? ra : 0.0f, rb == rb ? rb : 0.0f);
}

// One result at column n of the row at element offset `o` of the output.  Split operands
// (PLANES = 3) give FP32, or u's planes; 16-bit operands their own type (u: store_u).
template <int MODE, int PLANES>
__device__ __forceinline__ void store_out(const Params &p, int64_t o, int n, float v) {
  if constexpr (PLANES == 3) {
    if (MODE != kForward || p.out_type == kOutF32) {
      static_cast<float *>(p.out)[o + n] = v;
    } else {
      uint16_t h[3];
      split3(v, h);
#pragma unroll
      for (int i = 0; i < 3; ++i) static_cast<uint16_t *>(p.out)[o + n + i * p.stride_out] = h[i];
    }
  } else if (p.out_type == kOutBF16) {
    static_cast<__nv_bfloat16 *>(p.out)[o + n] = __float2bfloat16_rn(v);
  } else {
    static_cast<__half *>(p.out)[o + n] = __float2half_rn(v);
  }
}

// Offset of the result row that column `col` of the tile goes to; -1: none.
template <int MODE>
__device__ __forceinline__ int64_t out_row(const Params &p, const Tile &t, int col) {
  if (MODE == kWgrad) return int64_t(t.g) * p.stride_out + int64_t(t.q0 + col) * p.ld_out;
  int r = t.q0 + col;
  if (MODE == kLora && p.out_index) {
    r = p.out_index[r];
    if (r < 0 || r >= p.out_rows) return -1;
  }
  return int64_t(r) * p.ld_out;
}

// 16-bit results with rows on 16-byte boundaries go through 1 KiB of shared memory a warp, 16 result
// rows of 32 n, from which four lanes take the 64 bytes of a row: 2 stores of 16 bytes a lane in
// place of 16 of two bytes.  Piece `c` of 8 n of row `row` is at:
__device__ __forceinline__ uint32_t staged(uint32_t stage, int row, int c) {
  return stage + uint32_t(row * 64 + ((c ^ (row >> 1 & 3)) << 4));      // free of bank conflicts
}
template <int MODE>
__device__ __forceinline__ void store_staged(const Params &p, const Tile &t, int c0, int nw,
                                             uint32_t stage, const int *owner) {
  const int lane = threadIdx.x & 31;
  const int count = min(16, t.qn - c0);
  const bool by_row = MODE == kLora && p.out_index;
  const bool check = MODE == kLora && p.u;      // rows that are not written (see owner)
  const int64_t first = by_row ? 0 : out_row<MODE>(p, t, c0);
  const int n8 = nw + (lane & 3) * 8;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = (lane >> 2) + 8 * i;
    uint4 w;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "r"(staged(stage, row, lane & 3))
                 : "memory");
    if (row >= count || n8 >= p.N) continue;
    const int64_t o = by_row ? out_row<MODE>(p, t, c0 + row) : first + row * p.ld_out;
    if (o < 0 || (check && owner[t.q0 + c0 + row] == -2)) continue;
    uint16_t *dst = static_cast<uint16_t *>(p.out) + o + n8;
    if (n8 + 8 <= p.N) {
      *reinterpret_cast<uint4 *>(dst) = w;
    } else {
      const uint32_t part[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (n8 + j < p.N) dst[j] = uint16_t(part[j / 2] >> (16 * (j & 1)));
    }
  }
}
// 16 columns of the tile from c0 on, for the 32 n of the warp, as tmem_load_matrices leaves lanes
// 16 i to 16 i + 15 in f[i]: the matrices are transposed on their way to shared memory, two
// instructions in place of the 16 of store_columns (gradient of 32 groups of 64 rows, 4096 x 4096:
// 349 us -> 322 us; with two blocks' values loaded at a time 363 us).
template <int MODE>
__device__ __forceinline__ void store_matrices(const Params &p, const Tile &t, int c0, int nw,
                                               const uint32_t (&f)[2][8], float scale,
                                               uint32_t stage, const int *owner) {
  const int lane = threadIdx.x & 31;
  uint32_t h[2][4];      // [8 columns][8 n]: two neighbouring columns of one n
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float lo = __uint_as_float(f[m >> 1][4 * c + 2 * (m & 1)]) * scale;
      const float hi = __uint_as_float(f[m >> 1][4 * c + 2 * (m & 1) + 1]) * scale;
      if (p.out_type == kOutBF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[c][m]) : "f"(hi), "f"(lo));
      else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[c][m]) : "f"(hi), "f"(lo));
    }
  __syncwarp();      // the reads of the block before are done
#pragma unroll
  for (int c = 0; c < 2; ++c)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                     staged(stage, 8 * c + (lane & 7), lane >> 3)),
                 "r"(h[c][0]), "r"(h[c][1]), "r"(h[c][2]), "r"(h[c][3])
                 : "memory");
  __syncwarp();
  store_staged<MODE>(p, t, c0, nw, stage, owner);
}

// 16 consecutive columns of the tile from c0 on, for the 32 n of the warp from nw on (lane l
// holds nw + l).
template <int MODE, int PLANES>
__device__ __forceinline__ void store_columns(const Params &p, const Tile &t, int c0, int nw,
                                              const float (&v)[16], float scale, uint32_t stage,
                                              const int *owner) {
  const int lane = threadIdx.x & 31;
  const int count = min(16, t.qn - c0);
  const int n = nw + lane;
  const bool by_row = MODE == kLora && p.out_index;
  const bool check = MODE == kLora && p.u;      // rows that are not written (see owner)
  int64_t first = 0;
  if (!by_row) first = out_row<MODE>(p, t, c0);
  if constexpr (PLANES == 1) {
    if (p.vec_out) {
      uint16_t h[16];
      if (p.out_type == kOutBF16) {
#pragma unroll
        for (int j = 0; j < 16; ++j) h[j] = __bfloat16_as_ushort(__float2bfloat16_rn(v[j] * scale));
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) h[j] = __half_as_ushort(__float2half_rn(v[j] * scale));
      }
      __syncwarp();      // the reads of the block before are done
#pragma unroll
      for (int j = 0; j < 16; ++j)
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(staged(stage, j, lane >> 3) + (lane & 7) * 2),
                     "h"(h[j])
                     : "memory");
      __syncwarp();
      store_staged<MODE>(p, t, c0, nw, stage, owner);
      return;
    }
  } else if (!by_row && p.out_type == kOutF32) {
    // 32 lanes write 128 consecutive bytes.
    float *dst = static_cast<float *>(p.out) + first + n;
    const bool in = n < p.N;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (in && j < count && !(check && owner[t.q0 + c0 + j] == -2))
        dst[j * p.ld_out] = v[j] * scale;
    return;
  }
  int row = 0;      // the row of column c0 + lane % 16
  if (by_row) {
    const int l = lane & 15;
    row = l < count ? p.out_index[t.q0 + c0 + l] : -1;
    if (row >= p.out_rows) row = -1;
  }
  const bool in = n < p.n_out;
  if constexpr (MODE == kForward && PLANES == 1) {
    if (p.out_type == kOutU) {
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = n < p.N ? v[j + i] * scale : 0.0f;
        store_u(static_cast<uint16_t *>(p.out) + first + j * p.ld_out, p.ld_out, n, f, in,
                count - j, p.idesc & (1u << 7));
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    if (by_row) {
      const int r = __shfl_sync(~0u, row, j);
      if (in && r >= 0) store_out<MODE, PLANES>(p, int64_t(r) * p.ld_out, n, v[j] * scale);
    } else if (in && j < count && !(check && owner[t.q0 + c0 + j] == -2)) {
      store_out<MODE, PLANES>(p, first + j * p.ld_out, n, v[j] * scale);
    }
  }
}

// Eight values as they are stored, 16 bytes or 32.
template <typename T>
struct Eight {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ float get(int i) const {
    return float(reinterpret_cast<const T *>(w)[i]);
  }
};
// Eight values from p, those from `left` on (and all without `on`) as zeros.  VEC: p is on a
// 16-byte boundary and left >= 8.
template <bool VEC, typename T>
__device__ __forceinline__ Eight<T> load8(const T *p, bool on, int64_t left) {
  Eight<T> v;
#pragma unroll
  for (int i = 0; i < int(sizeof(T) / 2); ++i) v.w[i] = make_uint4(0, 0, 0, 0);
  if constexpr (VEC) {
    if (on) {
#pragma unroll
      for (int i = 0; i < int(sizeof(T) / 2); ++i) v.w[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (on && j < left) reinterpret_cast<T *>(v.w)[j] = p[j];
  }
  return v;
}

// All threads of the result warps; `tid` numbers them.
__device__ __forceinline__ void results_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
}

// The adapters' part of columns [c0, c1) of a tile (rows of x), to sums[column][lane]:
// sum_j u[row, j] b[g, j, n].  Few rows: b is read once per row and lane, on the CUDA cores,
// while the weights stream: `rank` loads of 16 bytes a thread in flight for eight n of one row.
template <typename T, bool VEC>
__device__ __forceinline__ void add_adapters_as(const Params &p, const int *owner, const Tile &t,
                                                int c0, int c1, float *sums, int tid) {
  const T *const b = static_cast<const T *>(p.b);
  constexpr int kAhead = VEC ? (sizeof(T) == 2 ? 16 : 4) : 2;      // loads in flight
  if (!p.trans_b) {
    // b stored rank x N: 16 threads a row, eight n each.
    const int l = (tid & 15) * 8, n = t.n0 + l;
    for (int col = c0 + (tid >> 4); col < c1; col += 32 * kEpiWarps / 16) {
      float v[8] = {};
      const int g = owner[t.q0 + col];
      if (g >= 0 && n < p.N) {
        const T *const bn = b + int64_t(g) * p.stride_b + n;
        const float *const u = p.u + int64_t(t.q0 + col) * p.ldu;
        for (int j0 = 0; j0 < p.rank; j0 += kAhead) {
          Eight<T> w[kAhead];
          float f[kAhead];
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            const bool on = j0 + j < p.rank;
            w[j] = load8<VEC>(bn + int64_t(j0 + j) * p.ldb, on, p.N - n);
            f[j] = on ? u[j0 + j] : 0.0f;
          }
#pragma unroll
          for (int j = 0; j < kAhead; ++j)
            if (VEC || j0 + j < p.rank)
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = fmaf(f[j], w[j].get(i), v[i]);
        }
      }
      float4 *const to = reinterpret_cast<float4 *>(sums + col * 128 + l);
      to[0] = make_float4(v[0], v[1], v[2], v[3]);
      to[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
    // b stored N x rank: a thread an n, eight ranks at a time.
    const int l = tid & 127, n = t.n0 + l;
    for (int col = c0 + (tid >> 7); col < c1; col += 32 * kEpiWarps / 128) {
      float v = 0.0f;
      const int g = owner[t.q0 + col];
      if (g >= 0 && n < p.N) {
        const T *const bn = b + int64_t(g) * p.stride_b + int64_t(n) * p.ldb;
        const float *const u = p.u + int64_t(t.q0 + col) * p.ldu;
        constexpr int kNow = kAhead / 2;
        for (int j0 = 0; j0 < p.rank; j0 += 8 * kNow) {
          Eight<T> w[kNow];
#pragma unroll
          for (int j = 0; j < kNow; ++j)
            w[j] = load8<VEC>(bn + j0 + 8 * j, j0 + 8 * j < p.rank, p.rank - j0 - 8 * j);
#pragma unroll
          for (int j = 0; j < kNow; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (j0 + 8 * j + i < p.rank) v = fmaf(u[j0 + 8 * j + i], w[j].get(i), v);
        }
      }
      sums[col * 128 + l] = v;
    }
  }
}
template <typename T>
__device__ __forceinline__ void add_adapters(const Params &p, const int *owner, const Tile &t,
                                             int c0, int c1, float *sums, int tid) {
  grid_wait();      // u is the launch before's
  if (p.vec_b) add_adapters_as<T, true>(p, owner, t, c0, c1, sums, tid);
  else add_adapters_as<T, false>(p, owner, t, c0, c1, sums, tid);
}

// FP32 on single blocks: one tile's slices [s0, s1), split into planes by the 16 copy warps.  A
// slice is 128 x 64 values of P and up to 64 x 64 of Q, split by eight of the warps -- the other
// eight have the next one's in flight -- in chunks of eight values that are contiguous as stored,
// so both majors are read in rows.  Reading FP32 operands in place costs 4 bytes a
// value, planes made by a kernel before 4 + 6 + 6.  False when a wait ran out.
template <int MODE, bool VEC>
__device__ __forceinline__ bool split_tile(const Params &p, const Tile &t, int s0, int s1,
                                           uint32_t base, uint32_t bar_full, uint32_t bar_empty,
                                           Ring &ring, bool &dropped, int64_t limit_ns) {
  using S = Shape<1, 3>;
  static_assert(S::kStages == 2 && S::kCopyWarps == 16, "eight warps for each of two stages");
  const int warp = (threadIdx.x >> 5) & 7, team = threadIdx.x >> 8, lane = threadIdx.x & 31;
  const bool mn = MODE == kWgrad || p.p_mn;
  const float *const P = p.fp + (MODE == kWgrad || p.p_shared ? 0 : int64_t(t.g) * p.stride_p);
  // Chunks of P: row r (of n, or of k where n is contiguous) and column 8 c; of Q likewise.
  const int pc = mn ? lane & 15 : lane & 7;
  const int pr = mn ? 8 * warp + (lane >> 4) : 16 * warp + (lane >> 3);
  const int pstep = mn ? 2 : 4;        // to the thread's next row
  const int qc = lane & 7, qr = 8 * warp + (lane >> 3);
  int qrow[2] = {-1, -1};              // forward: the rows of x
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (MODE != kWgrad && qr + 4 * i < t.qn) {
      const int at = t.q0 + qr + 4 * i;
      qrow[i] = MODE == kForward && p.row_index ? p.row_index[at] : at;
      if (qrow[i] >= p.q_rows) qrow[i] = -1;
    }
  struct Chunks {
    Eight<float> p[4], q[2];
  };
  const auto load = [&](int s) {
    Chunks v;
    const int k0 = s * kBK;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = pr + i * pstep;
      if (mn) {
        const int k = k0 + r, n = t.n0 + 8 * pc;
        v.p[i] = load8<VEC>(P + (MODE == kWgrad ? int64_t(t.k0) + k : int64_t(k)) * p.ldp + n,
                            k < t.klen && n < p.N, p.N - n);
      } else {
        const int n = t.n0 + r, k = k0 + 8 * pc;
        v.p[i] = load8<VEC>(P + int64_t(n) * p.ldp + k, n < p.N && k < t.klen, t.klen - k);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (MODE == kWgrad) {
        const int k = k0 + qr + 4 * i, c = t.q0 + 8 * qc;
        int row = -1;
        if (k < t.klen) {
          row = p.row_index ? p.row_index[t.k0 + k] : t.k0 + k;
          if (row >= p.q_rows) row = -1;
        }
        v.q[i] = load8<VEC>(p.fx + int64_t(max(row, 0)) * p.ldx + c, row >= 0 && c < p.q_cols,
                            p.q_cols - c);
      } else {
        const int k = k0 + 8 * qc;
        v.q[i] = load8<VEC>(p.fx + int64_t(max(qrow[i], 0)) * p.ldx + k,
                            qrow[i] >= 0 && k < t.klen, t.klen - k);
      }
    }
    return v;
  };
  const auto store8 = [&](const Eight<float> &v, uint32_t to, uint32_t plane) {
    float f[8];
    uint32_t h[3][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = v.get(i);
    split8(f, h);
#pragma unroll
    for (int pl = 0; pl < 3; ++pl)
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + pl * plane),
                   "r"(h[pl][0]), "r"(h[pl][1]), "r"(h[pl][2]), "r"(h[pl][3])
                   : "memory");
  };
  const auto put = [&](const Chunks &v) {
    const bool ok = mbar_wait(bar_empty + 8 * ring.stage, ring.parity ^ 1u, limit_ns);
    if (!__all_sync(~0u, ok)) return false;
    const uint32_t st = base + ring.stage * S::kStage, sq = st + 3 * kPTile;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = pr + i * pstep;
      const uint32_t at = mn ? uint32_t((pc >> 3) * 8192 + r * 128 + (((pc & 7) ^ (r & 7)) << 4))
                             : uint32_t(r * 128 + ((pc ^ (r & 7)) << 4));
      store8(v.p[i], st + at, kPTile);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = qr + 4 * i;
      store8(v.q[i], sq + uint32_t(r * 128 + ((qc ^ (r & 7)) << 4)), S::kQTile);
    }
    proxy_fence();
    __syncwarp();
    if (lane == 0 && !(dropped && warp == 0)) mbar_arrive_local(bar_full + 8 * ring.stage);
    return true;
  };
  for (int s = s0; s < s1; ++s) {
    if (ring.stage == team && !put(load(s))) return false;
    dropped = false;
    ring.template next<S::kStages>();
  }
  return true;
}

// ---- kernel -----------------------------------------------------------------------------

// BP: parts of b in the adapters' part on pairs, 2 where it is FP16 (half_parts).
template <int CG, int MODE, int PLANES, int BP = 1>
__global__ void __launch_bounds__(Shape<CG, PLANES>::kThreads, 1)
grouped_kernel(const __grid_constant__ CUtensorMap map_p,    // P tiles
               const __grid_constant__ CUtensorMap map_q,    // Q tiles
               const __grid_constant__ CUtensorMap map_qr,   // single rows of x; pairs: tiles of
                                                             // all the columns of a block
               const __grid_constant__ CUtensorMap map_e,    // b tiles; gradient: 16 rows of dy
               const __grid_constant__ CUtensorMap map_u,    // u tiles; gradient: 16 rows of x
               const __grid_constant__ CUtensorMap map_pr,   // gradient: single rows of dy
               const Params p) {
  using S = Shape<CG, PLANES>;
  // The adapters' part: pairs extend the sum (EXT); single blocks, whose rows are few, add it to
  // the results on the CUDA cores while the weights stream (FEW).
  constexpr bool EXT = MODE == kLora && CG == 2, FEW = MODE == kLora && CG == 1;
  constexpr int RS = rank_slice(PLANES, BP);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;    // the same offset in every block
  uint8_t *const smem = smem_raw + (base - raw);
  const uint32_t red = base + S::kStages * S::kStage;
  const uint32_t out_stage = red + S::kRed;
  const uint32_t table = out_stage + S::kOutStage;
  const uint32_t bar_full = (table + S::kTable + 7u) & ~7u;
  const uint32_t bar_empty = bar_full + 8 * S::kStages;
  const uint32_t bar_tfull = bar_empty + 8 * S::kStages;
  const uint32_t bar_tempty = bar_tfull + 16;      // pairs: used in the leader
  const uint32_t bar_drain = bar_tempty + 16;
  const uint32_t slot = bar_drain + 8;             // tensor memory address; then the counts

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int *const tab_gid = reinterpret_cast<int *>(smem + (table - base));
  int *const tab_row = tab_gid + kListed;
  int *const tab_tile = tab_row + kListed;
  // Row numbers that a copy warp is about to fetch, four to a copy; 16-byte aligned.
  int *const my_rows = reinterpret_cast<int *>(
      (reinterpret_cast<uintptr_t>(tab_tile + kListed) + 15) & ~uintptr_t(15)) + 32 * warp;
  int *const owner = tab_gid + (S::kTable / 4 - kFewRows);      // adapters on single blocks
  volatile uint32_t *const slot_ptr = reinterpret_cast<volatile uint32_t *>(smem + (slot - base));
  float *const red_ptr = reinterpret_cast<float *>(smem + (red - base));

  const uint32_t rank = cluster_rank();
  const int cluster_size = CG == 2 ? 2 : p.ksplit;
  const int cluster = int(blockIdx.x) / cluster_size;
  const int clusters = int(gridDim.x) / cluster_size;
  const bool leader = CG == 1 || rank == 0;
  const int half_rank = CG == 2 ? int(rank) : 0;   // which 128 lanes, which half of the columns

  // Barriers and tensor memory; then, once the launches before are done, the group offsets,
  // clamped, into the (still unused) ring.
  int *const offs = reinterpret_cast<int *>(smem);
  if (threadIdx.x == 0) {
    // A slice is there once every warp that waits for its stage to be free has arrived, whether or not
    // it had something to copy: one that nothing waits for could fall two rounds behind, and wait for
    // a phase that has passed.
    const int rows_by_number = CG == 1 && MODE != kLora && p.row_index ? S::kCopyWarps : 1;
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(bar_full + 8 * s, S::kDirect ? S::kCopyWarps / 2 : rows_by_number);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_tfull + 8 * b, 1);
      mbar_init(bar_tempty + 8 * b, CG * kEpiWarps);
    }
    mbar_init(bar_drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == S::kMmaWarp) {
    if constexpr (CG == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
                   "r"(S::kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
                   "r"(S::kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  if (!S::kDirect && warp == 0 && elect_one()) {
    prefetch_map(&map_p);
    prefetch_map(&map_q);
    prefetch_map(&map_qr);
  }
  // The adapters' product follows the one that makes u, and needs nothing else of it: its wait
  // comes before the first slice of u, so that the shared projection starts beside it.
  if (MODE != kLora) {
    grid_wait();
    grid_start_next();
  }
  for (int g = threadIdx.x; g <= p.groups; g += S::kThreads)
    offs[g] = max(0, min(p.offsets[g], p.rows));
  __syncthreads();
  if (warp == 0) {
    // Group bounds are the running maximum of the offsets: offsets that step back make an
    // empty group, never an overlap.  Groups without rows are left out of the list (kept in
    // the gradient, whose result has a matrix for each).
    int carry = offs[0], count = 0, tiles = 0;
    if (lane == 0) slot_ptr[3] = uint32_t(carry);       // first row of any group
    if (EXT && carry > 0) {
      if (lane == 0) {
        tab_gid[0] = -1;
        tab_row[0] = tab_tile[0] = 0;
      }
      count = 1;
      tiles = (carry + 31) / 32;
    }
    if (MODE == kWgrad && lane == 0) tab_row[0] = carry;
    for (int g0 = 0; g0 < p.groups; g0 += 32) {
      const int g = g0 + lane;
      int hi = g < p.groups ? offs[g + 1] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(~0u, hi, d);
        if (lane >= d) hi = max(hi, o);
      }
      hi = max(hi, carry);
      int lo = __shfl_up_sync(~0u, hi, 1);
      if (lane == 0) lo = carry;
      carry = __shfl_sync(~0u, hi, 31);
      if (MODE == kWgrad) {
        if (g < p.groups) tab_row[g + 1] = hi;
      } else {
        const int n = g < p.groups ? hi - lo : 0;
        const unsigned have = __ballot_sync(~0u, n > 0);
        const int at = count + __popc(have & ((1u << lane) - 1));
        const int mine = EXT ? (n + 31) / 32 : (n + p.tile_n - 1) / p.tile_n * p.panels;
        int sum = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(~0u, sum, d);
          if (lane >= d) sum += o;
        }
        if (n > 0) {
          tab_gid[at] = g;
          tab_row[at] = lo;
          tab_tile[at] = tiles + sum - mine;
        }
        tiles += __shfl_sync(~0u, sum, 31);
        count += __popc(have);
      }
    }
    if (lane == 0) {
      if (EXT && carry < p.rows) {
        tab_gid[count] = -1;
        tab_row[count] = carry;
        tab_tile[count++] = tiles;
        tiles += (p.rows - carry + 31) / 32;
      }
      if (EXT) {
        tab_row[count] = p.rows;
        tab_tile[count] = tiles;
        tiles = p.panels * ((32 * tiles + p.tile_n - 1) / p.tile_n);
      } else if (MODE != kWgrad) {
        tab_row[count] = carry;
      }
      if (MODE == kWgrad) tiles = p.groups * p.panels * ((p.q_cols + p.tile_n - 1) / p.tile_n);
      if (FEW) tiles = p.panels * ((p.rows + p.tile_n - 1) / p.tile_n);
      slot_ptr[1] = uint32_t(count);
      slot_ptr[2] = uint32_t(tiles);
      slot_ptr[4] = uint32_t(carry);                    // end of the last group
    }
    proxy_fence();      // the ring is written by the copy engine from here on
  }
  if constexpr (MODE == kWgrad) {
    // The order of the groups: most rows first, so that the rounds of tiles, handed out in turn,
    // end with the short ones (8 groups of a router's sizes, 4096 x 4096: 8 % less).
    __syncthreads();
    for (int g = threadIdx.x; g < p.groups; g += S::kThreads) {
      const int n = tab_row[g + 1] - tab_row[g];
      int before = 0;
      for (int h = 0; h < p.groups; ++h) {
        const int m = tab_row[h + 1] - tab_row[h];
        before += m > n || (m == n && h < g);
      }
      tab_gid[before] = g;
    }
  }
  if constexpr (FEW) {
    // The adapter of every row of x: its list entry's number, -1 for none, -2 for a row that the
    // order does not name (which is not written).
    for (int i = threadIdx.x; i < kFewRows; i += S::kThreads) owner[i] = -2;
    __syncthreads();
    const int count = int(slot_ptr[1]);
    for (int i = threadIdx.x; i < p.rows; i += S::kThreads) {
      const int row = p.row_index ? p.row_index[i] : i;
      int a = 0, b = count;        // entries that start at or before place i
      while (a < b) {
        const int m = (a + b) >> 1;
        if (tab_row[m] <= i) a = m + 1;
        else b = m;
      }
      if (row >= 0 && row < p.rows) owner[row] = a > 0 && i < tab_row[a] ? tab_gid[a - 1] : -1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();   // barriers exist before any remote arrival
  tc_fence_after();
  const uint32_t tmem = slot_ptr[0];
  const Table tab = {tab_gid, tab_row, tab_tile, int(slot_ptr[1]), int(slot_ptr[2])};

  bool timed_out = false;
  Ring ring = {0, 0};
  uint32_t q = 0;      // tensor-memory sums so far
  bool dropped = int(blockIdx.x) == p.drop_block;   // testing hook: the next expectation is wrong

  // Forward: rows of the result that belong to no group are zero, a warp a row.
  if (MODE == kForward && p.zero_rows && warp >= S::kEpi0 && warp < S::kMmaWarp) {
    const int lo = int(slot_ptr[3]), hi = int(slot_ptr[4]);
    const int64_t count = int64_t(lo) + (p.rows - hi);
    for (int64_t i = int64_t(blockIdx.x) * kEpiWarps + warp - S::kEpi0; i < count;
         i += int64_t(gridDim.x) * kEpiWarps) {
      const int64_t row = (i < lo ? i : hi + (i - lo)) * p.ld_out;
      if (p.vec_out && p.N % 8 == 0) {
        for (int n = lane * 8; n < p.N; n += 256)
          *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + row + n) =
              make_uint4(0, 0, 0, 0);
      } else {
        for (int n = lane; n < p.N; n += 32) store_out<MODE, PLANES>(p, row, n, 0.0f);
      }
    }
  }

  for (int t = cluster; t < tab.tiles; t += clusters) {
    if (timed_out && p.ksplit == 1 && !FEW) break;     // (else warps meet at every tile)
    const int64_t limit_ns = timed_out ? 0 : p.wait_limit_ns;      // a warp waits in vain only once
    const Tile tile = tile_at<CG, MODE, PLANES>(p, tab, t);
    int nbase, s0, s1;
    slices_of<EXT, RS>(p, tile, CG == 2 ? 0 : int(rank), nbase, s0, s1);
    const int per_rank = EXT ? (p.rank + RS - 1) / RS : 1;

    if (S::kDirect && warp < S::kCopyWarps) {
      if constexpr (S::kDirect) {
        const bool ok = p.vec ? split_tile<MODE, true>(p, tile, s0, s1, base, bar_full, bar_empty,
                                                       ring, dropped, limit_ns)
                              : split_tile<MODE, false>(p, tile, s0, s1, base, bar_full, bar_empty,
                                                        ring, dropped, limit_ns);
        if (!ok) timed_out = true;
      }
    } else if (!S::kDirect && warp < S::kCopyWarps) {
      // ---- copies ----
      const int hr = tile.bn / CG;                      // columns staged by this block
      const int qf = tile.q0 + half_rank * hr;          // the first of them
      const int n0 = tile.n0 + half_rank * 128;
      const int pg = (p.p_shared ? 0 : tile.g);
      const int pcount = p.p_shared ? 1 : p.groups;
      // Columns of a block that hold rows: the others' sums are not stored, so whatever their
      // part of the ring holds will do.
      const auto held = [&](int half) { return max(0, min(tile.qn - half * hr, hr)); };
      const int mine = held(half_rank);
      // (One at least: the slice waits for the warp that copies it, see the barriers' counts.)
      const auto boxes_of = [&](int half) { return max(1, (held(half) + S::kBox - 1) / S::kBox); };
      const auto whole = [&](int half) { return CG == 2 && held(half) * CG == p.tile_n; };
      const int boxes = boxes_of(half_rank);
      const int qblocks = hr / 64;
      // The first row of every copy of Q, and whether they follow one another in a full tile.
      constexpr int kBoxes = S::kBN / CG / S::kBox;
      int box_row[kBoxes];
      bool in_one = whole(half_rank);
      int e = tile.g;
#pragma unroll
      for (int b = 0; b < kBoxes; ++b) {
        box_row[b] = qf + b * S::kBox;
        if (EXT && b < boxes && mine > 0) {
          while (tab.tile[e + 1] * 32 <= qf + b * 32) ++e;
          box_row[b] = tab.row[e] + qf + b * 32 - tab.tile[e] * 32;
          in_one &= box_row[b] == box_row[0] + b * 32;
        }
      }
      const bool by_row = CG == 1 && MODE != kLora && p.row_index != nullptr;
      uint32_t usual = 0;      // bytes of an ordinary slice, of both blocks of a pair
      if (MODE == kWgrad) {
        usual = CG * PLANES * (kPTile + uint32_t(qblocks) * 8192u);
      } else {
#pragma unroll
        for (int h = 0; h < CG; ++h)
          usual += PLANES * (kPTile + uint32_t(by_row         ? (held(h) + 3) / 4 * 512
                                               : whole(h) ? hr * 128
                                                          : boxes_of(h) * (S::kBox * 128)));
      }

      // What a slice s is.  A group's last slice in the gradient has to end in rows of zeros: it
      // comes in copies of 16 rows and, for the rows that are not 16, of four by number, where one
      // outside the matrix reads as zeros.  (The copy of a whole slice, and its last rows zeroed in
      // shared memory afterwards, held the products up by 1250 cycles a tile, most of it the
      // cluster-wide release of the zeros: 1000 rows in each of 8 groups, 4096 x 4096,
      // 182 us in place of 167.)
      struct Slice {
        bool ext;
        int k0, g, gcount, rank0, row;      // ext: ranks from rank0, rows of u from row
        int cnt;                            // gradient: rows of the group; ext: copies of u
      };
      const auto slice_at = [&](int s) {
        Slice c = {EXT && s >= nbase, s * kBK, pg, pcount, 0, 0, kBK};
        if (MODE == kWgrad) {
          c.k0 += tile.k0;
          c.cnt = min(kBK, tile.klen - s * kBK);
        } else if (EXT && c.ext) {
          const int e = (s - nbase) / per_rank;
          const int j = s - nbase - e * per_rank;
          c.k0 = j * kBK;                    // of u
          c.rank0 = j * (p.e_mn ? RS : BP * RS);      // of b (N x rank, two parts: plan_parts)
          c.g = p.e_shared ? 0 : tab.gid[tile.e0 + e];
          c.gcount = p.e_shared ? 1 : p.groups;
          // This block's half of the entry's columns, 16 n32 rows.
          const Part part = part_of(p, tab, tile, tile.e0 + e);
          c.row = part.row + half_rank * 16 * part.n32;
          c.cnt = (part.n32 + 1) / 2;
        }
        return c;
      };
      const auto bytes_of = [&](const Slice &c) {
        if (MODE == kWgrad)
          return uint32_t(PLANES) * ((c.cnt + 15) / 16 * 2048 * (2 + qblocks));
        return PLANES * ((p.e_mn ? BP * 2 * RS * 128 : kPTile) +
                         uint32_t(c.cnt * (S::kBox * 128)));
      };
      // A slice that slice_at describes as ordinary in every respect.
      const auto is_plain = [&](int s) {
        if (MODE == kWgrad) return (s + 1) * kBK <= tile.klen;
        return !EXT || s < nbase;
      };
      const auto full_at = [&](int stage) {
        const uint32_t bar = bar_full + 8 * stage;
        return CG == 2 ? map_rank(bar, 0) : bar;
      };
      const auto expect = [&](int stage, uint32_t bytes) {
        mbar_expect(bar_full + 8 * stage, bytes + (dropped ? 16 : 0));
        dropped = false;
      };
      // A group's last rows, rounded up to 16 (one thread): `blocks` of 64 columns from column x,
      // planes `plane` bytes and `rows` rows apart.
      const auto copy_end = [&](const Slice &c, uint32_t to, const CUtensorMap *map16,
                                const CUtensorMap *map1, int x, int blocks, uint32_t plane,
                                int rows, uint32_t bar) {
        const int whole16 = c.cnt >> 4, left = c.cnt & 15;
#pragma unroll
        for (int pl = 0; pl < PLANES; ++pl) {
          const int row = c.k0 + pl * rows;
#pragma unroll
          for (int i = 0; i < 3; ++i)
            if (i < whole16) {
#pragma unroll
              for (int b = 0; b < 2; ++b)
                if (b < blocks)
                  tma_2d<CG>(to + uint32_t(b * 8192 + i * 2048), map16, x + b * 64, row + 16 * i,
                             bar);
            }
          if (left > 0) {
            const int out = PLANES * rows, first = row + 16 * whole16;
            const uint32_t at = to + uint32_t(whole16 * 2048);
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              int y[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) y[k] = 4 * f + k < left ? first + 4 * f + k : out;
#pragma unroll
              for (int b = 0; b < 2; ++b)
                if (b < blocks)
                  tma_rows4<CG>(at + uint32_t(b * 8192 + f * 512), map1, x + b * 64, y, bar);
            }
          }
          to += plane;
        }
      };
      // Copies of P, and of Q as tiles, of one slice (one thread).
      const auto copy_p = [&](const Slice &c, uint32_t st, uint32_t bar) {
        if (MODE == kWgrad && c.cnt < kBK) {
          copy_end(c, st, &map_e, &map_pr, n0, 2, 2 * 8192, p.rows, bar);
        } else if (MODE == kWgrad) {
#pragma unroll
          for (int i = 0; i < 2 * PLANES; ++i)
            tma_2d<CG>(st + i * 8192, &map_p, n0 + (i & 1) * 64, c.k0 + (i >> 1) * p.rows, bar);
        } else if (EXT && c.ext) {
          if (p.e_mn) {
#pragma unroll
            for (int i = 0; i < 2 * PLANES; ++i)
              tma_3d<CG>(st + i * 8192, &map_e, n0 + (i & 1) * 64, c.rank0,
                         c.g + (i >> 1) * c.gcount, bar);
            // The second part of b, 16 more values of the sum.
            if (BP == 2) {
#pragma unroll
              for (int i = 0; i < 2; ++i)
                tma_3d<CG>(st + i * 8192 + 2048, &map_e, n0 + i * 64, c.rank0, c.g + c.gcount, bar);
            }
          } else {
#pragma unroll
            for (int i = 0; i < PLANES; ++i)
              tma_3d<CG>(st + i * kPTile, &map_e, c.rank0, n0, c.g + i * c.gcount, bar);
          }
        } else if (p.p_mn) {
#pragma unroll
          for (int i = 0; i < 2 * PLANES; ++i)
            tma_3d<CG>(st + i * 8192, &map_p, n0 + (i & 1) * 64, c.k0, pg + (i >> 1) * pcount, bar);
        } else {
#pragma unroll
          for (int i = 0; i < PLANES; ++i)
            tma_3d<CG>(st + i * kPTile, &map_p, c.k0, n0, pg + i * pcount, bar);
        }
      };
      const auto copy_q = [&](const Slice &c, uint32_t sq, uint32_t bar) {
        if (MODE == kWgrad && c.cnt < kBK) {
          copy_end(c, sq, &map_u, &map_qr, qf, qblocks, S::kQTile, p.q_rows, bar);
        } else if (MODE == kWgrad) {
          for (int pl = 0; pl < PLANES; ++pl)
            for (int b = 0; b < qblocks; ++b)
              tma_2d<CG>(sq + pl * S::kQTile + b * 8192, &map_q, qf + b * 64, c.k0 + pl * p.q_rows,
                         bar);
        } else if (EXT && c.ext) {
          for (int pl = 0; pl < PLANES; ++pl)
            for (int b = 0; b < c.cnt; ++b)
              tma_2d<CG>(sq + pl * S::kQTile + b * (S::kBox * 128), &map_u, c.k0,
                         c.row + b * S::kBox + pl * p.rows, bar);
        } else if (in_one) {
          // A full tile: one copy a plane.
#pragma unroll
          for (int pl = 0; pl < PLANES; ++pl)
            tma_2d<CG>(sq + pl * S::kQTile, &map_qr, c.k0, box_row[0] + pl * p.q_rows, bar);
        } else {
#pragma unroll
          for (int pl = 0; pl < PLANES; ++pl)
#pragma unroll
            for (int b = 0; b < kBoxes; ++b)
              if (b < boxes)
                tma_2d<CG>(sq + pl * S::kQTile + b * (S::kBox * 128), &map_q, c.k0,
                           box_row[b] + pl * p.q_rows, bar);
        }
      };
      // The expectations of one slice (one thread, before or while its copies arrive).
      const auto announce = [&](const Slice &c, int stage) {
        if (leader) expect(stage, CG * bytes_of(c));      // of both blocks of a pair
      };
      if (!by_row) {
        // Warp 0 copies P, warp 1 copies Q, one thread each.
        if (warp < 2) {
          if (elect_one()) {
            for (int s = s0; s < s1; ++s) {
              const uint32_t st = base + ring.stage * S::kStage;
              if (!mbar_wait(bar_empty + 8 * ring.stage, ring.parity ^ 1u, limit_ns)) {
                timed_out = true;
                break;
              }
              if (is_plain(s)) {
                const Slice c = {false, MODE == kWgrad ? tile.k0 + s * kBK : s * kBK, 0, 0, 0, 0,
                                 kBK};
                const uint32_t full = full_at(ring.stage);
                if (warp == 0) {
                  if (leader) expect(ring.stage, usual);
                  copy_p(c, st, full);
                } else {
                  copy_q(c, st + PLANES * kPTile, full);
                }
              } else {
                if (EXT) grid_wait();
                const Slice c = slice_at(s);
                const uint32_t bar = full_at(ring.stage);
                if (warp == 0) {
                  announce(c, ring.stage);
                  copy_p(c, st, bar);
                } else {
                  copy_q(c, st + PLANES * kPTile, bar);
                }
              }
              ring.template next<S::kStages>();
            }
          }
          __syncwarp();
          timed_out = __any_sync(~0u, timed_out);
        }
      } else {
        // Rows by number, four to a copy (single blocks), by warps 1 to 3, while warp 0 copies P:
        // warp w issues fours w - 1, w + 2, ...; lane l looks up row l % 4 of the warp's four l / 4;
        // -1 is a row of zeros.  (Such a copy takes the copy engine about 40 cycles.  The 12 of a
        // slice of 48 columns keep up with the memory; more do not, and there, as on pairs, the
        // rows are gathered by a kernel first.  16384 rows x 4096 x 4096 on pairs: 620 us by
        // number, 331 us + 40 us gathered.  cp.async by the copy warps, counted by a barrier: 758
        // us.)
        const int row_in_slice = 4 * (warp - 1 + 3 * (lane >> 2)) + (lane & 3);
        const auto row_of = [&](int at, int limit) {
          if (at >= limit) return -1;
          const int row = p.row_index[at];
          return row >= 0 && row < p.q_rows ? row : -1;
        };
        int next = -1;      // gradient: this lane's row of the next slice
        if (warp == 0) {
        } else if (MODE != kWgrad) {
          __syncwarp();
          my_rows[lane] = row_of(qf + row_in_slice, tile.q0 + tile.qn);
          __syncwarp();
        } else if (s0 < s1 && lane < 24) {
          next = row_of(tile.k0 + s0 * kBK + row_in_slice, tile.k0 + tile.klen);
        }
        for (int s = s0; s < s1 && !timed_out; ++s) {
          const uint32_t st = base + ring.stage * S::kStage, sq = st + PLANES * kPTile;
          const bool ok = mbar_wait(bar_empty + 8 * ring.stage, ring.parity ^ 1u, limit_ns);
          if (!__all_sync(~0u, ok)) {
            timed_out = true;
            break;
          }
          const Slice c = slice_at(s);
          const uint32_t bar = bar_full + 8 * ring.stage;
          if (warp == 0 && elect_one()) {
            if (is_plain(s) && MODE != kWgrad) expect(ring.stage, usual);
            else announce(c, ring.stage);
            copy_p(c, st, bar);
          }
          dropped = false;
          __syncwarp();
          if (MODE == kWgrad && warp > 0) {
            if (lane < 24) my_rows[lane] = next;
            __syncwarp();
            if (s + 1 < s1 && lane < 24)
              next = row_of(c.k0 + kBK + row_in_slice, tile.k0 + tile.klen);
          }
          if (warp > 0 && elect_one()) {
            const int fours = MODE == kWgrad ? (c.cnt + 15) / 16 * 4 : (mine + 3) / 4;
            const int x = MODE == kWgrad ? qf : c.k0;
            for (int f = warp - 1, k = 0; f < fours; f += 3, ++k) {
              const int4 v = *reinterpret_cast<const int4 *>(my_rows + 4 * k);
#pragma unroll
              for (int pl = 0; pl < PLANES; ++pl) {
                const int out = PLANES * p.q_rows, add = pl * p.q_rows;
                const int y[4] = {v.x < 0 ? out : v.x + add, v.y < 0 ? out : v.y + add,
                                  v.z < 0 ? out : v.z + add, v.w < 0 ? out : v.w + add};
                for (int b = 0; b < (MODE == kWgrad ? qblocks : 1); ++b)
                  tma_rows4<CG>(sq + pl * S::kQTile + b * 8192 + f * 512, &map_qr, x + b * 64, y,
                                bar);
              }
            }
            mbar_arrive_local(bar);
          }
          __syncwarp();
          ring.template next<S::kStages>();
        }
      }
    } else if (warp == S::kMmaWarp) {
      // ---- products ---- (one thread)
      if (leader && elect_one()) {
        const auto size_of = [&](int columns) {
          return (uint32_t(columns >> 3) << 17) | (uint32_t(128 * CG >> 4) << 24) |
                 (MODE == kWgrad ? 1u << 16 : 0u);
        };
        const bool base_mn = MODE == kWgrad || p.p_mn;
        const uint32_t qstep = MODE == kWgrad ? 128 : 2;      // 16 values of K, in 16 bytes
        const int n = s1 - s0;
        // Slices [begin, last] of 16-bit operands make one tensor-memory sum; those of adapters
        // belong to the last one of the base sum.
        const int nb = EXT ? nbase : n;
        const int each = PLANES == 3 ? 0 : long_sum(nb);
        const auto last_of = [&](int from) { return nb - from <= each ? n - 1 : from + each - 1; };
        int begin = 0, last = last_of(0);
        // Waits for a slice's operands and, with the first of a tensor-memory sum, for its buffer.
        const auto ready = [&](bool first) {
          if (first) {
            if (q >= 2 && !mbar_wait(bar_tempty + 8 * (q & 1), ((q >> 1) - 1) & 1u,
                                     limit_ns))
              return false;
            ++q;
          }
          if (!mbar_wait(bar_full + 8 * ring.stage, ring.parity, limit_ns)) return false;
          tc_fence_after();
          return true;
        };
        // `steps` times 16 values of the sum to column c0 of the tile, `fresh`: its first ones.
        const auto products = [&](uint32_t idesc, bool mn, int c0, int steps, bool fresh) {
          const uint32_t st = base + ring.stage * S::kStage;
          const uint64_t dp = tile_desc(st, mn);
          const uint64_t dq = tile_desc(st + PLANES * kPTile, MODE == kWgrad);
          const uint32_t pstep = mn ? 128 : 2;
          const uint32_t d = tmem + ((q - 1) & 1) * S::kBN + c0;
          idesc |= mn ? 1u << 15 : 0u;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k >= steps) break;
            const uint64_t a = dp + k * pstep, b = dq + k * qstep;
            mma<CG>(d, a, b, idesc, !(fresh && k == 0));
            if constexpr (PLANES == 3) {
              constexpr uint64_t pa = kPTile >> 4, qa = S::kQTile >> 4;
              const uint32_t ds = d + 2 * S::kBN;      // the lower parts' products
              mma<CG>(ds, a + 2 * pa, b, idesc, !(fresh && k == 0));
              mma<CG>(ds, a, b + 2 * qa, idesc, true);
              mma<CG>(ds, a + pa, b + qa, idesc, true);
              mma<CG>(ds, a + pa, b, idesc, true);
              mma<CG>(ds, a, b + qa, idesc, true);
            }
          }
        };
        // Slice i's products have been issued.
        const auto finish = [&](int i) {
          mma_commit<CG>(bar_empty + 8 * ring.stage, true);
          if (PLANES == 3 ? i == n - 1 || i % kChunk == kChunk - 1 : i == last) {
            mma_commit<CG>(bar_tfull + 8 * ((q - 1) & 1), true);
            begin = i + 1;
            last = last_of(begin);
          }
          ring.template next<S::kStages>();
        };
        const uint32_t all = size_of(tile.bn) | p.idesc;
        bool ok = true;
        for (int i = 0; i < nb; ++i) {
          const bool first = PLANES == 3 ? i % kChunk == 0 : i == begin;
          if (!(ok = ready(first))) break;
          products(all, base_mn, 0, (min(kBK, tile.klen - (s0 + i) * kBK) + 15) / 16, first);
          finish(i);
        }
        if constexpr (EXT) {
          // The adapters' parts, each on its columns alone.
          int i = nb;
          for (int e = 0; ok && e < tile.en; ++e) {
            const Part part = part_of(p, tab, tile, tile.e0 + e);
            const uint32_t types = size_of(32 * part.n32) | p.idesc_e;
            for (int j = 0; j < per_rank; ++j, ++i) {
              if (!(ok = ready(PLANES == 3 && i % kChunk == 0))) break;
              const int steps = (min(RS, p.rank - j * RS) + 15) / 16;
              if constexpr (PLANES == 3) {
                // The first on these columns in this tensor-memory sum, if it holds adapters' slices
                // only.
                const bool fresh = i - i % kChunk >= nb && (i % kChunk == 0 || j == 0);
                products(types, p.e_mn, part.c0, steps, fresh);
              } else {
                const uint32_t st = base + ring.stage * S::kStage;
                const uint64_t dp = tile_desc(st, p.e_mn), dq = tile_desc(st + kPTile, false);
                const uint32_t pstep = p.e_mn ? 128 : 2;
                const uint32_t idesc = types | (p.e_mn ? 1u << 15 : 0u);
                const uint32_t d = tmem + ((q - 1) & 1) * S::kBN + part.c0;
                if constexpr (BP == 1) {
                  // b[g] times u's first part, and times its second, 32 columns on.
                  for (int k = 0; k < steps; ++k) {
                    const uint64_t a = dp + k * pstep, b = dq + k * 2;
                    mma<CG>(d, a, b, idesc, true);
                    mma<CG>(d, a, b + 4, idesc, true);
                  }
                } else {
                  // The first part of b times u's three, 16 columns apart, and the second times the
                  // second and, in the fourth place, the first (with the third: 2^-24 of the
                  // product).
#pragma unroll
                  for (int k = 0; k < 3; ++k) mma<CG>(d, dp, dq + 2 * k, idesc, true);
                  mma<CG>(d, dp + pstep, dq + 2, idesc, true);
                  mma<CG>(d, dp + pstep, dq + 6, idesc, true);
                }
              }
              finish(i);
            }
          }
        }
        if (!ok) timed_out = true;
      }
      __syncwarp();
      timed_out = __any_sync(~0u, timed_out);
    } else {
      // ---- results ----
      const int quarter = warp & 3, half = (warp - S::kEpi0) >> 2;
      const int n = s1 - s0;
      const uint32_t lanes = tmem + (uint32_t(32 * quarter) << 16);
      const uint32_t tempty = CG == 2 ? map_rank(bar_tempty, 0) : bar_tempty;
      const int nw = tile.n0 + half_rank * 128 + 32 * quarter;
      const uint32_t stage = out_stage + uint32_t(warp - S::kEpi0) * 1024;
      const float scale = MODE == kForward && p.scale ? p.scale[tile.g] : 1.0f;
      constexpr int kBlocks = S::kBN / 32;     // 16-column blocks of a warp, every other one
      // The columns that this block adds up and stores: all of them, or its share.
      const int own0 = CG == 1 ? tile.qn * int(rank) / p.ksplit : 0;
      const int own1 = CG == 1 ? tile.qn * int(rank + 1) / p.ksplit : tile.qn;
      if constexpr (FEW) {
        results_sync();      // the last tile's sums have been read
        const int tid = int(threadIdx.x) - 32 * S::kEpi0;
        if constexpr (PLANES == 3)
          add_adapters<float>(p, owner, tile, own0, own1, red_ptr, tid);
        else if (p.idesc & (1u << 7))
          add_adapters<__nv_bfloat16>(p, owner, tile, own0, own1, red_ptr, tid);
        else
          add_adapters<__half>(p, owner, tile, own0, own1, red_ptr, tid);
        results_sync();
      }
      int entry = tile.g;      // EXT: the entry of the last columns stored
      // EXT: the tile with the rows of the columns from c0 on, which are one entry's.
      auto rows_at = [&](int c0) {
        Tile t = tile;
        if (EXT && c0 < tile.qn) {
          const int at = tile.q0 + c0;
          while (tab.tile[entry + 1] * 32 <= at) ++entry;
          t.q0 = tab.row[entry] + at - tab.tile[entry] * 32 - c0;
          t.qn = tab.row[entry + 1] - t.q0;
        }
        return t;
      };
      auto put = [&](int c0, const float (&v)[16]) {
        if (EXT) {
          const Tile t = rows_at(c0);
          if (t.qn > c0) store_columns<MODE, PLANES>(p, t, c0, nw, v, scale, stage, owner);
        } else if (CG == 1 && (FEW || p.ksplit > 1)) {
          float w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float *const at = &red_ptr[(c0 + j) * 128 + 32 * quarter + lane];
            w[j] = v[j];
            if (FEW && c0 + j >= own0 && c0 + j < own1) w[j] += *at;
            if (p.ksplit > 1) *at = w[j];
          }
          if (p.ksplit == 1) store_columns<MODE, PLANES>(p, tile, c0, nw, w, scale, stage, owner);
        } else {
          store_columns<MODE, PLANES>(p, tile, c0, nw, v, scale, stage, owner);
        }
      };
      if constexpr (PLANES == 1) {
        if (n == 0) {
          const float v[16] = {};
          for (int c0 = 16 * half; c0 < tile.bn; c0 += 32) put(c0, v);
        } else if (const int nb = EXT ? nbase : n; nb <= kLong) {
          const uint32_t buf = q & 1;
          const bool ready =
              !timed_out && mbar_wait(bar_tfull + 8 * buf, (q >> 1) & 1u, limit_ns);
          ++q;
          if (!__all_sync(~0u, ready)) timed_out = true;
          tc_fence_after();
          if (!timed_out && p.vec_out && !FEW && p.ksplit == 1) {
            const uint32_t at = lanes + buf * S::kBN;
            for (int c0 = 16 * half; c0 < tile.bn; c0 += 32) {
              uint32_t f[2][8];
              __syncwarp();
              tmem_load_matrices(at + c0, f[0]);
              tmem_load_matrices(at + c0 + (16u << 16), f[1]);
              tmem_wait(f[0], f[1]);
              const Tile t = rows_at(c0);
              if (t.qn > c0) store_matrices<MODE>(p, t, c0, nw, f, scale, stage, owner);
            }
          } else if (!timed_out) {
            for (int c0 = 16 * half; c0 < tile.bn; c0 += 32) {
              float v[16];
              __syncwarp();
              tmem_load_16(lanes + buf * S::kBN + c0, v);
              put(c0, v);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_relaxed(tempty + 8 * buf);
        } else {
          // Several tensor-memory sums.  Their sum is kept in local memory (the loops over blocks
          // are not unrolled), as the registers of 128 values a thread are not there: 128 KB a block
          // and sum, on the way that the operands take (8 groups of 8320 rows, 2048 x 2048: 330 us
          // -> 350 us; K = 8320, 4096 rows of 8 groups, N = 2048: 89 us -> 101 us; up to 8192
          // unchanged).
          const bool matrices = p.vec_out && !FEW && p.ksplit == 1;
          const int each = long_sum(nb);
          float acc[kBlocks][16];
          for (int left = nb; left > 0; left -= each, ++q) {
            const uint32_t buf = q & 1;
            const bool ready =
                !timed_out && mbar_wait(bar_tfull + 8 * buf, (q >> 1) & 1u, limit_ns);
            if (!__all_sync(~0u, ready)) timed_out = true;
            if (timed_out) break;
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 16 * half; c0 < tile.bn; c0 += 32) {
              const uint32_t at = lanes + buf * S::kBN + c0;
              float a[16];
              uint32_t f[2][8];
#pragma unroll
              for (int j = 0; j < 16; ++j) a[j] = left == nb ? 0.0f : acc[c0 >> 5][j];
              __syncwarp();
              if (matrices) {
                tmem_load_matrices(at, f[0]);
                tmem_load_matrices(at + (16u << 16), f[1]);
                tmem_wait(f[0], f[1]);
#pragma unroll
                for (int j = 0; j < 16; ++j) a[j] += __uint_as_float(f[j >> 3][j & 7]);
              } else {
                float v[16];
                tmem_load_16(at, v);
#pragma unroll
                for (int j = 0; j < 16; ++j) a[j] += v[j];
              }
              if (left > each) {
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[c0 >> 5][j] = a[j];
              } else if (matrices) {
#pragma unroll
                for (int j = 0; j < 16; ++j) f[j >> 3][j & 7] = __float_as_uint(a[j]);
                const Tile t = rows_at(c0);
                if (t.qn > c0) store_matrices<MODE>(p, t, c0, nw, f, scale, stage, owner);
              } else {
                put(c0, a);
              }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed(tempty + 8 * buf);
          }
        }
      } else {
        float acc[kBlocks][16];
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[b][j] = 0.0f;
        const int chunks = (n + kChunk - 1) / kChunk;
        for (int c = 0; c < chunks && !timed_out; ++c, ++q) {
          const uint32_t buf = q & 1;
          const bool ready = mbar_wait(bar_tfull + 8 * buf, (q >> 1) & 1u, limit_ns);
          if (!__all_sync(~0u, ready)) {
            timed_out = true;
            break;
          }
          tc_fence_after();
          int from = 0, to = tile.bn;      // the columns of this part of the sum
          if (EXT && c * kChunk >= nbase) {
            const int e = tile.e0 + (c * kChunk - nbase) / per_rank;
            const int e1 = tile.e0 + (min(c * kChunk + kChunk, n) - 1 - nbase) / per_rank;
            from = part_of(p, tab, tile, e).c0;
            const Part end = part_of(p, tab, tile, e1);
            to = end.c0 + 32 * end.n32;
          }
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            const int c0 = 32 * b + 16 * half;
            if (c0 >= tile.bn) break;
            __syncwarp();
            if (EXT && (c0 < from || c0 >= to)) continue;
            // The two are added to each other first: the lower parts' sum is small, and rounded alone
            // to steps of the whole sum its errors need not be of either sign.  A leading sum that is
            // not finite stands alone: an infinity's lower parts are zeros, whose products with
            // another are NaN.
#pragma unroll
            for (int j0 = 0; j0 < 16; j0 += 8) {
              uint32_t v[8], low[8];
              tmem_load_8(lanes + buf * S::kBN + c0 + j0, v);
              tmem_load_8(lanes + (2 + buf) * S::kBN + c0 + j0, low);
              tmem_wait(v, low);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float top = __uint_as_float(v[j]);
                acc[b][j0 + j] += isfinite(top) ? top + __uint_as_float(low[j]) : top;
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_relaxed(tempty + 8 * buf);
        }
        if (!timed_out) {
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            const int c0 = 32 * b + 16 * half;
            if (c0 >= tile.bn) break;
            put(c0, acc[b]);
          }
        }
      }
    }
    if (CG == 1 && p.ksplit > 1) {
      // Every block holds its part of the sum in `red`: block c adds the columns of its share,
      // in block order, and stores them.
      __syncwarp();
      cluster_sync();
      if (warp >= S::kEpi0 && warp < S::kMmaWarp) {
        const int c0 = tile.qn * int(rank) / p.ksplit, c1 = tile.qn * int(rank + 1) / p.ksplit;
        const float scale = MODE == kForward && p.scale ? p.scale[tile.g] : 1.0f;
        // Four lanes' values a load and kBatch loads of every block in flight: read one by one
        // they took longer than the slices (4096 x 4096 x 64 shared by two: 17.5 us).
        constexpr int kBatch = 4, kStep = 32 * kEpiWarps;
        const int total = 32 * (c1 - c0);
        for (int i0 = int(threadIdx.x) - 32 * S::kEpi0; i0 < total; i0 += kStep * kBatch) {
          float4 v[kBatch] = {};
#pragma unroll 2
          for (int b = 0; b < p.ksplit; ++b) {
            const uint32_t from = map_rank(red, uint32_t(b)) + uint32_t(c0 * 512);
            float4 w[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
              w[u] = make_float4(0, 0, 0, 0);
              if (i0 + u * kStep < total) w[u] = ld_cluster4(from + uint32_t(i0 + u * kStep) * 16);
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
              v[u].x += w[u].x;
              v[u].y += w[u].y;
              v[u].z += w[u].z;
              v[u].w += w[u].w;
            }
          }
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            const int i = i0 + u * kStep;
            if (i >= total) break;
            const int col = c0 + (i >> 5), n = tile.n0 + (i & 31) * 4;
            int64_t o = out_row<MODE>(p, tile, col);
            if (FEW && owner[tile.q0 + col] == -2) o = -1;
            if (o < 0) continue;
            const float f[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
            if constexpr (MODE == kForward && PLANES == 1) {
              if (p.out_type == kOutU) {
                float g[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) g[j] = n + j < p.N ? f[j] * scale : 0.0f;
                if (n < p.n_out)
                  store_u4(static_cast<uint16_t *>(p.out) + o, n, g, p.idesc & (1u << 7));
                continue;
              }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (n + j < p.n_out) store_out<MODE, PLANES>(p, o, n + j, f[j] * scale);
          }
        }
      }
      __syncwarp();
      cluster_sync();
    }
  }

  if (MODE == kLora) {
    grid_wait();       // no grid ends before the one it follows
    grid_start_next();
  }
  if (warp == S::kMmaWarp && leader) {
    if (elect_one()) mma_commit<CG>(bar_drain, false);
    __syncwarp();
    if (!mbar_wait(bar_drain, 0u, p.wait_limit_ns)) timed_out = true;
  }
  __syncwarp();
  if (timed_out && lane == 0) atomicOr(&g_grouped_status, 2u);
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
  if (warp == S::kMmaWarp) {
    if constexpr (CG == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(S::kTmemCols)
                   : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(S::kTmemCols)
                   : "memory");
  }
}

// ---- operand planes -----------------------------------------------------------------------

// Copies stacks of matrices into 16-bit planes whose rows start on 16-byte boundaries: FP32
// values into their three bf16 parts (planes), 16-bit values as they are (one plane), the FP16 b of
// adapters on pairs into its two bf16 parts: two planes, or (`side`) side by side in a row, 16
// columns each by turns.  Layout:
// [plane][matrix][row][ld8].  With `index` (one matrix only) row r is the source's row index[r],
// zeros for a number outside [0, src_rows).  Matrices of groups without rows are left out.
// One launch makes the planes of all of a call's operands; bound by memory, each thread has
// kPlaneAhead units of eight values in flight.  16384 rows of 4096 bf16 gathered: 40 us, 201 MB at
// 5.0 TB/s (74 % of the measured copy rate).
struct PlaneJob {
  const void *src;
  int64_t rows, cols, ld, stride, src_rows, ld8, plane;   // plane: values between planes
  int64_t count;
  const int *offsets, *index;
  uint16_t *dst;
  int64_t units;        // units of eight values of a row
  int64_t tiles;        // tiles of kPlaneTile units of a matrix
  int vec;              // whole 16-byte loads
  int parts, side;      // 16-bit values: parts of each, and whether they lie side by side
};
struct PlaneJobs {
  PlaneJob job[4];
  int64_t first[5];     // tiles (of all matrices) before each job
  int count;
};
constexpr int kPlaneThreads = 256, kPlaneAhead = 4;
constexpr int kPlaneTile = kPlaneThreads * kPlaneAhead;

// One tile of units; VEC: whole 16-byte loads throughout.
template <bool F32, bool PARTS, bool VEC>
__device__ __forceinline__ void plane_tile(const PlaneJob &j, int64_t m, int64_t unit0) {
  using T = std::conditional_t<F32, float, uint16_t>;
  const int64_t per_row = j.units, total = j.rows * per_row;
  Eight<T> x[kPlaneAhead];
  int64_t to[kPlaneAhead];
#pragma unroll
  for (int k = 0; k < kPlaneAhead; ++k) {
    const int64_t i = unit0 + k * kPlaneThreads;
    const int64_t row = total <= UINT32_MAX ? uint32_t(i) / uint32_t(per_row) : i / per_row;
    const int64_t c = (i - row * per_row) * 8;
    int64_t from = row;
    bool on = i < total && (!PARTS || c < j.cols);
    if (j.index) {
      from = on ? j.index[row] : -1;
      on = from >= 0 && from < j.src_rows;
    }
    to[k] = i < total ? (m * j.rows + row) * j.ld8 +
                          (PARTS && j.side ? (c >> 4) * 32 + (c & 15) : c)
                    : -1;
    x[k] = load8<VEC>(static_cast<const T *>(j.src) + m * j.stride + (on ? from : 0) * j.ld + c, on,
                      j.cols - c);
  }
#pragma unroll
  for (int k = 0; k < kPlaneAhead; ++k) {
    if (to[k] < 0) continue;
    if constexpr (F32) {
      float f[8];
      uint32_t h[3][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = x[k].get(i);
      split8(f, h);
#pragma unroll
      for (int pl = 0; pl < 3; ++pl)
        *reinterpret_cast<uint4 *>(j.dst + pl * j.plane + to[k]) =
            make_uint4(h[pl][0], h[pl][1], h[pl][2], h[pl][3]);
    } else if (PARTS && j.parts == 2) {
      const uint4 v = x[k].w[0];
      const uint32_t two[4] = {v.x, v.y, v.z, v.w};
      uint32_t h[2][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t parts[2];
        half_parts(two[i], parts);
        h[0][i] = parts[0];
        h[1][i] = parts[1];
      }
      uint16_t *const dst = j.dst + to[k];
      *reinterpret_cast<uint4 *>(dst) = make_uint4(h[0][0], h[0][1], h[0][2], h[0][3]);
      *reinterpret_cast<uint4 *>(dst + (j.side ? 16 : j.plane)) =
          make_uint4(h[1][0], h[1][1], h[1][2], h[1][3]);
    } else {
      *reinterpret_cast<uint4 *>(j.dst + to[k]) = x[k].w[0];
    }
  }
}

// PARTS: a job makes parts of 16-bit values.
template <bool F32, bool PARTS>
__global__ void __launch_bounds__(kPlaneThreads)
planes_kernel(const __grid_constant__ PlaneJobs jobs) {
  grid_wait();
  grid_start_next();
  for (int64_t t = blockIdx.x; t < jobs.first[jobs.count]; t += gridDim.x) {
    int n = 0;
    while (t >= jobs.first[n + 1]) ++n;
    const PlaneJob &j = jobs.job[n];
    const int64_t m = (t - jobs.first[n]) / j.tiles;
    if (j.offsets && j.offsets[m + 1] <= j.offsets[m]) continue;
    const int64_t unit0 = (t - jobs.first[n] - m * j.tiles) * kPlaneTile + threadIdx.x;
    if (j.vec) plane_tile<F32, PARTS, true>(j, m, unit0);
    else plane_tile<F32, PARTS, false>(j, m, unit0);
  }
}

// ---- u for few rows ------------------------------------------------------------------------

constexpr int kRowThreads = 512;
constexpr int kRowRanks = 16;            // values of u a block makes

// u[r(p), j] = scale[g] sum_k x[r(p), k] a[g, k, j] for one place p (blockIdx.x) and 16 j
// (blockIdx.y), in FP32.
// For a batch of few rows with an adapter each, a is read once per row and everything else is
// small: the bound is the latency of reading K x 16 values, so one block takes them all at once
// (512 threads, 16 bytes each, K / 256 rounds) instead of a product kernel's ring of slices, and
// rows that share an adapter read it from L2.  FP32 throughout; sums of 512 threads in a fixed
// order.  64 rows of 64 adapters, K = 4096, rank 16, bf16 (8.4 MB): 8.9 us with nothing in L2; w's
// first tiles are on their way meanwhile.
template <typename T, bool TRANS_A, bool VEC>
__global__ void __launch_bounds__(kRowThreads)
row_ranks_kernel(const T *__restrict__ x, int64_t ldx, int64_t x_rows,
                 const int *__restrict__ row_index, const int *__restrict__ offsets, int groups,
                 const T *__restrict__ a, int64_t lda, int64_t stride_a,
                 const float *__restrict__ scale, int K, int rank, float *__restrict__ u,
                 int64_t ldu) {
  grid_wait();
  grid_start_next();
  __shared__ float sums[kRowThreads / 32][kRowRanks];
  const int p = blockIdx.x, j0 = blockIdx.y * kRowRanks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The group of place p: the first whose end is past p (ends never step back, and the first
  // start must not be past p).  Every warp looks for itself.
  const int64_t row = row_index ? row_index[p] : p;
  const int start = offsets[0];
  int g = groups;
  for (int g0 = 0; g0 < groups && g == groups; g0 += 32) {
    const bool past = g0 + lane < groups && offsets[g0 + lane + 1] > p;
    const unsigned any = __ballot_sync(~0u, past);
    if (any) g = g0 + __ffs(any) - 1;
  }
  if (g == groups || start > p || row < 0 || row >= x_rows) return;
  const T *const xr = x + row * ldx;
  const T *const ag = a + int64_t(g) * stride_a;
  const int ranks = min(kRowRanks, rank - j0);
  constexpr int kAhead = VEC ? 8 : 2;      // loads in flight
  if constexpr (TRANS_A) {
    // a stored rank x K: a warp a rank, 256 k a round.
    static_assert(kRowRanks == kRowThreads / 32, "a rank for every warp");
    float sum = 0.0f;
    if (warp < ranks) {
      const T *const aj = ag + int64_t(j0 + warp) * lda;
      for (int k0 = lane * 8; k0 < K; k0 += 256 * kAhead) {
        Eight<T> w[kAhead], v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int k = k0 + 256 * i;
          w[i] = load8<VEC>(aj + k, k < K, K - k);
          v[i] = load8<VEC>(xr + k, k < K, K - k);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (k0 + 256 * i + e < K) sum = fmaf(w[i].get(e), v[i].get(e), sum);
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
    if (lane == 0) sums[0][warp] = sum;
  } else {
    // a stored K x rank: two threads a k, eight ranks each, 256 k a round.
    const int half = threadIdx.x & 1;
    const int left = ranks - 8 * half;
    float sum[8] = {};
    for (int k0 = threadIdx.x >> 1; k0 < K && left > 0; k0 += kRowThreads / 2 * kAhead) {
      Eight<T> w[kAhead];
      float v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int k = k0 + kRowThreads / 2 * i;
        w[i] = load8<VEC>(ag + int64_t(k) * lda + j0 + 8 * half, k < K, left);
        v[i] = k < K ? float(xr[k]) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (k0 + kRowThreads / 2 * i < K)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] = fmaf(w[i].get(e), v[i], sum[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int d = 16; d > 1; d >>= 1) sum[e] += __shfl_xor_sync(~0u, sum[e], d);
      if (lane < 2) sums[warp][8 * lane + e] = sum[e];
    }
  }
  __syncthreads();
  if (int(threadIdx.x) < ranks) {
    float v = 0.0f;
    if constexpr (TRANS_A) {
      v = sums[0][threadIdx.x];
    } else {
#pragma unroll
      for (int w = 0; w < kRowThreads / 32; ++w) v += sums[w][threadIdx.x];
    }
    u[row * ldu + j0 + threadIdx.x] = v * scale[g];
  }
}

// ---- host -------------------------------------------------------------------------------

std::atomic<int64_t> g_wait_limit_ns{int64_t(10) * 1000 * 1000 * 1000};
std::atomic<int> g_drop_block{-1};

// The launch may begin its prologue while the one before it in the stream ends (grid_wait).
cudaLaunchAttribute overlap_attribute() {
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

int64_t round8(int64_t v) { return (v + 7) / 8 * 8; }

// Rows (and matrices) of `size`-byte elements on 16-byte boundaries.
int on16(const Stack &s, int64_t size) {
  return (reinterpret_cast<uintptr_t>(s.data) & 15u) == 0 && s.ld * size % 16 == 0 &&
         (s.count == 1 || s.stride * size % 16 == 0);
}

// Whether the copy engine can read the matrices in place: 16-bit values, rows and matrices on
// 16-byte boundaries.
bool in_place(const Stack &s, int dtype) {
  return dtype != TMM_F32 && on16(s, 2);
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// Bytes of an operand's planes in the workspace (0: read in place), or SIZE_MAX; `gathered`:
// rows fetched through the row index (0: none).
size_t plane_bytes(const Stack &s, int dtype, int64_t gathered = 0) {
  if (in_place(s, dtype) && gathered == 0) return 0;
  const __int128 n = __int128(dtype == TMM_F32 ? 6 : 2) * s.count *
                     (gathered ? gathered : s.rows) * round8(s.cols);
  return n > __int128(INT64_MAX / 4) ? SIZE_MAX : round256(size_t(n));
}

size_t add_sizes(std::initializer_list<size_t> sizes) {
  size_t t = 0;
  for (size_t s : sizes) {
    if (s == SIZE_MAX) return SIZE_MAX;
    t += s;      // each is at most 2^61, and there are at most five
  }
  return t;
}

// An operand as the copy engine reads it: `planes` stacks of 16-bit matrices after each other.
struct Planes {
  const void *data;
  int64_t count, rows, cols, ld, stride;   // count: matrices of all planes
};

// The operand in place, or a job that makes its planes in *ws (which advances past them);
// matrices of groups without rows (by `offsets`, a matrix per group) are not made.  With
// `gathered` the planes hold the rows that `index` names.
Planes plan_planes(const Stack &s, int dtype, const int32_t *offsets, char **ws, PlaneJobs *jobs,
                   int64_t gathered = 0, const int32_t *index = nullptr) {
  if (in_place(s, dtype) && gathered == 0)
    return {s.data, s.count, s.rows, s.cols, s.ld, s.count > 1 ? s.stride : s.rows * s.ld};
  const int planes = dtype == TMM_F32 ? 3 : 1;
  PlaneJob &j = jobs->job[jobs->count];
  j.src = s.data;
  j.rows = gathered ? gathered : s.rows;
  j.cols = s.cols;
  j.ld = s.ld;
  j.stride = s.count > 1 ? s.stride : 0;
  j.src_rows = s.rows;
  j.ld8 = round8(s.cols);
  j.units = j.ld8 / 8;
  j.parts = 1;
  j.count = s.count;
  j.plane = s.count * j.rows * j.ld8;
  j.offsets = s.count > 1 ? offsets : nullptr;      // one matrix may serve every group
  j.index = gathered ? index : nullptr;
  j.dst = reinterpret_cast<uint16_t *>(*ws);
  j.tiles = (j.rows * j.units + kPlaneTile - 1) / kPlaneTile;
  j.vec = on16(s, dtype == TMM_F32 ? 4 : 2) && s.cols % 8 == 0;
  jobs->first[jobs->count + 1] = jobs->first[jobs->count] + j.tiles * j.count;
  ++jobs->count;
  *ws += plane_bytes(s, dtype, gathered);
  return {j.dst, planes * s.count, j.rows, s.cols, j.ld8, j.rows * j.ld8};
}

// The FP16 b of adapters on pairs as two BF16 parts: its product with the BF16 parts of u is one of
// equal types.  Stored rank x N, two planes; stored N x rank, the parts of 16 ranks side by side, so
// that one box of the copy engine brings both.
int64_t side_columns(const Stack &s) { return (s.cols + 15) / 16 * 32; }
size_t part_bytes(const Stack &s, bool side) {
  const __int128 n =
      __int128(2) * s.count * s.rows * (side ? side_columns(s) : 2 * round8(s.cols));
  return n > __int128(INT64_MAX / 4) ? SIZE_MAX : round256(size_t(n));
}
Planes plan_parts(const Stack &s, bool side, const int32_t *offsets, char **ws, PlaneJobs *jobs) {
  PlaneJob &j = jobs->job[jobs->count];
  j.src = s.data;
  j.rows = s.rows;
  j.cols = s.cols;
  j.ld = s.ld;
  j.stride = s.count > 1 ? s.stride : 0;
  j.src_rows = s.rows;
  j.ld8 = side ? side_columns(s) : round8(s.cols);
  j.units = side ? j.ld8 / 16 : j.ld8 / 8;
  j.parts = 2;
  j.side = side;
  j.count = s.count;
  j.plane = s.count * j.rows * j.ld8;
  j.offsets = s.count > 1 ? offsets : nullptr;
  j.index = nullptr;
  j.dst = reinterpret_cast<uint16_t *>(*ws);
  j.tiles = (j.rows * j.units + kPlaneTile - 1) / kPlaneTile;
  j.vec = on16(s, 2) && s.cols % 8 == 0;
  jobs->first[jobs->count + 1] = jobs->first[jobs->count] + j.tiles * j.count;
  ++jobs->count;
  *ws += part_bytes(s, side);
  return {j.dst, side ? s.count : 2 * s.count, j.rows, side ? j.ld8 : s.cols, j.ld8, j.rows * j.ld8};
}

cudaError_t make_planes(const PlaneJobs &jobs, int dtype, const DeviceInfo &dev,
                        cudaStream_t stream) {
  if (jobs.count == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0] = overlap_attribute();
  cfg.gridDim =
      dim3(unsigned(std::min<int64_t>(jobs.first[jobs.count], 8 * dev.sm_count)), 1, 1);
  cfg.blockDim = dim3(kPlaneThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  bool parts = false;
  for (int i = 0; i < jobs.count; ++i) parts |= jobs.job[i].parts == 2;
  return cudaLaunchKernelEx(&cfg,
                            dtype == TMM_F32 ? planes_kernel<true, false>
                            : parts          ? planes_kernel<false, true>
                                             : planes_kernel<false, false>,
                            jobs);
}

// Maps of an operand: tiles of `box_rows` rows x 64 values in matrix z, or of the rows of all
// matrices under one another (which are contiguous or only one), singly with box_rows = 1.
cudaError_t tile_map(CUtensorMap *map, const Planes &o, uint32_t box_rows) {
  const uint64_t size[3] = {uint64_t(o.cols), uint64_t(o.rows), uint64_t(o.count)};
  const uint64_t stride[2] = {uint64_t(o.ld), uint64_t(o.stride)};
  const uint32_t box[3] = {kBK, box_rows, 1};
  return encode_16bit(map, o.data, 3, size, stride, box);
}
cudaError_t row_map(CUtensorMap *map, const Planes &o, uint32_t box_rows) {
  const uint64_t size[2] = {uint64_t(o.cols), uint64_t(o.rows) * uint64_t(o.count)};
  const uint64_t stride[1] = {uint64_t(o.ld)};
  const uint32_t box[2] = {kBK, box_rows};
  return encode_16bit(map, o.data, 2, size, stride, box);
}

struct Maps {
  CUtensorMap p, q, qr, e, u, pr;
};

template <int CG, int MODE, int PLANES, int BP = 1>
cudaError_t launch_shape(const Maps &m, Params &prm, int64_t tiles, const DeviceInfo &dev,
                         cudaStream_t stream) {
  using S = Shape<CG, PLANES>;
  static std::atomic<uint64_t> configured{0};
  auto kernel = grouped_kernel<CG, MODE, PLANES, BP>;
  const uint64_t bit = uint64_t(1) << (dev.id & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(S::kSmem));
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_release);
  }
  const int cluster = CG == 2 ? 2 : prm.ksplit;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[1] = overlap_attribute();
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.blockDim = dim3(S::kThreads, 1, 1);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = stream;
  // Persistent: a cluster for every tile there can be, at most one per resident slot.
  const int64_t slots = std::max(1, dev.sm_count / cluster);
  cfg.gridDim = dim3(unsigned(cluster * std::max<int64_t>(1, std::min(tiles, slots))), 1, 1);
  return cudaLaunchKernelEx(&cfg, kernel, m.p, m.q, m.qr, m.e, m.u, m.pr, prm);
}

template <int CG, int PLANES>
cudaError_t launch_mode(int mode, const Maps &m, Params &prm, int64_t tiles,
                        const DeviceInfo &dev, cudaStream_t stream) {
  if (mode == kForward) return launch_shape<CG, kForward, PLANES>(m, prm, tiles, dev, stream);
  if (mode == kWgrad) return launch_shape<CG, kWgrad, PLANES>(m, prm, tiles, dev, stream);
  if constexpr (CG == 2 && PLANES == 1)
    if (prm.out_type == kOutF16) return launch_shape<2, kLora, 1, 2>(m, prm, tiles, dev, stream);
  return launch_shape<CG, kLora, PLANES>(m, prm, tiles, dev, stream);
}

cudaError_t launch_any(int cg, int planes, int mode, const Maps &m, Params &prm, int64_t tiles,
                       const DeviceInfo &dev, cudaStream_t stream) {
  prm.wait_limit_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  prm.drop_block = g_drop_block.load(std::memory_order_relaxed);
  prm.vec_out = (prm.out_type == kOutBF16 || prm.out_type == kOutF16) &&
                (reinterpret_cast<uintptr_t>(prm.out) & 15u) == 0 && prm.ld_out % 8 == 0 &&
                prm.stride_out % 8 == 0;
  if (cg == 2)
    return planes == 3 ? launch_mode<2, 3>(mode, m, prm, tiles, dev, stream)
                       : launch_mode<2, 1>(mode, m, prm, tiles, dev, stream);
  return planes == 3 ? launch_mode<1, 3>(mode, m, prm, tiles, dev, stream)
                     : launch_mode<1, 1>(mode, m, prm, tiles, dev, stream);
}

// Instruction descriptor of kind::f16 without majors and sizes: D FP32 (bit 4), A and B bf16
// (1 in bits 7-9 and 10-12) or FP16 (0).
uint32_t type_desc(int dtype) {
  return (1u << 4) | (dtype == TMM_F16 ? 0u : (1u << 7) | (1u << 10));
}
int out_type(int dtype) {
  return dtype == TMM_F32 ? kOutF32 : dtype == TMM_BF16 ? kOutBF16 : kOutF16;
}
int box_of(int cg) { return cg == 2 ? 32 : 16; }
int columns_of(int cg, int planes) { return cg == 1 ? 64 : planes == 3 ? 128 : 256; }

// A GB300's SMs and pairs of them: the rules that give workspace sizes are asked without a device.
constexpr int64_t kSms = 152, kPairs = kSms / 2;

// Blocks that share a tile's sum: the largest power of two up to eight that leaves every block
// enough slices to pay for meeting, about 3 us, and needs no more blocks than there are SMs (where a
// GPC's SMs are not a multiple of the cluster some of them wait, which is slower, not wrong).  16
// slices of 16-bit operands take about that long (K = 512 in two groups of 32 rows, N = 320: 9.7 us
// shared by two, 6.6 us not), four of split ones (64 rows of K = 1000, N = 2047 with adapters: 48 us
// not shared, 27 us by four).
int split_slices(int planes) { return planes == 3 ? 4 : 16; }
int split_of(int64_t tiles, int64_t slices, int planes, const DeviceInfo &dev) {
  int s = 1;
  while (s < 8 && tiles * (2 * s) <= dev.sm_count && slices >= split_slices(planes) * (2 * s))
    s *= 2;
  return s;
}

// Columns of a pair's tile: the fewest of which one round of tiles is enough, so that few tiles
// spread over more pairs and every slice is copied sooner; else the widest.  `most` bounds the tiles
// of a width.  (4096 x 4096, 257 rows of 4 adapters, rank 16: 128 columns 31.7 us, 256 34.2 us; one
// group of 300 rows 24.3 us and 27.8 us; FP32, 2 groups of 300 rows, 2048 x 1024: 64 columns 32 us,
// 128 42 us.  Two rounds of narrow tiles are slower: 2048 rows of 16 adapters at N = 1024, 128
// columns 51 us, 256 40 us.)
template <typename Tiles>
int pair_columns(int planes, Tiles most) {
  const int widest = columns_of(2, planes);
  for (int n = 64; n < widest; n *= 2)
    if (most(n) <= kPairs) return n;
  return widest;
}

// Pairs or single blocks for a forward product, by an estimate of its cycles for groups of equal
// size: rounds of tiles times what a K slice of 64 takes in one.  16-bit: products at 8192
// multiply-adds a cycle and SM, copies at 64 bytes.  FP32: six products of three planes on pairs,
// after making the planes (10 bytes a value at 23 bytes a cycle and SM, and a launch); on single
// blocks, the measured 2600 + 8 cycles a column of splitting on the way.  (FP32, K = 2048,
// N = 4096: 1024 rows in 64 groups 706 us on single blocks, 1177 us by planes; 2048 rows in 8
// groups 406 us and 275 us.)
int forward_shape(int64_t rows, int64_t groups, int64_t N, int64_t K, int dtype) {
  if (N <= 128) return 1;      // 256 lanes would be half empty
  const bool f32 = dtype == TMM_F32;
  const int64_t live = std::max<int64_t>(1, std::min(groups, rows));
  const int64_t each = (rows + live - 1) / live, slices = (K + kBK - 1) / kBK;
  const auto cost = [&](int cg, int64_t widest, int64_t unit) {      // double: no size overflows it
    const int64_t across = (each + widest - 1) / widest;
    const int64_t cols = ((each + across - 1) / across + unit - 1) / unit * unit;
    const int64_t tiles = live * across * ((N + 128 * cg - 1) / (128 * cg));
    const double slice = cg == 1 ? (f32 ? 2600 + 8 * cols : 256 + 2 * cols)
                                 : (f32 ? std::max(12 * cols, 768 + 3 * cols)
                                        : std::max(2 * cols, 256 + cols));
    const double before =
        f32 && cg == 2 ? 4000 + 10 * (double(live) * N + rows) * K / (23 * kSms) : 0;
    // Fewer tiles than blocks: single blocks split a long sum.
    if (cg == 1 && 2 * tiles <= kSms && slices >= 2 * split_slices(f32 ? 3 : 1))
      return slices * slice * (double(tiles) / kSms + 0.125);
    return before + slices * slice * double((tiles + kSms / cg - 1) / (kSms / cg));
  };
  return cost(2, f32 ? 128 : 256, 64) <= cost(1, 64, 16) ? 2 : 1;
}
// Adapters: single blocks while the part on the CUDA cores (rows x rank) is small and their tiles
// are few, or pairs would need more than one round of tiles, an adapter's rows taking about 24
// columns more than they are.  (K = 4096, BF16, rank 16, on single blocks and on pairs: 257 rows of
// 4 adapters 22 us and 34 us at N = 1024, 45 us and 35 us at N = 4096; of 32 adapters 46 us and 59
// us at N = 4096; 512 rows of 32 adapters 55 us and 61 us.  FP32, K = 2048: 128 rows of 7 adapters
// 43 us and 55 us, 256 rows of 4 75 us and 56 us, of 32 73 us and 109 us, all at N = 4096; sizes
// that do not allow vector loads, K = 1000 and N = 2047: 128 rows 29 us and 32 us, 200 rows 48 us
// and 34 us.)
int lora_shape(const LoraProblem &p) {
  if (p.rows <= 64) return 1;
  if (p.rows > kFewRows || p.rows * p.rank > 8192) return 2;
  const bool f32 = p.dtype == TMM_F32;
  const int64_t tiles = (p.rows + 63) / 64 * ((p.N + 127) / 128);
  if (tiles <= (!f32 ? kSms : p.K % 8 == 0 && p.N % 8 == 0 ? kSms / 2 : kSms / 4)) return 1;
  if (f32 && p.rows > 256) return 2;
  const int64_t width = f32 ? 128 : 256, columns = p.rows + 24 * std::min(p.groups, p.rows);
  return (columns + width - 1) / width * ((p.N + 255) / 256) > kPairs ? 1 : 2;
}
// Gradient: pairs where results fill more than 128 lanes, whatever the rows.  (Single blocks and pairs,
// groups x rows and K x N: BF16 8 x 1024, 4096 x 136 41 us and 19 us, 4096 x 320 53 us and 28 us; 32 x
// 64, 2048 x 192 20 us and 15 us, 2048 x 515 83 us and 52 us; 64 x 16, 1024 x 256 21 us and 15 us; FP32
// the same 212 us and 128 us, 313 us and 164 us, 49 us and 40 us, 134 us and 88 us, 49 us and 33 us.  At
// N = 128, where half of a pair's lanes are empty, few rows a group are faster on single blocks: 32 x
// 64, 2048 12.0 us and 14.7 us, FP32 27 us and 35 us; and many are not: 8 x 1024, 4096 22 us and 17
// us, FP32 131 us and 122 us.)
int wgrad_shape(int64_t N) { return N > 128 ? 2 : 1; }

// The maps of x: rows by number; or tiles of box_of rows, and (pairs) of a whole block's columns.
cudaError_t q_maps(Maps *m, const Planes &x, const int32_t *index, int cg, int bn) {
  cudaError_t e;
  if (index) {
    e = row_map(&m->qr, x, 1);
    m->q = m->qr;
    return e;
  }
  if ((e = row_map(&m->q, x, uint32_t(box_of(cg)))) != cudaSuccess) return e;
  if (cg == 2) return row_map(&m->qr, x, uint32_t(bn / 2));
  m->qr = m->q;
  return cudaSuccess;
}

// FP32 operands read as they are stored (single blocks; see split_tile).
bool direct(int cg, int dtype) { return cg == 1 && dtype == TMM_F32; }
void set_direct(Params *prm, const Stack &P, const Stack &x) {
  prm->fp = static_cast<const float *>(P.data);
  prm->ldp = P.ld;
  prm->stride_p = P.stride;
  prm->fx = static_cast<const float *>(x.data);
  prm->ldx = x.ld;
  prm->vec = on16(P, 4) && on16(x, 4) && P.cols % 8 == 0 && x.cols % 8 == 0;
}

// Forward product: on the planes (x, w) of the stacks (xs, ws), or on FP32 stacks directly;
// `index`: the rows of x by number, or NULL.
cudaError_t run_forward(int dtype, const Planes &x, const Stack &xs, const int32_t *index,
                        const Planes &w, const Stack &ws, bool trans_w, Params prm,
                        const DeviceInfo &dev, cudaStream_t stream) {
  const int planes = dtype == TMM_F32 ? 3 : 1;
  const int cg = forward_shape(prm.rows, prm.groups, prm.N, prm.K, dtype);
  prm.panels = int((prm.N + 128 * cg - 1) / (128 * cg));
  const auto most = [&](int n) {
    return prm.panels * (std::min<int64_t>(prm.groups, prm.rows) + prm.rows / n);
  };
  const int bn = cg == 1 ? columns_of(cg, planes) : pair_columns(planes, most);
  prm.tile_n = bn;
  const int64_t tiles = most(bn);
  if (tiles > INT32_MAX / 2) return cudaErrorInvalidConfiguration;
  prm.ksplit = cg == 2 ? 1 : split_of(tiles, (prm.K + kBK - 1) / kBK, planes, dev);
  if (prm.n_out == 0) prm.n_out = prm.N;
  prm.row_index = index;
  prm.p_mn = trans_w ? 0 : 1;
  prm.p_shared = prm.groups > 1 && ws.count == 1;
  Maps m = {};
  if (direct(cg, dtype)) {
    prm.q_rows = int(xs.rows);
    set_direct(&prm, ws, xs);
  } else {
    prm.q_rows = int(x.rows);
    cudaError_t e;
    if ((e = tile_map(&m.p, w, trans_w ? 128 : 64)) != cudaSuccess ||
        (e = q_maps(&m, x, index, cg, bn)) != cudaSuccess)
      return e;
    m.e = m.p;
    m.u = m.q;
  }
  return launch_any(cg, planes, kForward, m, prm, tiles, dev, stream);
}

}  // namespace

// Rows that are gathered by a kernel before a product (0: none): for pairs all, for single blocks
// `many`, where the copies by number of a slice would take longer.  FP32 on single blocks reads rows
// by number as cheaply as others.
static int64_t gathered_rows(int cg, int dtype, const int32_t *row_index, int64_t rows, bool many) {
  return row_index && !direct(cg, dtype) && (cg == 2 || many) ? rows : 0;
}
// Groups of more than 32 rows (of equal size), long sums.  (Single blocks, 4096 x 4096, bf16, one
// group, by number and gathered: 33 rows 12.4 us and 12.8 us, 64 rows 21.4 us and 16.5 us, 200 rows
// 34 us and 24 us; 64 rows of K = 1024 10.8 us both.)
static int64_t grouped_gathered(const GroupedProblem &p, int cg) {
  return gathered_rows(cg, p.dtype, p.row_index, p.rows, p.rows > 32 * p.groups && p.K > 1024);
}

static int shape_of(const GroupedProblem &p) {
  return forward_shape(p.rows, p.groups, p.N, p.K, p.dtype);
}

size_t grouped_workspace_bytes(const GroupedProblem &p) {
  const int cg = shape_of(p);
  if (direct(cg, p.dtype)) return 0;
  return add_sizes({plane_bytes(p.x, p.dtype, grouped_gathered(p, cg)),
                    plane_bytes(p.w, p.dtype)});
}

cudaError_t launch_grouped(const GroupedProblem &p, const DeviceInfo &dev, void *workspace,
                           cudaStream_t stream) {
  char *ws = static_cast<char *>(workspace);
  const int cg = shape_of(p);
  const int64_t gathered = grouped_gathered(p, cg);
  Planes x = {}, w = {};
  if (!direct(cg, p.dtype)) {
    PlaneJobs jobs = {};
    x = plan_planes(p.x, p.dtype, nullptr, &ws, &jobs, gathered, p.row_index);
    w = plan_planes(p.w, p.dtype, p.offsets, &ws, &jobs);
    const cudaError_t e = make_planes(jobs, p.dtype, dev, stream);
    if (e != cudaSuccess) return e;
  }
  Params prm = {};
  prm.rows = int(p.rows);
  prm.groups = int(p.groups);
  prm.offsets = p.offsets;
  prm.K = int(p.K);
  prm.N = int(p.N);
  prm.idesc = type_desc(p.dtype);
  prm.out = p.y;
  prm.ld_out = p.ldy;
  prm.out_type = out_type(p.dtype);
  prm.zero_rows = 1;
  return run_forward(p.dtype, x, p.x, gathered ? nullptr : p.row_index, w, p.w, p.trans_w != 0,
                     prm, dev, stream);
}

// Every 64 columns of x read the group's rows again.  (Single blocks, 4096 x 128, bf16, by number and
// gathered: 128 rows of a group 6.6 us and 7.7 us, 512 of each of 8 44 us and 30 us.)
static int64_t wgrad_gathered(const WgradProblem &p) {
  return gathered_rows(wgrad_shape(p.N), p.dtype, p.row_index, p.rows, p.rows > 128 * p.groups);
}

size_t wgrad_workspace_bytes(const WgradProblem &p) {
  if (direct(wgrad_shape(p.N), p.dtype)) return 0;
  return add_sizes(
      {plane_bytes(p.x, p.dtype, wgrad_gathered(p)),
       plane_bytes(p.dy, p.dtype)});
}

cudaError_t launch_wgrad(const WgradProblem &p, const DeviceInfo &dev, void *workspace,
                         cudaStream_t stream) {
  char *ws = static_cast<char *>(workspace);
  const int cg = wgrad_shape(p.N);
  const int64_t gathered = wgrad_gathered(p);
  const int32_t *index = gathered ? nullptr : p.row_index;
  Planes x = {}, dy = {};
  cudaError_t e;
  if (!direct(cg, p.dtype)) {
    PlaneJobs jobs = {};
    x = plan_planes(p.x, p.dtype, nullptr, &ws, &jobs, gathered, p.row_index);
    dy = plan_planes(p.dy, p.dtype, nullptr, &ws, &jobs);
    if ((e = make_planes(jobs, p.dtype, dev, stream)) != cudaSuccess) return e;
  }
  const int planes = p.dtype == TMM_F32 ? 3 : 1;
  Params prm = {};
  prm.rows = int(p.rows);
  prm.groups = int(p.groups);
  prm.offsets = p.offsets;
  prm.row_index = index;
  prm.q_rows = int(gathered ? p.rows : p.x.rows);
  prm.q_cols = int(p.K);
  prm.N = int(p.N);
  prm.idesc = type_desc(p.dtype);
  prm.out = p.dw;
  prm.ld_out = p.lddw;
  prm.stride_out = p.groups > 1 ? p.stride_dw : 0;
  prm.out_type = out_type(p.dtype);
  prm.n_out = prm.N;
  prm.ksplit = 1;
  const int bn = columns_of(cg, planes);
  prm.tile_n = bn;
  prm.panels = int((p.N + 128 * cg - 1) / (128 * cg));
  const int64_t tiles = p.groups * prm.panels * ((p.K + bn - 1) / bn);
  if (tiles > INT32_MAX / 2) return cudaErrorInvalidConfiguration;
  if (cg == 1) prm.ksplit = split_of(tiles, (p.rows / p.groups + kBK - 1) / kBK, planes, dev);
  Maps m = {};
  if (direct(cg, p.dtype)) {
    set_direct(&prm, p.dy, p.x);
  } else {
    if ((e = row_map(&m.p, dy, kBK)) != cudaSuccess ||
        (e = row_map(&m.e, dy, 16)) != cudaSuccess || (e = row_map(&m.pr, dy, 1)) != cudaSuccess ||
        (e = row_map(&m.qr, x, 1)) != cudaSuccess)
      return e;
    m.q = m.u = m.qr;
    if (!index && ((e = row_map(&m.q, x, kBK)) != cudaSuccess ||
                   (e = row_map(&m.u, x, 16)) != cudaSuccess))
      return e;
  }
  return launch_any(cg, planes, kWgrad, m, prm, tiles, dev, stream);
}

template <typename T, bool TRANS_A>
static cudaError_t launch_row_ranks_as(const LoraProblem &p, float *u, int64_t ldu,
                                       cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0] = overlap_attribute();
  cfg.gridDim = dim3(unsigned(p.rows), unsigned((p.rank + kRowRanks - 1) / kRowRanks), 1);
  cfg.blockDim = dim3(kRowThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Whole vectors: rows on 16-byte boundaries, and eight values at a time end with the rows.
  const bool vec = on16(p.a, sizeof(T)) && (!TRANS_A || on16(p.x, sizeof(T))) && p.a.cols % 8 == 0;
  return cudaLaunchKernelEx(&cfg,
                            vec ? row_ranks_kernel<T, TRANS_A, true>
                                : row_ranks_kernel<T, TRANS_A, false>,
                            static_cast<const T *>(p.x.data), p.x.ld, p.x.rows,
                            static_cast<const int *>(p.row_index),
                            static_cast<const int *>(p.offsets), int(p.groups),
                            static_cast<const T *>(p.a.data), p.a.ld,
                            p.a.count > 1 ? p.a.stride : int64_t(0), p.scale, int(p.K),
                            int(p.rank), u, ldu);
}

static cudaError_t launch_row_ranks(const LoraProblem &p, float *u, int64_t ldu,
                                    cudaStream_t stream) {
  if (p.dtype == TMM_F32)
    return p.trans_a ? launch_row_ranks_as<float, true>(p, u, ldu, stream)
                     : launch_row_ranks_as<float, false>(p, u, ldu, stream);
  if (p.dtype == TMM_BF16)
    return p.trans_a ? launch_row_ranks_as<__nv_bfloat16, true>(p, u, ldu, stream)
                     : launch_row_ranks_as<__nv_bfloat16, false>(p, u, ldu, stream);
  return p.trans_a ? launch_row_ranks_as<__half, true>(p, u, ldu, stream)
                   : launch_row_ranks_as<__half, false>(p, u, ldu, stream);
}

// Columns of u: FP32 values on single blocks; for pairs a plane's 16-byte rows, or the parts of 32
// values (BF16) or 16 (FP16) in blocks of 64.
static int rank_slice_of(int dtype) {
  return rank_slice(dtype == TMM_F32 ? 3 : 1, dtype == TMM_F16 ? 2 : 1);
}
static int64_t u_columns(const LoraProblem &p) {
  if (p.dtype == TMM_F32 || lora_shape(p) == 1) return round8(p.rank);
  return (p.rank + rank_slice_of(p.dtype) - 1) / rank_slice_of(p.dtype) * 64;
}
static size_t u_bytes(const LoraProblem &p) {
  const int size = lora_shape(p) == 1 ? 4 : p.dtype == TMM_F32 ? 6 : 2;
  return round256(size_t(p.rows) * size_t(u_columns(p)) * size);   // below 2^29 * 2^12 * 6
}

// How the product with a is computed on pairs: a forward product of its own.
static int low_shape(const LoraProblem &p) {
  return forward_shape(p.rows, p.groups, p.rank, p.K, p.dtype);
}

// The workspace holds u and the planes of the operands.
size_t lora_workspace_bytes(const LoraProblem &p) {
  if (lora_shape(p) == 1)
    return p.dtype == TMM_F32 ? u_bytes(p)
                              : add_sizes({u_bytes(p), plane_bytes(p.x, p.dtype),
                                           plane_bytes(p.w, p.dtype),
                                           plane_bytes(p.b, p.dtype)});
  return add_sizes({u_bytes(p),
                    plane_bytes(p.x, p.dtype, p.row_index ? p.rows : 0),
                    plane_bytes(p.w, p.dtype),
                    direct(low_shape(p), p.dtype) ? 0 : plane_bytes(p.a, p.dtype),
                    p.dtype == TMM_F16 ? part_bytes(p.b, p.trans_b != 0)
                                       : plane_bytes(p.b, p.dtype)});
}

cudaError_t launch_lora(const LoraProblem &p, const DeviceInfo &dev, void *workspace,
                        cudaStream_t stream) {
  char *ws = static_cast<char *>(workspace);
  const int planes = p.dtype == TMM_F32 ? 3 : 1;
  const int cg = lora_shape(p);
  const int64_t ldu = u_columns(p);
  void *u = ws;
  ws += u_bytes(p);
  const int64_t gathered = cg == 2 && p.row_index ? p.rows : 0;
  const bool low_direct = direct(low_shape(p), p.dtype);
  Planes x = {}, w = {}, a = {}, b = {};
  cudaError_t e;
  if (!direct(cg, p.dtype)) {
    PlaneJobs jobs = {};
    x = plan_planes(p.x, p.dtype, nullptr, &ws, &jobs, gathered, p.row_index);
    w = plan_planes(p.w, p.dtype, nullptr, &ws, &jobs);
    if (!low_direct && cg == 2) a = plan_planes(p.a, p.dtype, p.offsets, &ws, &jobs);
    b = cg == 2 && p.dtype == TMM_F16
            ? plan_parts(p.b, p.trans_b != 0, p.offsets, &ws, &jobs)
            : plan_planes(p.b, p.dtype, p.offsets, &ws, &jobs);
    if ((e = make_planes(jobs, p.dtype, dev, stream)) != cudaSuccess) return e;
  }
  Params prm = {};
  prm.rows = int(p.rows);
  prm.groups = int(p.groups);
  prm.offsets = p.offsets;
  prm.K = int(p.K);
  prm.rank = int(p.rank);
  prm.idesc = type_desc(p.dtype);
  Maps m = {};
  if (cg == 1) {
    if ((e = launch_row_ranks(p, static_cast<float *>(u), ldu, stream)) != cudaSuccess) return e;
    prm.row_index = p.row_index;
    prm.u = static_cast<const float *>(u);
    prm.ldu = ldu;
    // b off 16-byte boundaries is copied beside w, 16-bit types (3 rows, K = 896, N = 205, rank 100:
    // 52 us read as it is, 18 us copied); the copies' rows are whole vectors.
    const bool as_is = direct(cg, p.dtype) || b.data == p.b.data;
    prm.b = as_is ? p.b.data : b.data;
    prm.ldb = as_is ? p.b.ld : b.ld;
    prm.stride_b = p.b.count == 1 ? 0 : as_is ? p.b.stride : b.stride;
    prm.trans_b = p.trans_b;
    prm.vec_b = !as_is || (on16(p.b, p.dtype == TMM_F32 ? 4 : 2) && p.b.cols % 8 == 0);
  } else {
    Params up = prm;
    up.N = int(p.rank);
    up.out = u;
    up.ld_out = ldu;
    up.stride_out = p.rows * ldu;
    up.out_type = kOutU;
    up.n_out = int(p.dtype == TMM_F32 ? p.rank : ldu / 64 * rank_slice_of(p.dtype));
    up.scale = p.scale;
    const int32_t *index = gathered && !low_direct ? nullptr : p.row_index;
    if ((e = run_forward(p.dtype, x, p.x, index, a, p.a, p.trans_a != 0, up, dev, stream)) !=
        cudaSuccess)
      return e;
    prm.out_index = p.row_index;
    prm.out_rows = int(p.rows);
    prm.e_mn = p.trans_b ? 0 : 1;
    prm.e_shared = p.groups > 1 && p.b.count == 1;
    prm.idesc_e = type_desc(TMM_BF16);
    const Planes um = {u, planes, p.rows, planes == 3 ? p.rank : ldu, ldu, p.rows * ldu};
    if ((e = tile_map(&m.e, b, p.trans_b ? 128 : uint32_t(rank_slice_of(p.dtype)))) != cudaSuccess ||
        (e = row_map(&m.u, um, uint32_t(box_of(cg)))) != cudaSuccess)
      return e;
  }
  prm.N = prm.n_out = int(p.N);
  prm.q_rows = int(p.rows);
  prm.panels = int((p.N + 128 * cg - 1) / (128 * cg));
  // Pairs: columns at most, every adapter's rounded up to 32.
  const int64_t columns = cg == 1 ? p.rows : p.rows + 31 * (std::min(p.groups, p.rows) + 2);
  const auto most = [&](int n) { return prm.panels * ((columns + n - 1) / n); };
  const int bn = cg == 1 ? columns_of(cg, planes) : pair_columns(planes, most);
  prm.tile_n = bn;
  const int64_t tiles = most(bn);
  if (tiles > INT32_MAX / 2 || columns > INT32_MAX - bn || (cg == 2 && p.rows * planes > INT32_MAX))
    return cudaErrorInvalidConfiguration;
  prm.ksplit = cg == 2 ? 1 : split_of(tiles, (p.K + kBK - 1) / kBK, planes, dev);
  prm.p_mn = p.trans_w ? 0 : 1;
  prm.p_shared = 1;
  prm.out = p.y;
  prm.ld_out = p.ldy;
  prm.out_type = out_type(p.dtype);
  if (direct(cg, p.dtype)) {
    set_direct(&prm, p.w, p.x);
  } else {
    if ((e = tile_map(&m.p, w, p.trans_w ? 128 : 64)) != cudaSuccess ||
        (e = q_maps(&m, x, nullptr, cg, bn)) != cudaSuccess)
      return e;
    if (cg == 1) m.e = m.u = m.p;
  }
  return launch_any(cg, planes, kLora, m, prm, tiles, dev, stream);
}

cudaError_t grouped_device_status(unsigned int *status, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(status, g_grouped_status, sizeof(unsigned int));
  if (e != cudaSuccess || !clear) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_grouped_status, &zero, sizeof(unsigned int));
}

void grouped_set_test_hooks(int drop_block, int64_t wait_limit_ns) {
  g_drop_block.store(drop_block, std::memory_order_relaxed);
  g_wait_limit_ns.store(wait_limit_ns > 0 ? wait_limit_ns : int64_t(10) * 1000 * 1000 * 1000,
                        std::memory_order_relaxed);
}

}  // namespace tmm
