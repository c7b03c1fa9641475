// group_rows.cu -- stable grouping of rows by a number each carries (its expert, its adapter).
//
// A counting sort: with H[g] the count of group g and h[b][g] that of block b's slots,
//     place(s) = sum_{g' < g} H[g'] + sum_{b' < b} h[b'][g] + rank of s among block b's slots
// of its group g; slots of no group are group G.  The rank is made of the counts of the warps
// before (each warp owns a contiguous run of the block's slots) and of the lanes before it in
// the warp that hold the same number, so equal numbers keep their order and no atomic decides
// a place.
//
// The work is 4 bytes read and 12 written a slot, below a microsecond of memory time in any
// real batch: launches and dependent loads are the cost.  Up to kOneBlock slots one block does
// everything in one launch; more take two (counts per block, then places), each block adding up
// the counts of all blocks for itself.  Measured: 74 slots of 8 groups 2.1 us, 131072 slots of 256
// groups 14.4 us (a quarter of it the two launches, the rest the passes over shared memory).
#include <atomic>
#include <cstdint>

#include "grouped.h"

namespace tmm {
namespace {

constexpr int kMaxWarps = 32;
constexpr int64_t kOneBlock = 2048;     // slots that one block handles alone
constexpr int64_t kChunk = 1024;        // slots of a block, at least, otherwise

template <typename T>
__device__ __forceinline__ int key_of(const void *index, int64_t s, int groups) {
  const T v = static_cast<const T *>(index)[s];
  return v >= 0 && v < groups ? int(v) : groups;
}

// Programmatic dependent launch: wait for the launch before, then let the next one start.
__device__ __forceinline__ void grid_wait() {
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}

// h[b][g] for g <= groups.
template <typename T>
__global__ void __launch_bounds__(1024)
count_kernel(const void *__restrict__ index, int64_t slots, int64_t chunk, int groups,
             int *__restrict__ counts) {
  __shared__ int h[kMaxGroups + 1];
  grid_wait();
  for (int g = threadIdx.x; g <= groups; g += blockDim.x) h[g] = 0;
  __syncthreads();
  const int64_t s0 = blockIdx.x * chunk, s1 = min(s0 + chunk, slots);
  for (int64_t s = s0 + threadIdx.x; s < s1; s += blockDim.x)
    atomicAdd(&h[key_of<T>(index, s, groups)], 1);
  __syncthreads();
  for (int g = threadIdx.x; g <= groups; g += blockDim.x)
    counts[int64_t(blockIdx.x) * (groups + 1) + g] = h[g];
}

// Places of block b's slots.  Shared memory: the totals of all blocks and of the blocks before
// (groups + 1 each), then a count per warp and group.
template <typename T>
__global__ void __launch_bounds__(1024)
place_kernel(const void *__restrict__ index, int64_t slots, int64_t chunk, int fan, int groups,
             const int *__restrict__ counts, int *__restrict__ offsets, int *__restrict__ order,
             int *__restrict__ rows, int *__restrict__ position) {
  extern __shared__ int sh[];
  const int G = groups + 1;
  int *const total = sh, *const before = sh + G, *const mine = sh + 2 * G;
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t s0 = blockIdx.x * chunk, s1 = min(s0 + chunk, slots);
  const int64_t run = ((s1 - s0 + warps - 1) / warps + 31) / 32 * 32;   // slots of a warp
  const int64_t w0 = min(s0 + warp * run, s1), w1 = min(w0 + run, s1);
  for (int i = threadIdx.x; i < G * (warps + 2); i += blockDim.x) sh[i] = 0;
  grid_wait();
  __syncthreads();
  for (int64_t s = w0 + lane; s < w1; s += 32)
    atomicAdd(&mine[warp * G + key_of<T>(index, s, groups)], 1);
  if (counts) {
    // Several threads per group, each adding up every `step`-th block's count.
    const int step = max(1, int(blockDim.x) / G);
    for (int i = threadIdx.x; i < G * step; i += blockDim.x) {
      const int g = i % G;
      int all = 0, low = 0;
#pragma unroll 8
      for (int b = i / G; b < int(gridDim.x); b += step) {
        const int c = counts[int64_t(b) * G + g];
        all += c;
        low += b < int(blockIdx.x) ? c : 0;
      }
      atomicAdd(&total[g], all);
      atomicAdd(&before[g], low);
    }
  }
  __syncthreads();
  // Per group: counts of the warps become sums of the warps before.
  for (int g = threadIdx.x; g < G; g += blockDim.x) {
    int sum = 0;
    for (int w = 0; w < warps; ++w) {
      const int c = mine[w * G + g];
      mine[w * G + g] = sum;
      sum += c;
    }
    if (!counts) total[g] = sum;
  }
  __syncthreads();
  // First place of every group: an exclusive sum of the totals, by the first warp.
  if (warp == 0) {
    int carry = 0;
    for (int g0 = 0; g0 < G; g0 += 32) {
      const int g = g0 + lane;
      const int c = g < G ? total[g] : 0;
      int sum = c;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(~0u, sum, d);
        if (lane >= d) sum += o;
      }
      if (g < G) {
        total[g] = carry + sum - c;
        if (blockIdx.x == 0) offsets[g] = carry + sum - c;
      }
      carry += __shfl_sync(~0u, sum, 31);
    }
  }
  __syncthreads();
  for (int64_t b = w0; b < w1; b += 32) {
    const int64_t s = b + lane;
    const int g = s < w1 ? key_of<T>(index, s, groups) : -1;
    const unsigned same = __match_any_sync(~0u, g);
    const int ahead = __popc(same & ((1u << lane) - 1));
    int place = 0;
    if (g >= 0) place = total[g] + before[g] + mine[warp * G + g] + ahead;
    __syncwarp();
    if (g >= 0) {
      if (ahead == 0) mine[warp * G + g] += __popc(same);
      order[place] = int(s);
      if (rows) rows[place] = int(s / fan);
      position[s] = place;
    }
    __syncwarp();
  }
}

int64_t blocks_of(int64_t slots, int64_t sms, int64_t *chunk) {
  if (slots <= kOneBlock) {
    *chunk = slots;
    return 1;
  }
  *chunk = ((slots + sms - 1) / sms + kChunk - 1) / kChunk * kChunk;
  return (slots + *chunk - 1) / *chunk;
}

template <typename T>
cudaError_t launch(int64_t slots, int fan, int groups, const void *index, int32_t *offsets,
                   int32_t *order, int32_t *rows, int32_t *position, void *workspace,
                   const DeviceInfo &dev, cudaStream_t stream) {
  int64_t chunk;
  const int64_t blocks = blocks_of(slots, dev.sm_count, &chunk);
  int *counts = blocks > 1 ? static_cast<int *>(workspace) : nullptr;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(unsigned(blocks), 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (counts) {
    cfg.blockDim = dim3(1024, 1, 1);
    const cudaError_t e =
        cudaLaunchKernelEx(&cfg, count_kernel<T>, index, slots, chunk, groups, counts);
    if (e != cudaSuccess) return e;
  }
  const int64_t in_block = chunk < slots ? chunk : slots;
  const int64_t want = (in_block + 31) / 32;
  const int warps = int(want < 1 ? 1 : want > kMaxWarps ? kMaxWarps : want);
  const size_t smem = size_t(groups + 1) * (warps + 2) * sizeof(int);
  // Up to 513 x 34 counts (70 KB): above the default limit, so the kernel is opted in.
  static std::atomic<uint64_t> configured{0};
  const uint64_t bit = uint64_t(1) << (dev.id & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(
        place_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
        int((kMaxGroups + 1) * (kMaxWarps + 2) * sizeof(int)));
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_release);
  }
  cfg.blockDim = dim3(unsigned(32 * warps), 1, 1);
  cfg.dynamicSmemBytes = smem;
  return cudaLaunchKernelEx(&cfg, place_kernel<T>, index, slots, chunk, fan, groups,
                            static_cast<const int *>(counts), offsets, order, rows, position);
}

}  // namespace

size_t group_rows_workspace_bytes(int64_t slots, int64_t groups) {
  // A count per block and group for the most blocks a GPU has (one per SM, 256 at most).
  return slots <= kOneBlock ? 0 : size_t(256) * size_t(groups + 1) * sizeof(int);
}

cudaError_t launch_group_rows(int64_t slots, int fan, int groups, const void *index,
                              int index_bits, int32_t *offsets, int32_t *order, int32_t *rows,
                              int32_t *position, void *workspace, const DeviceInfo &dev,
                              cudaStream_t stream) {
  DeviceInfo d = dev;
  if (d.sm_count > 256) d.sm_count = 256;
  return index_bits == 64 ? launch<int64_t>(slots, fan, groups, index, offsets, order, rows,
                                            position, workspace, d, stream)
                          : launch<int32_t>(slots, fan, groups, index, offsets, order, rows,
                                            position, workspace, d, stream);
}

}  // namespace tmm
