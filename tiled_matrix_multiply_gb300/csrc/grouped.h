// grouped.h -- declarations of the grouped operators (row grouping, grouped products, adapters)
// shared by their translation units.  Not part of the public ABI (that is include/tmm_gemm.h).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "tmm_internal.h"

namespace tmm {

constexpr int kMaxGroups = 512;       // groups (experts, adapters) of one call
constexpr int kMaxAdapterRank = 1024;

// A stack of `count` row-major matrices (one for a plain operand), `stride` elements apart.
struct Stack {
  const void *data;
  int64_t count, rows, cols, ld, stride;
};

// y[p] = x[row(p)] w[g] for the rows p of group g.  trans_w: w holds N x K matrices.
struct GroupedProblem {
  int dtype;                    // TMM_F32, TMM_BF16, TMM_F16
  int64_t groups, rows, K, N;
  Stack x, w;                   // x: x.rows x K
  const int32_t *offsets;       // groups + 1
  const int32_t *row_index;     // rows, or NULL: row(p) = p
  int trans_w;
  void *y;
  int64_t ldy;
};
// dw[g] (K x N) = sum over the rows p of group g of x[row(p)]^T dy[p].
struct WgradProblem {
  int dtype;
  int64_t groups, rows, K, N;
  Stack x, dy;
  const int32_t *offsets, *row_index;
  void *dw;
  int64_t lddw, stride_dw;
};
// y[row(p)] = x[row(p)] w + scale[g] (x[row(p)] a[g]) b[g], row(p) over all rows of x.
struct LoraProblem {
  int dtype;
  int64_t groups, rows, K, N, rank;
  Stack x, w, a, b;
  int trans_w, trans_a, trans_b;
  const float *scale;           // groups
  const int32_t *offsets, *row_index;
  void *y;
  int64_t ldy;
};

// Workspace bytes (0: none needed; SIZE_MAX: the count does not fit in size_t).
size_t grouped_workspace_bytes(const GroupedProblem &p);
size_t wgrad_workspace_bytes(const WgradProblem &p);
size_t lora_workspace_bytes(const LoraProblem &p);

// Sizes reaching a launcher are > 0.
cudaError_t launch_grouped(const GroupedProblem &p, const DeviceInfo &dev, void *workspace,
                           cudaStream_t stream);
cudaError_t launch_wgrad(const WgradProblem &p, const DeviceInfo &dev, void *workspace,
                         cudaStream_t stream);
cudaError_t launch_lora(const LoraProblem &p, const DeviceInfo &dev, void *workspace,
                        cudaStream_t stream);
// Status word of the grouped kernels: bit 1 a bounded wait ran out of time.
cudaError_t grouped_device_status(unsigned int *status, bool clear);
void grouped_set_test_hooks(int drop_block, int64_t wait_limit_ns);

// A tensor map (TMA descriptor) over 16-bit elements: 2 or 3 dimensions, innermost first;
// strides (elements) of dimensions 1..; 128-byte swizzle; reads outside return zeros.
cudaError_t encode_16bit(CUtensorMap *map, const void *base, int dims, const uint64_t *size,
                         const uint64_t *stride, const uint32_t *box);

// Stable grouping of `slots` numbers (see group_rows in tmm_gemm.h).
// index holds 32- or 64-bit integers; rows may be NULL.
size_t group_rows_workspace_bytes(int64_t slots, int64_t groups);
cudaError_t launch_group_rows(int64_t slots, int fan, int groups, const void *index,
                              int index_bits, int32_t *offsets, int32_t *order, int32_t *rows,
                              int32_t *position, void *workspace, const DeviceInfo &dev,
                              cudaStream_t stream);

}  // namespace tmm
