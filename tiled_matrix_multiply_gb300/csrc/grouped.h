// grouped.h -- declarations of the grouped operators (row grouping, grouped products, adapters)
// shared by their translation units.  Not part of the public ABI (that is include/tmm_gemm.h).
#pragma once

#include <cstddef>
#include <cstdint>
#include <initializer_list>

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

// y = act(x w + bias) + residual, z = x w + bias.  trans_w: w is stored N x K.
struct LinearProblem {
  int dtype, act;
  int64_t rows, K, N;
  Stack x, w;
  int trans_w;
  const void *bias;             // N, or NULL
  int bias_f32;                 // FP32, else of the operands' type
  const void *residual;         // rows x N, or NULL
  int64_t ld_residual;
  void *y;
  int64_t ldy;
  void *pre;                    // z: rows x N, or NULL
  int64_t ld_pre;
};
// dz = dy act'(z), dx = dz w^T, dw = x^T dz, dbias = the sum of dz's rows; any of the last three
// NULL.
struct LinearGradProblem {
  int dtype, act;
  int64_t rows, K, N;
  Stack dy, x, w;
  int trans_w;
  const void *pre;              // z: rows x N (act other than none)
  int64_t ld_pre;
  void *dx;
  int64_t lddx;
  void *dw;                     // K x N, or N x K with trans_dw
  int64_t lddw;
  int trans_dw;
  float *dbias;
};

// An operand as the copy engine reads it: `planes` stacks of 16-bit matrices after each other.
struct Planes {
  const void *data;
  int64_t count, rows, cols, ld, stride;   // count: matrices of all planes
};
// A linear layer of few rows in FP32, on the FP32 units: no planes, no workspace.
bool linear_is_few(int dtype, int64_t rows);
cudaError_t launch_linear_few(const LinearProblem &p, const DeviceInfo &dev, cudaStream_t stream);

// Planes of up to four plain operands, in place where the copy engine can read them, else in *ws
// (which advances past planes_bytes of each), made by one launch.
size_t planes_bytes(const Stack &s, int dtype);
cudaError_t make_operand_planes(const Stack *const *operands, Planes *planes, int count, int dtype,
                                char **ws, const DeviceInfo &dev, cudaStream_t stream);
cudaError_t linear_device_status(unsigned int *status, bool clear);
void linear_set_test_hooks(int drop_block, int64_t wait_limit_ns);

// A workspace's parts start on 256-byte boundaries; SIZE_MAX: the count does not fit.
inline size_t round256(size_t b) { return (b + 255) / 256 * 256; }
inline size_t add_sizes(std::initializer_list<size_t> sizes) {
  size_t t = 0;
  for (size_t s : sizes) {
    if (s == SIZE_MAX) return SIZE_MAX;
    t += s;      // each is at most 2^61, and there are at most six
  }
  return t;
}
// Workspace bytes (0: none needed; SIZE_MAX: the count does not fit in size_t).
size_t grouped_workspace_bytes(const GroupedProblem &p);
size_t wgrad_workspace_bytes(const WgradProblem &p);
size_t lora_workspace_bytes(const LoraProblem &p);
size_t linear_workspace_bytes(const LinearProblem &p);
size_t linear_grad_workspace_bytes(const LinearGradProblem &p);

// Sizes reaching a launcher are > 0 (but K of launch_linear may be 0).
cudaError_t launch_linear(const LinearProblem &p, const DeviceInfo &dev, void *workspace,
                          cudaStream_t stream);
cudaError_t launch_linear_grad(const LinearGradProblem &p, const DeviceInfo &dev, void *workspace,
                               cudaStream_t stream);
// dz (rows x N, ldz, of the type, or with `planes` an FP32 value's three bf16 parts; NULL: not written)
// and dbias; `partial`: linear_bias_bytes of scratch.  `unscale` (FP16; NULL: dz as it is):
// linear_unscale_bytes, whose first value is left as what the written dz has to be multiplied by.
size_t linear_bias_bytes(int64_t rows, int64_t N, int dtype);
size_t linear_unscale_bytes();
cudaError_t launch_linear_slopes(const LinearGradProblem &p, void *dz, int64_t ldz, bool planes,
                                 float *unscale, float *partial, cudaStream_t stream);
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
