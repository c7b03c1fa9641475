// gemm_abi.cpp -- the extern "C" boundary: argument checks, device checks,
// path selection and launch-status reporting.  No device memory is allocated.
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>

#include <cuda_runtime.h>

#include "bounds_check.cuh"
#include "grouped.h"
#include "rows.h"
#include "tmm_gemm.h"
#include "tmm_internal.h"

namespace {

thread_local char g_last_error[256] = "";

int fail(int code, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return code;
}

constexpr int kMaxDevices = 64;
std::mutex g_dev_mutex;
bool g_dev_known[kMaxDevices] = {};
tmm::DeviceInfo g_dev_info[kMaxDevices];

// Properties of the current device, queried once per device.
int current_device(tmm::DeviceInfo *out) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(TMM_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices)
    return fail(TMM_ERR_UNSUPPORTED_DEVICE, "device ordinal %d out of range", dev);
  {
    std::lock_guard<std::mutex> lock(g_dev_mutex);
    if (g_dev_known[dev]) {
      *out = g_dev_info[dev];
      return TMM_OK;
    }
  }
  tmm::DeviceInfo info = {};
  info.id = dev;
  if ((e = cudaDeviceGetAttribute(&info.cc_major, cudaDevAttrComputeCapabilityMajor, dev)) ||
      (e = cudaDeviceGetAttribute(&info.cc_minor, cudaDevAttrComputeCapabilityMinor, dev)) ||
      (e = cudaDeviceGetAttribute(&info.sm_count, cudaDevAttrMultiProcessorCount, dev)) ||
      (e = cudaDeviceGetAttribute(&info.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin,
                                  dev)))
    return fail(TMM_ERR_CUDA, "cudaDeviceGetAttribute: %s", cudaGetErrorString(e));
  if (info.cc_major != 10 || info.cc_minor != 3)
    return fail(TMM_ERR_UNSUPPORTED_DEVICE,
                "device %d has compute capability %d.%d; this library is built for 10.3 (sm_103a)",
                dev, info.cc_major, info.cc_minor);
  {
    std::lock_guard<std::mutex> lock(g_dev_mutex);
    g_dev_info[dev] = info;
    g_dev_known[dev] = true;
  }
  *out = info;
  return TMM_OK;
}

// a * b + c without int64 overflow; false when it would overflow.
bool span_ok(int64_t rows, int64_t ld, int64_t cols) {
  if (rows <= 0 || cols <= 0) return true;
  const __int128 last = (__int128)(rows - 1) * ld + cols;
  return last <= (__int128)(INT64_MAX / 4);
}

// Byte range [lo, hi) spanned by the rows x cols window of a row-major matrix.
void byte_span(const void *p, int64_t rows, int64_t ld, int64_t cols, uintptr_t *lo,
               uintptr_t *hi) {
  *lo = reinterpret_cast<uintptr_t>(p);
  *hi = *lo + uintptr_t(((rows - 1) * ld + cols) * int64_t(sizeof(float)));
}

bool overlaps(uintptr_t a_lo, uintptr_t a_hi, uintptr_t b_lo, uintptr_t b_hi) {
  return a_lo < b_hi && b_lo < a_hi;
}

// Checks shared by every entry point; on success *nothing_to_do tells whether
// the call is a no-op (M == 0 or N == 0).  transa/transb select how A and B
// are stored: A as M x K (0) or K x M (1), B as K x N (0) or N x K (1).
int check_args(const char *who, int64_t M, int64_t N, int64_t K, int transa, int transb,
               const float *A, int64_t lda, const float *B, int64_t ldb, const float *C,
               int64_t ldc, bool *nothing_to_do) {
  *nothing_to_do = false;
  if ((transa != 0 && transa != 1) || (transb != 0 && transb != 1))
    return fail(TMM_ERR_INVALID_ARG, "%s: transa and transb must be 0 or 1", who);
  if (M < 0 || N < 0 || K < 0)
    return fail(TMM_ERR_INVALID_ARG, "%s: negative size (M=%lld N=%lld K=%lld)", who,
                (long long)M, (long long)N, (long long)K);
  if (M > INT32_MAX || N > INT32_MAX || K > INT32_MAX)
    return fail(TMM_ERR_INVALID_ARG, "%s: sizes above 2^31-1 are not supported", who);
  const int64_t a_rows = transa ? K : M, a_cols = transa ? M : K;
  const int64_t b_rows = transb ? N : K, b_cols = transb ? K : N;
  const int64_t min_lda = a_cols > 1 ? a_cols : 1, min_ldb = b_cols > 1 ? b_cols : 1;
  const int64_t min_ldc = N > 1 ? N : 1;
  if (lda < min_lda || ldb < min_ldb || ldc < min_ldc)
    return fail(TMM_ERR_INVALID_ARG,
                "%s: leading dimension too small (lda=%lld ldb=%lld ldc=%lld for stored A %lldx%lld, "
                "B %lldx%lld, C %lldx%lld)",
                who, (long long)lda, (long long)ldb, (long long)ldc, (long long)a_rows,
                (long long)a_cols, (long long)b_rows, (long long)b_cols, (long long)M,
                (long long)N);
  if (M == 0 || N == 0) {
    *nothing_to_do = true;
    return TMM_OK;
  }
  if (C == nullptr) return fail(TMM_ERR_INVALID_ARG, "%s: C is NULL", who);
  if (K > 0 && (A == nullptr || B == nullptr))
    return fail(TMM_ERR_INVALID_ARG, "%s: A or B is NULL", who);
  if (!span_ok(a_rows, lda, a_cols) || !span_ok(b_rows, ldb, b_cols) || !span_ok(M, ldc, N))
    return fail(TMM_ERR_INVALID_ARG, "%s: matrix extent overflows 64-bit byte offsets", who);
  if ((reinterpret_cast<uintptr_t>(A) | reinterpret_cast<uintptr_t>(B) |
       reinterpret_cast<uintptr_t>(C)) & 3u)
    return fail(TMM_ERR_INVALID_ARG, "%s: pointers must be 4-byte aligned", who);
  if (K > 0) {
    uintptr_t c_lo, c_hi, a_lo, a_hi, b_lo, b_hi;
    byte_span(C, M, ldc, N, &c_lo, &c_hi);
    byte_span(A, a_rows, lda, a_cols, &a_lo, &a_hi);
    byte_span(B, b_rows, ldb, b_cols, &b_lo, &b_hi);
    if (overlaps(c_lo, c_hi, a_lo, a_hi) || overlaps(c_lo, c_hi, b_lo, b_hi))
      return fail(TMM_ERR_ALIAS, "%s: the byte range of C overlaps A or B", who);
  }
  return TMM_OK;
}

using Launcher = cudaError_t (*)(const tmm::GemmProblem &, const tmm::DeviceInfo &, cudaStream_t);

int run(const char *who, Launcher launch, int transa, int transb, int64_t M, int64_t N,
        int64_t K, const float *A, int64_t lda, const float *B, int64_t ldb, float *C,
        int64_t ldc, tmm_stream_t stream) {
  bool noop = false;
  int rc = check_args(who, M, N, K, transa, transb, A, lda, B, ldb, C, ldc, &noop);
  if (rc != TMM_OK || noop) return rc;
  tmm::DeviceInfo dev;
  if ((rc = current_device(&dev)) != TMM_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (K == 0) {
    // The empty sum: zero the M x N window of C, leaving the row gaps alone.
    e = cudaMemset2DAsync(C, size_t(ldc) * sizeof(float), 0, size_t(N) * sizeof(float),
                          size_t(M), s);
    if (e != cudaSuccess)
      return fail(TMM_ERR_CUDA, "%s: cudaMemset2DAsync: %s", who, cudaGetErrorString(e));
    return TMM_OK;
  }
  tmm::GemmProblem p = {M, N, K, A, lda, B, ldb, C, ldc};
  p.transa = transa;
  p.transb = transb;
  e = launch(p, dev, s);
  if (e != cudaSuccess) return fail(TMM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return TMM_OK;
}

// ---- grouped operators ------------------------------------------------------------------

constexpr int64_t kMaxExtent = int64_t(1) << 29;   // rows and columns (3 planes stay below 2^31)

int element_size(int dtype) { return dtype == TMM_F32 ? 4 : 2; }

bool extent_ok(int64_t v) { return v >= 0 && v < kMaxExtent; }

// An operand's stored matrices: `count` of rows x cols, ld, stride (0: one for all groups).
tmm::Stack stack_of(const void *data, int64_t count, int64_t rows, int64_t cols, int64_t ld,
                    int64_t stride) {
  return {data, stride == 0 ? 1 : count, rows, cols, ld, stride};
}

// Elements from the first to the last of a stack, or -1 when the bytes do not fit in int64.
int64_t stack_span(const tmm::Stack &s) {
  if (s.count <= 0 || s.rows <= 0 || s.cols <= 0) return 0;
  const __int128 last =
      __int128(s.count - 1) * s.stride + __int128(s.rows - 1) * s.ld + s.cols;
  return last > __int128(INT64_MAX / 8) ? -1 : int64_t(last);
}

// Checks of one operand; `name` for the message.
int check_stack(const char *who, const char *name, const tmm::Stack &s, int size) {
  if (s.ld < (s.cols > 1 ? s.cols : 1))
    return fail(TMM_ERR_INVALID_ARG, "%s: leading dimension of %s too small (%lld for %lld columns)",
                who, name, (long long)s.ld, (long long)s.cols);
  if (s.stride < 0)
    return fail(TMM_ERR_INVALID_ARG, "%s: negative stride of %s", who, name);
  if (stack_span(s) < 0)
    return fail(TMM_ERR_INVALID_ARG, "%s: extent of %s overflows 64-bit byte offsets", who, name);
  if (stack_span(s) > 0 && s.data == nullptr)
    return fail(TMM_ERR_INVALID_ARG, "%s: %s is NULL", who, name);
  if (reinterpret_cast<uintptr_t>(s.data) % unsigned(size))
    return fail(TMM_ERR_INVALID_ARG, "%s: %s must be %d-byte aligned", who, name, size);
  return TMM_OK;
}

struct Bytes {
  const char *name;
  const void *p;
  int64_t n;
};

// Whether the written range [0] overlaps one of the others.
int check_alias(const char *who, const Bytes *r, int count) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(r[0].p), hi = lo + uintptr_t(r[0].n);
  for (int i = 1; i < count; ++i) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(r[i].p);
    if (r[i].p && r[i].n > 0 && r[0].n > 0 && overlaps(lo, hi, a, a + uintptr_t(r[i].n)))
      return fail(TMM_ERR_ALIAS, "%s: %s overlaps %s", who, r[0].name, r[i].name);
  }
  return TMM_OK;
}

int check_common(const char *who, int dtype, int64_t groups, int64_t rows, int64_t N, int64_t K,
                 const int32_t *offsets, const int32_t *row_index) {
  if (dtype != TMM_F32 && dtype != TMM_BF16 && dtype != TMM_F16)
    return fail(TMM_ERR_INVALID_ARG, "%s: unknown dtype %d", who, dtype);
  if (groups < 1 || groups > tmm::kMaxGroups)
    return fail(TMM_ERR_INVALID_ARG, "%s: need 1 <= groups <= %d (groups=%lld)", who,
                tmm::kMaxGroups, (long long)groups);
  if (!extent_ok(rows) || !extent_ok(N) || !extent_ok(K))
    return fail(TMM_ERR_INVALID_ARG, "%s: sizes must be >= 0 and below 2^29 (rows=%lld N=%lld K=%lld)",
                who, (long long)rows, (long long)N, (long long)K);
  if (offsets == nullptr) return fail(TMM_ERR_INVALID_ARG, "%s: offsets is NULL", who);
  if ((reinterpret_cast<uintptr_t>(offsets) | reinterpret_cast<uintptr_t>(row_index)) & 3u)
    return fail(TMM_ERR_INVALID_ARG, "%s: offsets and row_index must be 4-byte aligned", who);
  return TMM_OK;
}

int check_x_rows(const char *who, int64_t rows, int64_t x_rows, const int32_t *row_index) {
  if (!extent_ok(x_rows) || (row_index == nullptr && x_rows < rows))
    return fail(TMM_ERR_INVALID_ARG, "%s: x has %lld rows (below 2^29, and without row_index at "
                "least the %lld that are read)", who, (long long)x_rows, (long long)rows);
  return TMM_OK;
}

int check_workspace(const char *who, size_t need, const void *workspace, size_t bytes) {
  if (need == SIZE_MAX)
    return fail(TMM_ERR_INVALID_ARG, "%s: the workspace size overflows size_t", who);
  if (need == 0) return TMM_OK;
  if (workspace == nullptr || bytes < need)
    return fail(TMM_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, %zu given", who, need,
                workspace == nullptr ? size_t(0) : bytes);
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return fail(TMM_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  return TMM_OK;
}

// Zeros in every matrix of an output (the empty sum), leaving gaps alone.
int zero_output(const char *who, void *p, int64_t count, int64_t rows, int64_t cols, int64_t ld,
                int64_t stride, int size, cudaStream_t s) {
  for (int64_t i = 0; i < count; ++i) {
    const cudaError_t e =
        cudaMemset2DAsync(static_cast<char *>(p) + i * stride * size, size_t(ld) * size, 0,
                          size_t(cols) * size, size_t(rows), s);
    if (e != cudaSuccess)
      return fail(TMM_ERR_CUDA, "%s: cudaMemset2DAsync: %s", who, cudaGetErrorString(e));
  }
  return TMM_OK;
}

tmm::GroupedProblem grouped_problem(int dtype, int transw, int64_t groups, int64_t rows, int64_t N,
                                    int64_t K, const void *x, int64_t x_rows, int64_t ldx,
                                    const void *w, int64_t ldw, int64_t stride_w) {
  tmm::GroupedProblem p = {};
  p.dtype = dtype;
  p.groups = groups;
  p.rows = rows;
  p.K = K;
  p.N = N;
  p.x = stack_of(x, 1, x_rows, K, ldx, 0);
  p.w = stack_of(w, groups, transw ? N : K, transw ? K : N, ldw, stride_w);
  p.trans_w = transw;
  return p;
}

tmm::LoraProblem lora_problem(int dtype, int transw, int transa, int transb, int64_t groups,
                              int64_t rows, int64_t N, int64_t K, int64_t rank, const void *x,
                              int64_t ldx, const void *w, int64_t ldw, const void *a, int64_t lda,
                              int64_t stride_a, const void *b, int64_t ldb, int64_t stride_b) {
  tmm::LoraProblem p = {};
  p.dtype = dtype;
  p.groups = groups;
  p.rows = rows;
  p.K = K;
  p.N = N;
  p.rank = rank;
  p.x = stack_of(x, 1, rows, K, ldx, 0);
  p.w = stack_of(w, 1, transw ? N : K, transw ? K : N, ldw, 0);
  p.a = stack_of(a, groups, transa ? rank : K, transa ? K : rank, lda, stride_a);
  p.b = stack_of(b, groups, transb ? N : rank, transb ? rank : N, ldb, stride_b);
  p.trans_w = transw;
  p.trans_a = transa;
  p.trans_b = transb;
  return p;
}

// Sizes for a *_workspace_size call, which has no status to return.
bool sizes_ok(int dtype, int64_t groups, int64_t rows, int64_t N, int64_t K) {
  return (dtype == TMM_F32 || dtype == TMM_BF16 || dtype == TMM_F16) && groups >= 1 &&
         groups <= tmm::kMaxGroups && extent_ok(rows) && extent_ok(N) && extent_ok(K) &&
         rows > 0 && N > 0 && K > 0;
}

}  // namespace

extern "C" {

int gemm_f32(int64_t M, int64_t N, int64_t K, const float *A, int64_t lda, const float *B,
             int64_t ldb, float *C, int64_t ldc, tmm_stream_t stream) {
  return run("gemm_f32", tmm::launch_simt, 0, 0, M, N, K, A, lda, B, ldb, C, ldc, stream);
}

int gemm_f32_ex(int transa, int transb, int64_t M, int64_t N, int64_t K, const float *A,
                int64_t lda, const float *B, int64_t ldb, float *C, int64_t ldc,
                tmm_stream_t stream) {
  return run("gemm_f32_ex", tmm::launch_simt, transa, transb, M, N, K, A, lda, B, ldb, C, ldc,
             stream);
}

int gemm_f32_naive(int64_t M, int64_t N, int64_t K, const float *A, int64_t lda, const float *B,
                   int64_t ldb, float *C, int64_t ldc, tmm_stream_t stream) {
  return run("gemm_f32_naive", tmm::launch_naive, 0, 0, M, N, K, A, lda, B, ldb, C, ldc,
             stream);
}

int tmm_check_device(tmm_stream_t stream) {
  cudaError_t e = cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess)
    return fail(TMM_ERR_CUDA, "tmm_check_device: cudaStreamSynchronize: %s", cudaGetErrorString(e));
  unsigned int simt = 0, tc3 = 0, win = 0, sm = 0, naive = 0, stage = 0, grouped = 0, linear = 0;
  e = tmm::simt_device_status(&simt, true);
  if (e == cudaSuccess) e = tmm::tc3_device_status(&tc3, true);
  if (e == cudaSuccess) e = tmm::window_device_status(&win, true);
  if (e == cudaSuccess) e = tmm::softmax_device_status(&sm, true);
  if (e == cudaSuccess) e = tmm::naive_device_status(&naive, true);
  if (e == cudaSuccess) e = tmm::stage_device_status(&stage, true);
  if (e == cudaSuccess) e = tmm::grouped_device_status(&grouped, true);
  if (e == cudaSuccess) e = tmm::linear_device_status(&linear, true);
  if (e != cudaSuccess)
    return fail(TMM_ERR_CUDA, "tmm_check_device: status read: %s", cudaGetErrorString(e));
  if ((simt | tc3 | naive | stage) & tmm::kStatusBounds)
    return fail(TMM_ERR_BOUNDS,
                "tmm_check_device: a range check of the bounds-checked build failed inside %s",
                (simt & tmm::kStatusBounds)    ? "gemm_f32"
                : (stage & tmm::kStatusBounds) ? "gemm_f32 (operand restaging)"
                : (tc3 & tmm::kStatusBounds)   ? "gemm_f32_tc3"
                                               : "gemm_f32_naive");
  if (simt | tc3 | win | sm | grouped | linear)
    return fail(TMM_ERR_DEVICE_TIMEOUT,
                "tmm_check_device: a bounded wait inside %s ran out of time; the affected "
                "results are not valid",
                simt      ? "gemm_f32"
                : tc3     ? "gemm_f32_tc3"
                : win     ? "window_sum_f32"
                : grouped ? "a grouped product"
                : linear  ? "a linear layer's product"
                          : "softmax_rows_f32");
  return TMM_OK;
}

int tmm_testing_simt_plan(int64_t M, int64_t N, int64_t K, int wide, int vec_c, int may_reduce,
                          int64_t slots, int64_t *out) {
  if (M <= 0 || N <= 0 || K <= 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX ||
      slots <= 0 || out == nullptr)
    return fail(TMM_ERR_INVALID_ARG, "tmm_testing_simt_plan: bad arguments");
  tmm::simt_plan_for_testing(M, N, K, wide, vec_c, may_reduce, slots, out);
  return TMM_OK;
}

int tmm_testing_tc3_plan(int64_t M, int64_t N, int64_t K, int pairs, int64_t slots,
                         int64_t *out) {
  if (M <= 0 || N <= 0 || K <= 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX ||
      slots <= 0 || out == nullptr)
    return fail(TMM_ERR_INVALID_ARG, "tmm_testing_tc3_plan: bad arguments");
  tmm::tc3_plan_for_testing(M, N, K, pairs, slots, out);
  return TMM_OK;
}

int tmm_testing_set_wait_hooks(int drop_signal_block, int64_t wait_limit_ns) {
  tmm::simt_set_test_hooks(drop_signal_block, wait_limit_ns);
  tmm::tc3_set_test_hooks(drop_signal_block, wait_limit_ns);
  tmm::window_set_test_hooks(drop_signal_block, wait_limit_ns);
  tmm::softmax_set_test_hooks(drop_signal_block, wait_limit_ns);
  tmm::grouped_set_test_hooks(drop_signal_block, wait_limit_ns);
  tmm::linear_set_test_hooks(drop_signal_block, wait_limit_ns);
  return TMM_OK;
}

size_t gemm_f32_tc3_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX) return 0;
  return tmm::tc3_workspace_bytes(M, N, K);
}

int gemm_f32_tc3_ex(int transa, int transb, int64_t M, int64_t N, int64_t K, const float *A,
                    int64_t lda, const float *B, int64_t ldb, float *C, int64_t ldc,
                    void *workspace, size_t workspace_bytes, tmm_stream_t stream) {
  const char *who = "gemm_f32_tc3";
  bool noop = false;
  int rc = check_args(who, M, N, K, transa, transb, A, lda, B, ldb, C, ldc, &noop);
  if (rc != TMM_OK || noop) return rc;
  tmm::DeviceInfo dev;
  if ((rc = current_device(&dev)) != TMM_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) {
    cudaError_t e = cudaMemset2DAsync(C, size_t(ldc) * sizeof(float), 0,
                                      size_t(N) * sizeof(float), size_t(M), s);
    if (e != cudaSuccess)
      return fail(TMM_ERR_CUDA, "%s: cudaMemset2DAsync: %s", who, cudaGetErrorString(e));
    return TMM_OK;
  }
  const size_t need = tmm::tc3_workspace_bytes(M, N, K);
  if (need == SIZE_MAX)
    return fail(TMM_ERR_INVALID_ARG, "%s: the workspace size of this product overflows size_t",
                who);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(TMM_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, %zu given", who, need,
                workspace == nullptr ? size_t(0) : workspace_bytes);
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return fail(TMM_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  {
    uintptr_t c_lo, c_hi, a_lo, a_hi, b_lo, b_hi;
    byte_span(C, M, ldc, N, &c_lo, &c_hi);
    byte_span(A, transa ? K : M, lda, transa ? M : K, &a_lo, &a_hi);
    byte_span(B, transb ? N : K, ldb, transb ? K : N, &b_lo, &b_hi);
    const uintptr_t w_lo = reinterpret_cast<uintptr_t>(workspace), w_hi = w_lo + need;
    if (overlaps(w_lo, w_hi, c_lo, c_hi) || overlaps(w_lo, w_hi, a_lo, a_hi) ||
        overlaps(w_lo, w_hi, b_lo, b_hi))
      return fail(TMM_ERR_ALIAS, "%s: the workspace overlaps A, B or C", who);
  }
  tmm::GemmProblem p = {M, N, K, A, lda, B, ldb, C, ldc};
  p.transa = transa;
  p.transb = transb;
  cudaError_t e = tmm::launch_tc3(p, dev, workspace, s);
  if (e != cudaSuccess) return fail(TMM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return TMM_OK;
}

int gemm_f32_tc3(int64_t M, int64_t N, int64_t K, const float *A, int64_t lda, const float *B,
                 int64_t ldb, float *C, int64_t ldc, void *workspace, size_t workspace_bytes,
                 tmm_stream_t stream) {
  return gemm_f32_tc3_ex(0, 0, M, N, K, A, lda, B, ldb, C, ldc, workspace, workspace_bytes,
                         stream);
}

int gemm_f32_tc3_noalloc(int64_t M, int64_t N, int64_t K, const float *A, int64_t lda,
                         const float *B, int64_t ldb, float *C, int64_t ldc,
                         tmm_stream_t stream) {
  const char *who = "gemm_f32_tc3_noalloc";
  bool noop = false;
  int rc = check_args(who, M, N, K, 0, 0, A, lda, B, ldb, C, ldc, &noop);
  if (rc != TMM_OK || noop) return rc;
  // The size limit is checked before any CUDA call, so a refused product
  // reaches neither the device nor the scratch.
  const size_t need = K > 0 ? tmm::tc3_workspace_bytes(M, N, K) : 0;
  const size_t limit = tmm::tc3_noalloc_scratch_bytes();
  if (need > limit)
    return fail(TMM_ERR_INVALID_ARG,
                "%s: this product needs %zu bytes of scratch but the fixed scratch holds %zu; "
                "use gemm_f32_tc3 with a caller-supplied workspace",
                who, need, limit);
  tmm::DeviceInfo dev;
  if ((rc = current_device(&dev)) != TMM_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) {
    cudaError_t e = cudaMemset2DAsync(C, size_t(ldc) * sizeof(float), 0,
                                      size_t(N) * sizeof(float), size_t(M), s);
    if (e != cudaSuccess)
      return fail(TMM_ERR_CUDA, "%s: cudaMemset2DAsync: %s", who, cudaGetErrorString(e));
    return TMM_OK;
  }
  void *scratch = nullptr;
  cudaError_t e = tmm::tc3_noalloc_scratch(&scratch);
  if (e != cudaSuccess)
    return fail(TMM_ERR_CUDA, "%s: scratch address lookup: %s", who, cudaGetErrorString(e));
  const tmm::GemmProblem p = {M, N, K, A, lda, B, ldb, C, ldc};
  e = tmm::launch_tc3(p, dev, scratch, s);
  if (e != cudaSuccess) return fail(TMM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return TMM_OK;
}

int window_sum_f32(int64_t n, int W, const float *x, float *y, tmm_stream_t stream) {
  const char *who = "window_sum_f32";
  if (n < 0 || W < 1 || W > tmm::kMaxWindow)
    return fail(TMM_ERR_INVALID_ARG, "%s: need n >= 0 and 1 <= W <= %d (n=%lld W=%d)", who,
                tmm::kMaxWindow, (long long)n, W);
  if (n == 0) return TMM_OK;
  if (n > (int64_t(1) << 40))
    return fail(TMM_ERR_INVALID_ARG, "%s: n above 2^40 is not supported", who);
  if (x == nullptr || y == nullptr) return fail(TMM_ERR_INVALID_ARG, "%s: x or y is NULL", who);
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) & 3u)
    return fail(TMM_ERR_INVALID_ARG, "%s: pointers must be 4-byte aligned", who);
  const uintptr_t x_lo = reinterpret_cast<uintptr_t>(x), x_hi = x_lo + uintptr_t(n + W - 1) * 4;
  const uintptr_t y_lo = reinterpret_cast<uintptr_t>(y), y_hi = y_lo + uintptr_t(n) * 4;
  if (overlaps(x_lo, x_hi, y_lo, y_hi))
    return fail(TMM_ERR_ALIAS, "%s: the output overlaps the input", who);
  tmm::DeviceInfo dev;
  int rc = current_device(&dev);
  if (rc != TMM_OK) return rc;
  cudaError_t e = tmm::launch_window_sum(n, W, x, y, dev, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(TMM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return TMM_OK;
}

size_t sum_f32_workspace_size(int64_t n) {
  (void)n;
  return size_t(tmm::kSumMaxPartials) * sizeof(float);
}

int sum_f32(int64_t n, const float *x, float *out, void *workspace, size_t workspace_bytes,
            tmm_stream_t stream) {
  const char *who = "sum_f32";
  if (n < 0 || n > (int64_t(1) << 40))
    return fail(TMM_ERR_INVALID_ARG, "%s: need 0 <= n <= 2^40 (n=%lld)", who, (long long)n);
  if (out == nullptr) return fail(TMM_ERR_INVALID_ARG, "%s: out is NULL", who);
  if (reinterpret_cast<uintptr_t>(out) & 3u)
    return fail(TMM_ERR_INVALID_ARG, "%s: out must be 4-byte aligned", who);
  const size_t need = sum_f32_workspace_size(n);
  if (n > 0) {
    if (x == nullptr) return fail(TMM_ERR_INVALID_ARG, "%s: x is NULL", who);
    if (reinterpret_cast<uintptr_t>(x) & 3u)
      return fail(TMM_ERR_INVALID_ARG, "%s: x must be 4-byte aligned", who);
    if (workspace == nullptr || workspace_bytes < need)
      return fail(TMM_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, %zu given", who, need,
                  workspace == nullptr ? size_t(0) : workspace_bytes);
    if (reinterpret_cast<uintptr_t>(workspace) & 15u)
      return fail(TMM_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", who);
    const uintptr_t x_lo = reinterpret_cast<uintptr_t>(x), x_hi = x_lo + uintptr_t(n) * 4;
    const uintptr_t w_lo = reinterpret_cast<uintptr_t>(workspace), w_hi = w_lo + need;
    if (overlaps(x_lo, x_hi, w_lo, w_hi))
      return fail(TMM_ERR_ALIAS, "%s: the workspace overlaps x", who);
  }
  tmm::DeviceInfo dev;
  int rc = current_device(&dev);
  if (rc != TMM_OK) return rc;
  cudaError_t e = tmm::launch_sum(n, x, out, static_cast<float *>(workspace), dev,
                                  reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(TMM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return TMM_OK;
}

int softmax_rows_f32(int64_t rows, int64_t cols, const float *x, int64_t ldx, float *y,
                     int64_t ldy, tmm_stream_t stream) {
  const char *who = "softmax_rows_f32";
  if (rows < 0 || cols < 0)
    return fail(TMM_ERR_INVALID_ARG, "%s: negative size (rows=%lld cols=%lld)", who,
                (long long)rows, (long long)cols);
  if (cols > INT32_MAX)
    return fail(TMM_ERR_INVALID_ARG, "%s: cols above 2^31-1 is not supported", who);
  const int64_t min_ld = cols > 1 ? cols : 1;
  if (ldx < min_ld || ldy < min_ld)
    return fail(TMM_ERR_INVALID_ARG, "%s: row stride too small (ldx=%lld ldy=%lld, cols=%lld)",
                who, (long long)ldx, (long long)ldy, (long long)cols);
  if (rows == 0 || cols == 0) return TMM_OK;
  if (x == nullptr || y == nullptr) return fail(TMM_ERR_INVALID_ARG, "%s: x or y is NULL", who);
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) & 3u)
    return fail(TMM_ERR_INVALID_ARG, "%s: pointers must be 4-byte aligned", who);
  if (!span_ok(rows, ldx, cols) || !span_ok(rows, ldy, cols))
    return fail(TMM_ERR_INVALID_ARG, "%s: matrix extent overflows 64-bit byte offsets", who);
  const bool in_place = x == y && ldx == ldy;
  if (!in_place) {
    uintptr_t x_lo, x_hi, y_lo, y_hi;
    byte_span(x, rows, ldx, cols, &x_lo, &x_hi);
    byte_span(y, rows, ldy, cols, &y_lo, &y_hi);
    if (overlaps(x_lo, x_hi, y_lo, y_hi))
      return fail(TMM_ERR_ALIAS, "%s: y overlaps x without being x itself", who);
  }
  tmm::DeviceInfo dev;
  int rc = current_device(&dev);
  if (rc != TMM_OK) return rc;
  cudaError_t e = tmm::launch_softmax_rows(rows, int(cols), x, ldx, y, ldy, dev,
                                           reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(TMM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return TMM_OK;
}

size_t group_rows_workspace_size(int64_t tokens, int64_t fan, int64_t groups) {
  if (tokens < 1 || fan < 1 || groups < 1 || groups > tmm::kMaxGroups ||
      __int128(tokens) * fan > INT32_MAX)
    return 0;
  return tmm::group_rows_workspace_bytes(tokens * fan, groups);
}

int group_rows(int64_t tokens, int64_t fan, int64_t groups, const void *index, int index_bits,
               int32_t *offsets, int32_t *order, int32_t *rows, int32_t *position,
               void *workspace, size_t workspace_bytes, tmm_stream_t stream) {
  const char *who = "group_rows";
  if (tokens < 0 || fan < 1 || __int128(tokens) * fan > INT32_MAX)
    return fail(TMM_ERR_INVALID_ARG, "%s: need tokens >= 0, fan >= 1 and tokens * fan < 2^31 "
                "(tokens=%lld fan=%lld)", who, (long long)tokens, (long long)fan);
  if (groups < 1 || groups > tmm::kMaxGroups)
    return fail(TMM_ERR_INVALID_ARG, "%s: need 1 <= groups <= %d (groups=%lld)", who,
                tmm::kMaxGroups, (long long)groups);
  if (index_bits != 32 && index_bits != 64)
    return fail(TMM_ERR_INVALID_ARG, "%s: index_bits must be 32 or 64", who);
  if (offsets == nullptr) return fail(TMM_ERR_INVALID_ARG, "%s: offsets is NULL", who);
  const int64_t slots = tokens * fan;
  if (slots > 0 && (index == nullptr || order == nullptr || position == nullptr))
    return fail(TMM_ERR_INVALID_ARG, "%s: index, order or position is NULL", who);
  if (reinterpret_cast<uintptr_t>(index) % unsigned(index_bits / 8) ||
      ((reinterpret_cast<uintptr_t>(offsets) | reinterpret_cast<uintptr_t>(order) |
        reinterpret_cast<uintptr_t>(rows) | reinterpret_cast<uintptr_t>(position)) & 3u))
    return fail(TMM_ERR_INVALID_ARG, "%s: arrays must be naturally aligned", who);
  const size_t need = tmm::group_rows_workspace_bytes(slots, groups);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(TMM_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, %zu given", who, need,
                workspace == nullptr ? size_t(0) : workspace_bytes);
  if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 15u))
    return fail(TMM_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", who);
  const Bytes all[6] = {{"index", index, slots * (index_bits / 8)},
                        {"offsets", offsets, (groups + 1) * 4},
                        {"order", order, slots * 4},
                        {"rows", rows, rows ? slots * 4 : 0},
                        {"position", position, slots * 4},
                        {"the workspace", workspace, int64_t(need)}};
  for (int i = 1; i < 6; ++i) {        // every array written, against those before it
    Bytes r[6];
    r[0] = all[i];
    for (int j = 0; j < i; ++j) r[j + 1] = all[j];
    if (all[i].p == nullptr) continue;
    const int rc = check_alias(who, r, i + 1);
    if (rc != TMM_OK) return rc;
  }
  tmm::DeviceInfo dev;
  int rc = current_device(&dev);
  if (rc != TMM_OK) return rc;
  const cudaError_t e = tmm::launch_group_rows(slots, int(fan), int(groups), index, index_bits,
                                               offsets, order, rows, position, workspace, dev,
                                               reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(TMM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return TMM_OK;
}

size_t gemm_grouped_workspace_size(int dtype, int transw, int64_t groups, int64_t rows, int64_t N,
                                   int64_t K, const void *x, int64_t x_rows, int64_t ldx,
                                   const int32_t *row_index, const void *w, int64_t ldw,
                                   int64_t stride_w) {
  if (!sizes_ok(dtype, groups, rows, N, K) || !extent_ok(x_rows)) return 0;
  tmm::GroupedProblem p =
      grouped_problem(dtype, transw, groups, rows, N, K, x, x_rows, ldx, w, ldw, stride_w);
  p.row_index = row_index;
  return tmm::grouped_workspace_bytes(p);
}

int gemm_grouped(int dtype, int transw, int64_t groups, int64_t rows, int64_t N, int64_t K,
                 const void *x, int64_t x_rows, int64_t ldx, const int32_t *offsets,
                 const int32_t *row_index, const void *w, int64_t ldw, int64_t stride_w, void *y,
                 int64_t ldy, void *workspace, size_t workspace_bytes, tmm_stream_t stream) {
  const char *who = "gemm_grouped";
  int rc = check_common(who, dtype, groups, rows, N, K, offsets, row_index);
  if (rc != TMM_OK) return rc;
  if (transw != 0 && transw != 1)
    return fail(TMM_ERR_INVALID_ARG, "%s: transw must be 0 or 1", who);
  if ((rc = check_x_rows(who, rows, x_rows, row_index)) != TMM_OK) return rc;
  tmm::GroupedProblem p =
      grouped_problem(dtype, transw, groups, rows, N, K, x, x_rows, ldx, w, ldw, stride_w);
  p.offsets = offsets;
  p.row_index = row_index;
  const int size = element_size(dtype);
  const tmm::Stack y_s = stack_of(y, 1, rows, N, ldy, 0);
  if ((rc = check_stack(who, "x", p.x, size)) != TMM_OK ||
      (rc = check_stack(who, "w", p.w, size)) != TMM_OK ||
      (rc = check_stack(who, "y", y_s, size)) != TMM_OK)
    return rc;
  if (rows == 0 || N == 0) return TMM_OK;
  const size_t need = K > 0 ? tmm::grouped_workspace_bytes(p) : 0;
  if ((rc = check_workspace(who, need, workspace, workspace_bytes)) != TMM_OK) return rc;
  const Bytes out[6] = {{"y", y, stack_span(y_s) * size},
                        {"x", x, stack_span(p.x) * size},
                        {"w", w, stack_span(p.w) * size},
                        {"offsets", offsets, (groups + 1) * 4},
                        {"row_index", row_index, rows * 4},
                        {"the workspace", workspace, int64_t(need)}};
  const Bytes ws[5] = {out[5], out[1], out[2], out[3], out[4]};
  if ((rc = check_alias(who, out, 6)) != TMM_OK || (rc = check_alias(who, ws, 5)) != TMM_OK)
    return rc;
  tmm::DeviceInfo dev;
  if ((rc = current_device(&dev)) != TMM_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) return zero_output(who, y, 1, rows, N, ldy, 0, size, s);
  p.y = y;
  p.ldy = ldy;
  if (x_rows == 0) return zero_output(who, y, 1, rows, N, ldy, 0, size, s);   // all zero rows
  const cudaError_t e = tmm::launch_grouped(p, dev, workspace, s);
  if (e != cudaSuccess) return fail(TMM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return TMM_OK;
}

size_t gemm_grouped_wgrad_workspace_size(int dtype, int64_t groups, int64_t rows, int64_t N,
                                         int64_t K, const void *x, int64_t x_rows, int64_t ldx,
                                         const int32_t *row_index, const void *dy,
                                         int64_t lddy) {
  if (!sizes_ok(dtype, groups, rows, N, K) || !extent_ok(x_rows)) return 0;
  tmm::WgradProblem p = {};
  p.dtype = dtype;
  p.groups = groups;
  p.rows = rows;
  p.N = N;
  p.row_index = row_index;
  p.x = stack_of(x, 1, x_rows, K, ldx, 0);
  p.dy = stack_of(dy, 1, rows, N, lddy, 0);
  return tmm::wgrad_workspace_bytes(p);
}

int gemm_grouped_wgrad(int dtype, int64_t groups, int64_t rows, int64_t N, int64_t K,
                       const void *x, int64_t x_rows, int64_t ldx, const int32_t *offsets,
                       const int32_t *row_index, const void *dy, int64_t lddy, void *dw,
                       int64_t lddw, int64_t stride_dw, void *workspace, size_t workspace_bytes,
                       tmm_stream_t stream) {
  const char *who = "gemm_grouped_wgrad";
  int rc = check_common(who, dtype, groups, rows, N, K, offsets, row_index);
  if (rc != TMM_OK) return rc;
  if ((rc = check_x_rows(who, rows, x_rows, row_index)) != TMM_OK) return rc;
  const int size = element_size(dtype);
  tmm::WgradProblem p = {};
  p.dtype = dtype;
  p.groups = groups;
  p.rows = rows;
  p.K = K;
  p.N = N;
  p.offsets = offsets;
  p.row_index = row_index;
  p.x = stack_of(x, 1, x_rows, K, ldx, 0);
  p.dy = stack_of(dy, 1, rows, N, lddy, 0);
  tmm::Stack dw_s = {dw, groups, K, N, lddw, stride_dw};
  if ((rc = check_stack(who, "x", p.x, size)) != TMM_OK ||
      (rc = check_stack(who, "dy", p.dy, size)) != TMM_OK ||
      (rc = check_stack(who, "dw", dw_s, size)) != TMM_OK)
    return rc;
  if (K == 0 || N == 0) return TMM_OK;
  if (groups > 1 && stride_dw < (K - 1) * lddw + N)
    return fail(TMM_ERR_INVALID_ARG, "%s: the matrices of dw overlap (stride %lld)", who,
                (long long)stride_dw);
  const size_t need = rows > 0 ? tmm::wgrad_workspace_bytes(p) : 0;
  if ((rc = check_workspace(who, need, workspace, workspace_bytes)) != TMM_OK) return rc;
  const Bytes out[6] = {{"dw", dw, stack_span(dw_s) * size},
                        {"x", x, stack_span(p.x) * size},
                        {"dy", dy, stack_span(p.dy) * size},
                        {"offsets", offsets, (groups + 1) * 4},
                        {"row_index", row_index, rows * 4},
                        {"the workspace", workspace, int64_t(need)}};
  const Bytes ws[5] = {out[5], out[1], out[2], out[3], out[4]};
  if ((rc = check_alias(who, out, 6)) != TMM_OK || (rc = check_alias(who, ws, 5)) != TMM_OK)
    return rc;
  tmm::DeviceInfo dev;
  if ((rc = current_device(&dev)) != TMM_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0 || x_rows == 0)
    return zero_output(who, dw, groups, K, N, lddw, stride_dw, size, s);
  p.dw = dw;
  p.lddw = lddw;
  p.stride_dw = stride_dw;
  const cudaError_t e = tmm::launch_wgrad(p, dev, workspace, s);
  if (e != cudaSuccess) return fail(TMM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return TMM_OK;
}

size_t gemm_lora_workspace_size(int dtype, int transw, int transa, int transb, int64_t groups,
                                int64_t rows, int64_t N, int64_t K, int64_t rank, const void *x,
                                int64_t ldx, const int32_t *row_index, const void *w, int64_t ldw,
                                const void *a, int64_t lda, int64_t stride_a, const void *b,
                                int64_t ldb, int64_t stride_b) {
  if (!sizes_ok(dtype, groups, rows, N, K) || rank < 1 || rank > tmm::kMaxAdapterRank) return 0;
  tmm::LoraProblem p = lora_problem(dtype, transw, transa, transb, groups, rows, N, K, rank, x,
                                    ldx, w, ldw, a, lda, stride_a, b, ldb, stride_b);
  p.row_index = row_index;
  return tmm::lora_workspace_bytes(p);
}

int gemm_lora(int dtype, int transw, int transa, int transb, int64_t groups, int64_t rows,
              int64_t N, int64_t K, int64_t rank, const void *x, int64_t ldx,
              const int32_t *offsets, const int32_t *row_index, const void *w, int64_t ldw,
              const void *a, int64_t lda, int64_t stride_a, const void *b, int64_t ldb,
              int64_t stride_b, const float *scale, void *y, int64_t ldy, void *workspace,
              size_t workspace_bytes, tmm_stream_t stream) {
  const char *who = "gemm_lora";
  int rc = check_common(who, dtype, groups, rows, N, K, offsets, row_index);
  if (rc != TMM_OK) return rc;
  if ((transw | transa | transb) & ~1)
    return fail(TMM_ERR_INVALID_ARG, "%s: transw, transa and transb must be 0 or 1", who);
  if (rank < 1 || rank > tmm::kMaxAdapterRank)
    return fail(TMM_ERR_INVALID_ARG, "%s: need 1 <= rank <= %d (rank=%lld)", who,
                tmm::kMaxAdapterRank, (long long)rank);
  tmm::LoraProblem p = lora_problem(dtype, transw, transa, transb, groups, rows, N, K, rank, x,
                                    ldx, w, ldw, a, lda, stride_a, b, ldb, stride_b);
  p.offsets = offsets;
  p.row_index = row_index;
  const int size = element_size(dtype);
  const tmm::Stack y_s = stack_of(y, 1, rows, N, ldy, 0);
  if ((rc = check_stack(who, "x", p.x, size)) != TMM_OK ||
      (rc = check_stack(who, "w", p.w, size)) != TMM_OK ||
      (rc = check_stack(who, "a", p.a, size)) != TMM_OK ||
      (rc = check_stack(who, "b", p.b, size)) != TMM_OK ||
      (rc = check_stack(who, "y", y_s, size)) != TMM_OK)
    return rc;
  if (scale == nullptr || (reinterpret_cast<uintptr_t>(scale) & 3u))
    return fail(TMM_ERR_INVALID_ARG, "%s: scale is NULL or not 4-byte aligned", who);
  if (rows == 0 || N == 0) return TMM_OK;
  const size_t need = K > 0 ? tmm::lora_workspace_bytes(p) : 0;
  if ((rc = check_workspace(who, need, workspace, workspace_bytes)) != TMM_OK) return rc;
  const Bytes out[9] = {{"y", y, stack_span(y_s) * size},
                        {"x", x, stack_span(p.x) * size},
                        {"w", w, stack_span(p.w) * size},
                        {"a", a, stack_span(p.a) * size},
                        {"b", b, stack_span(p.b) * size},
                        {"offsets", offsets, (groups + 1) * 4},
                        {"row_index", row_index, rows * 4},
                        {"scale", scale, groups * 4},
                        {"the workspace", workspace, int64_t(need)}};
  const Bytes ws[8] = {out[8], out[1], out[2], out[3], out[4], out[5], out[6], out[7]};
  if ((rc = check_alias(who, out, 9)) != TMM_OK || (rc = check_alias(who, ws, 8)) != TMM_OK)
    return rc;
  tmm::DeviceInfo dev;
  if ((rc = current_device(&dev)) != TMM_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) return zero_output(who, y, 1, rows, N, ldy, 0, size, s);
  p.scale = scale;
  p.y = y;
  p.ldy = ldy;
  const cudaError_t e = tmm::launch_lora(p, dev, workspace, s);
  if (e != cudaSuccess) return fail(TMM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return TMM_OK;
}

// ---- rows of scores -----------------------------------------------------------------------

namespace {

// A row-major matrix of scores: rows below 2^29, as the grids and 32-bit columns need.
int check_scores(const char *who, const char *name, int dtype, int64_t rows, int64_t cols,
                 const void *data, int64_t ld) {
  if (dtype != TMM_F32 && dtype != TMM_BF16 && dtype != TMM_F16)
    return fail(TMM_ERR_INVALID_ARG, "%s: unknown dtype %d", who, dtype);
  if (!extent_ok(rows) || !extent_ok(cols))
    return fail(TMM_ERR_INVALID_ARG, "%s: sizes must be >= 0 and below 2^29 (%lld x %lld)", who,
                (long long)rows, (long long)cols);
  return check_stack(who, name, stack_of(data, 1, rows, cols, ld, 0), element_size(dtype));
}

int64_t scores_bytes(int dtype, int64_t rows, int64_t cols, int64_t ld) {
  return stack_span(stack_of(nullptr, 1, rows, cols, ld, 0)) * element_size(dtype);
}

// Arrays of 4-byte values (or, with `size`, others): there and naturally aligned.
int check_array(const char *who, const char *name, const void *p, int64_t n, int size = 4) {
  if (n > 0 && p == nullptr) return fail(TMM_ERR_INVALID_ARG, "%s: %s is NULL", who, name);
  if (reinterpret_cast<uintptr_t>(p) % unsigned(size))
    return fail(TMM_ERR_INVALID_ARG, "%s: %s must be %d-byte aligned", who, name, size);
  return TMM_OK;
}

int check_scale(const char *who, float scale, bool positive) {
  if (!(scale - scale == 0.0f) || (positive && !(scale > 0.0f)))
    return fail(TMM_ERR_INVALID_ARG, "%s: scale must be finite%s", who,
                positive ? " and positive" : "");
  return TMM_OK;
}

// The `outs` arrays first in `r` are written: each against all after it.
int check_outputs(const char *who, const Bytes *r, int outs, int count) {
  for (int i = 0; i < outs; ++i) {
    if (r[i].p == nullptr) continue;
    const int rc = check_alias(who, r + i, count - i);
    if (rc != TMM_OK) return rc;
  }
  return TMM_OK;
}

int check_route(const char *who, int64_t experts, int64_t k, int score, int renormalise) {
  if (experts < 1 || experts > tmm::kMaxExperts)
    return fail(TMM_ERR_INVALID_ARG, "%s: need 1 <= experts <= %d (experts=%lld)", who,
                tmm::kMaxExperts, (long long)experts);
  if (k < 1 || k > tmm::kMaxFan || k > experts)
    return fail(TMM_ERR_INVALID_ARG, "%s: need 1 <= k <= min(%d, experts) (k=%lld)", who,
                tmm::kMaxFan, (long long)k);
  if (score != TMM_SOFTMAX && score != TMM_SIGMOID)
    return fail(TMM_ERR_INVALID_ARG, "%s: unknown score %d", who, score);
  if (renormalise != 0 && renormalise != 1)
    return fail(TMM_ERR_INVALID_ARG, "%s: renormalise must be 0 or 1", who);
  return TMM_OK;
}

int check_logprob(const char *who, int top, int token_bits, const void *tokens, float scale) {
  if (top < 0 || top > tmm::kMaxTop)
    return fail(TMM_ERR_INVALID_ARG, "%s: need 0 <= top <= %d (top=%d)", who, tmm::kMaxTop, top);
  if (token_bits != 32 && token_bits != 64)
    return fail(TMM_ERR_INVALID_ARG, "%s: token_bits must be 32 or 64", who);
  if (reinterpret_cast<uintptr_t>(tokens) % unsigned(token_bits / 8))
    return fail(TMM_ERR_INVALID_ARG, "%s: tokens must be naturally aligned", who);
  return check_scale(who, scale, true);
}

}  // namespace

int route_rows(int dtype, int64_t tokens, int64_t experts, const void *logits, int64_t ld,
               const float *bias, int score, int64_t groups, int64_t top_groups, int group_best,
               int64_t k, int renormalise, float scale, int32_t *chosen, float *weights,
               tmm_stream_t stream) {
  const char *who = "route_rows";
  int rc;
  if ((rc = check_scores(who, "logits", dtype, tokens, experts, logits, ld)) != TMM_OK ||
      (rc = check_route(who, experts, k, score, renormalise)) != TMM_OK ||
      (rc = check_scale(who, scale, false)) != TMM_OK)
    return rc;
  if (groups < 1 || groups > tmm::kMaxRouteGroups || experts % groups != 0 || top_groups < 1 ||
      top_groups > groups)
    return fail(TMM_ERR_INVALID_ARG, "%s: need groups <= %d that divide the experts, and 1 <= "
                "top_groups <= groups (groups=%lld top_groups=%lld)", who, tmm::kMaxRouteGroups,
                (long long)groups, (long long)top_groups);
  if (group_best != 1 && group_best != 2)
    return fail(TMM_ERR_INVALID_ARG, "%s: group_best must be 1 or 2", who);
  if (k > experts / groups * top_groups)
    return fail(TMM_ERR_INVALID_ARG, "%s: k=%lld experts of %lld in the chosen groups", who,
                (long long)k, (long long)(experts / groups * top_groups));
  if ((rc = check_array(who, "bias", bias, 0)) != TMM_OK ||
      (rc = check_array(who, "chosen", chosen, tokens)) != TMM_OK ||
      (rc = check_array(who, "weights", weights, tokens)) != TMM_OK)
    return rc;
  if (tokens == 0) return TMM_OK;
  const Bytes all[4] = {{"chosen", chosen, tokens * k * 4},
                        {"weights", weights, tokens * k * 4},
                        {"logits", logits, scores_bytes(dtype, tokens, experts, ld)},
                        {"bias", bias, experts * 4}};
  if ((rc = check_outputs(who, all, 2, 4)) != TMM_OK) return rc;
  tmm::DeviceInfo dev;
  if ((rc = current_device(&dev)) != TMM_OK) return rc;
  tmm::RouteProblem p = {};
  p.dtype = dtype;
  p.tokens = tokens;
  p.experts = int(experts);
  p.k = int(k);
  p.logits = logits;
  p.ld = ld;
  p.bias = bias;
  p.sigmoid = score == TMM_SIGMOID;
  p.renormalise = renormalise;
  p.groups = int(groups);
  p.top_groups = int(top_groups);
  p.best = group_best;
  p.scale = scale;
  p.chosen = chosen;
  p.weights = weights;
  const cudaError_t e = tmm::launch_route(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(TMM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return TMM_OK;
}

int route_rows_grad(int dtype, int64_t tokens, int64_t experts, int64_t k, const float *dweights,
                    const void *logits, int64_t ld, const int32_t *chosen, int score,
                    int renormalise, float scale, void *dlogits, int64_t ldd,
                    tmm_stream_t stream) {
  const char *who = "route_rows_grad";
  int rc;
  if ((rc = check_scores(who, "logits", dtype, tokens, experts, logits, ld)) != TMM_OK ||
      (rc = check_scores(who, "dlogits", dtype, tokens, experts, dlogits, ldd)) != TMM_OK ||
      (rc = check_route(who, experts, k, score, renormalise)) != TMM_OK ||
      (rc = check_scale(who, scale, false)) != TMM_OK ||
      (rc = check_array(who, "dweights", dweights, tokens)) != TMM_OK ||
      (rc = check_array(who, "chosen", chosen, tokens)) != TMM_OK)
    return rc;
  if (tokens == 0) return TMM_OK;
  const bool in_place = dlogits == logits && ldd == ld;
  const Bytes all[4] = {{"dlogits", dlogits, scores_bytes(dtype, tokens, experts, ldd)},
                        {"dweights", dweights, tokens * k * 4},
                        {"chosen", chosen, tokens * k * 4},
                        {"logits", in_place ? nullptr : logits,
                         scores_bytes(dtype, tokens, experts, ld)}};
  if ((rc = check_outputs(who, all, 1, 4)) != TMM_OK) return rc;
  tmm::DeviceInfo dev;
  if ((rc = current_device(&dev)) != TMM_OK) return rc;
  tmm::RouteGradProblem p = {};
  p.dtype = dtype;
  p.tokens = tokens;
  p.experts = int(experts);
  p.k = int(k);
  p.dweights = dweights;
  p.logits = logits;
  p.ld = ld;
  p.chosen = chosen;
  p.sigmoid = score == TMM_SIGMOID;
  p.renormalise = renormalise;
  p.scale = scale;
  p.dlogits = dlogits;
  p.ldd = ldd;
  const cudaError_t e = tmm::launch_route_grad(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(TMM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return TMM_OK;
}

int logprob_rows(int dtype, int64_t rows, int64_t cols, const void *logits, int64_t ld,
                 float scale, const void *tokens, int token_bits, int top, float *logprob,
                 float *entropy, float *lse, int32_t *top_ids, float *top_logprobs,
                 tmm_stream_t stream) {
  const char *who = "logprob_rows";
  int rc;
  if ((rc = check_scores(who, "logits", dtype, rows, cols, logits, ld)) != TMM_OK ||
      (rc = check_logprob(who, top, token_bits, tokens, scale)) != TMM_OK ||
      (rc = check_array(who, "logprob", logprob, tokens ? rows : 0)) != TMM_OK ||
      (rc = check_array(who, "entropy", entropy, rows)) != TMM_OK ||
      (rc = check_array(who, "lse", lse, rows)) != TMM_OK ||
      (rc = check_array(who, "top_ids", top_ids, rows * top)) != TMM_OK ||
      (rc = check_array(who, "top_logprobs", top_logprobs, rows * top)) != TMM_OK)
    return rc;
  if (logprob != nullptr && tokens == nullptr && rows > 0)
    return fail(TMM_ERR_INVALID_ARG, "%s: logprob without tokens", who);
  if (rows == 0) return TMM_OK;
  const Bytes all[7] = {{"logprob", logprob, rows * 4},
                        {"entropy", entropy, rows * 4},
                        {"lse", lse, rows * 4},
                        {"top_ids", top_ids, rows * top * 4},
                        {"top_logprobs", top_logprobs, rows * top * 4},
                        {"logits", logits, scores_bytes(dtype, rows, cols, ld)},
                        {"tokens", tokens, rows * (token_bits / 8)}};
  if ((rc = check_outputs(who, all, 5, 7)) != TMM_OK) return rc;
  tmm::DeviceInfo dev;
  if ((rc = current_device(&dev)) != TMM_OK) return rc;
  const tmm::LogprobProblem p = {dtype, rows,  cols,    logits,  ld,  tokens,  token_bits,
                                 top,   scale, logprob, entropy, lse, top_ids, top_logprobs};
  const cudaError_t e = tmm::launch_logprob(p, dev, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(TMM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return TMM_OK;
}

int logprob_rows_grad(int dtype, int64_t rows, int64_t cols, const void *logits, int64_t ld,
                      float scale, const float *lse, const void *tokens, int token_bits,
                      const float *dlogprob, const float *entropy, const float *dentropy, int top,
                      const int32_t *top_ids, const float *dtop, void *dlogits, int64_t ldd,
                      tmm_stream_t stream) {
  const char *who = "logprob_rows_grad";
  int rc;
  if ((rc = check_scores(who, "logits", dtype, rows, cols, logits, ld)) != TMM_OK ||
      (rc = check_scores(who, "dlogits", dtype, rows, cols, dlogits, ldd)) != TMM_OK ||
      (rc = check_logprob(who, top, token_bits, tokens, scale)) != TMM_OK ||
      (rc = check_array(who, "lse", lse, rows)) != TMM_OK ||
      (rc = check_array(who, "dlogprob", dlogprob, 0)) != TMM_OK ||
      (rc = check_array(who, "tokens", tokens, dlogprob ? rows : 0)) != TMM_OK ||
      (rc = check_array(who, "dentropy", dentropy, 0)) != TMM_OK ||
      (rc = check_array(who, "entropy", entropy, dentropy ? rows : 0)) != TMM_OK ||
      (rc = check_array(who, "top_ids", top_ids, rows * top)) != TMM_OK ||
      (rc = check_array(who, "dtop", dtop, rows * top)) != TMM_OK)
    return rc;
  if (rows == 0 || cols == 0) return TMM_OK;
  const bool in_place = dlogits == logits && ldd == ld;
  const Bytes all[9] = {{"dlogits", dlogits, scores_bytes(dtype, rows, cols, ldd)},
                        {"logits", in_place ? nullptr : logits,
                         scores_bytes(dtype, rows, cols, ld)},
                        {"lse", lse, rows * 4},
                        {"tokens", tokens, rows * (token_bits / 8)},
                        {"dlogprob", dlogprob, rows * 4},
                        {"entropy", entropy, rows * 4},
                        {"dentropy", dentropy, rows * 4},
                        {"top_ids", top_ids, rows * top * 4},
                        {"dtop", dtop, rows * top * 4}};
  if ((rc = check_outputs(who, all, 1, 9)) != TMM_OK) return rc;
  tmm::DeviceInfo dev;
  if ((rc = current_device(&dev)) != TMM_OK) return rc;
  tmm::LogprobGradProblem p = {};
  p.dtype = dtype;
  p.rows = rows;
  p.cols = cols;
  p.logits = logits;
  p.ld = ld;
  p.tokens = tokens;
  p.token_bits = token_bits;
  p.top = top;
  p.scale = scale;
  p.lse = lse;
  p.entropy = entropy;
  p.dlogprob = dlogprob;
  p.dentropy = dentropy;
  p.top_ids = top_ids;
  p.dtop = top > 0 ? dtop : nullptr;
  p.dlogits = dlogits;
  p.ldd = ldd;
  const cudaError_t e = tmm::launch_logprob_grad(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(TMM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return TMM_OK;
}

// ---- linear layers --------------------------------------------------------------------------

namespace {

int check_linear(const char *who, int dtype, int trans, int act, int64_t M, int64_t N, int64_t K) {
  if (dtype != TMM_F32 && dtype != TMM_BF16 && dtype != TMM_F16)
    return fail(TMM_ERR_INVALID_ARG, "%s: unknown dtype %d", who, dtype);
  if (trans != 0 && trans != 1)
    return fail(TMM_ERR_INVALID_ARG, "%s: transw must be 0 or 1", who);
  if (act < TMM_ACT_NONE || act > TMM_ACT_GELU_TANH)
    return fail(TMM_ERR_INVALID_ARG, "%s: unknown activation %d", who, act);
  if (!extent_ok(M) || !extent_ok(N) || !extent_ok(K))
    return fail(TMM_ERR_INVALID_ARG, "%s: sizes must be >= 0 and below 2^29 (M=%lld N=%lld K=%lld)",
                who, (long long)M, (long long)N, (long long)K);
  return TMM_OK;
}

tmm::LinearProblem linear_problem(int dtype, int transw, int64_t M, int64_t N, int64_t K,
                                  const void *x, int64_t ldx, const void *w, int64_t ldw) {
  tmm::LinearProblem p = {};
  p.dtype = dtype;
  p.rows = M;
  p.K = K;
  p.N = N;
  p.x = stack_of(x, 1, M, K, ldx, 0);
  p.w = stack_of(w, 1, transw ? N : K, transw ? K : N, ldw, 0);
  p.trans_w = transw;
  return p;
}

// An optional matrix: nothing to check where it is NULL.
int check_optional(const char *who, const char *name, const void *m, int64_t rows, int64_t cols,
                   int64_t ld, int size) {
  if (m == nullptr) return TMM_OK;
  return check_stack(who, name, stack_of(m, 1, rows, cols, ld, 0), size);
}

int64_t matrix_bytes(const void *m, int64_t rows, int64_t cols, int64_t ld, int size) {
  return m == nullptr ? 0 : stack_span(stack_of(m, 1, rows, cols, ld, 0)) * size;
}

}  // namespace

size_t gemm_bias_act_workspace_size(int dtype, int transw, int64_t M, int64_t N, int64_t K,
                                    const void *x, int64_t ldx, const void *w, int64_t ldw) {
  if (!extent_ok(M) || !extent_ok(N) || !extent_ok(K) || M == 0 || N == 0 || K == 0) return 0;
  return tmm::linear_workspace_bytes(linear_problem(dtype, transw, M, N, K, x, ldx, w, ldw));
}

int gemm_bias_act(int dtype, int transw, int act, int64_t M, int64_t N, int64_t K, const void *x,
                  int64_t ldx, const void *w, int64_t ldw, const void *bias, int bias_f32,
                  const void *residual, int64_t ldr, void *y, int64_t ldy, void *pre,
                  int64_t ldpre, void *workspace, size_t workspace_bytes, tmm_stream_t stream) {
  const char *who = "gemm_bias_act";
  int rc = check_linear(who, dtype, transw, act, M, N, K);
  if (rc != TMM_OK) return rc;
  tmm::LinearProblem p = linear_problem(dtype, transw, M, N, K, x, ldx, w, ldw);
  const int size = element_size(dtype), bias_size = bias_f32 ? 4 : size;
  if (bias_f32 != 0 && bias_f32 != 1)
    return fail(TMM_ERR_INVALID_ARG, "%s: bias_f32 must be 0 or 1", who);
  if ((rc = check_stack(who, "x", p.x, size)) != TMM_OK ||
      (rc = check_stack(who, "w", p.w, size)) != TMM_OK ||
      (rc = check_stack(who, "y", stack_of(y, 1, M, N, ldy, 0), size)) != TMM_OK ||
      (rc = check_optional(who, "residual", residual, M, N, ldr, size)) != TMM_OK ||
      (rc = check_optional(who, "pre", pre, M, N, ldpre, size)) != TMM_OK ||
      (rc = check_array(who, "bias", bias, 0, bias_size)) != TMM_OK)
    return rc;
  if (M == 0 || N == 0) return TMM_OK;
  const size_t need = tmm::linear_workspace_bytes(p);
  if ((rc = check_workspace(who, need, workspace, workspace_bytes)) != TMM_OK) return rc;
  const bool in_place = y == residual && ldy == ldr;
  const Bytes all[7] = {{"y", y, matrix_bytes(y, M, N, ldy, size)},
                        {"pre", pre, matrix_bytes(pre, M, N, ldpre, size)},
                        {"the workspace", need ? workspace : nullptr, int64_t(need)},
                        {"x", x, stack_span(p.x) * size},
                        {"w", w, stack_span(p.w) * size},
                        {"bias", bias, bias ? N * bias_size : 0},
                        {"residual", residual, matrix_bytes(residual, M, N, ldr, size)}};
  if ((rc = check_alias(who, all, in_place ? 6 : 7)) != TMM_OK ||
      (rc = check_outputs(who, all + 1, 2, 6)) != TMM_OK)
    return rc;
  tmm::DeviceInfo dev;
  if ((rc = current_device(&dev)) != TMM_OK) return rc;
  p.act = act;
  p.bias = bias;
  p.bias_f32 = bias_f32;
  p.residual = residual;
  p.ld_residual = ldr;
  p.y = y;
  p.ldy = ldy;
  p.pre = pre;
  p.ld_pre = ldpre;
  const cudaError_t e =
      tmm::launch_linear(p, dev, workspace, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(TMM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return TMM_OK;
}

namespace {

tmm::LinearGradProblem linear_grad_problem(int dtype, int transw, int act, int64_t M, int64_t N,
                                           int64_t K, const void *dy, int64_t lddy, const void *x,
                                           int64_t ldx, const void *w, int64_t ldw,
                                           const void *pre, int64_t ldpre, void *dx, int64_t lddx,
                                           void *dw, int64_t lddw, int transdw, float *dbias) {
  tmm::LinearGradProblem p = {};
  p.dtype = dtype;
  p.act = act;
  p.rows = M;
  p.K = K;
  p.N = N;
  p.dy = stack_of(dy, 1, M, N, lddy, 0);
  p.x = stack_of(x, 1, M, K, ldx, 0);
  p.w = stack_of(w, 1, transw ? N : K, transw ? K : N, ldw, 0);
  p.trans_w = transw;
  p.pre = pre;
  p.ld_pre = ldpre;
  p.dx = K > 0 ? dx : nullptr;
  p.lddx = lddx;
  p.dw = K > 0 ? dw : nullptr;
  p.lddw = lddw;
  p.trans_dw = transdw;
  p.dbias = dbias;
  return p;
}

}  // namespace

size_t gemm_bias_act_grad_workspace_size(int dtype, int transw, int act, int64_t M, int64_t N,
                                         int64_t K, const void *dy, int64_t lddy, const void *x,
                                         int64_t ldx, const void *w, int64_t ldw, const void *dx,
                                         const void *dw, int transdw, const void *dbias) {
  if (!extent_ok(M) || !extent_ok(N) || !extent_ok(K) || M == 0 || N == 0) return 0;
  return tmm::linear_grad_workspace_bytes(linear_grad_problem(
      dtype, transw, act, M, N, K, dy, lddy, x, ldx, w, ldw, nullptr, 1, const_cast<void *>(dx), 1,
      const_cast<void *>(dw), 1, transdw, static_cast<float *>(const_cast<void *>(dbias))));
}

int gemm_bias_act_grad(int dtype, int transw, int act, int64_t M, int64_t N, int64_t K,
                       const void *dy, int64_t lddy, const void *x, int64_t ldx, const void *w,
                       int64_t ldw, const void *pre, int64_t ldpre, void *dx, int64_t lddx,
                       void *dw, int64_t lddw, int transdw, float *dbias, void *workspace,
                       size_t workspace_bytes, tmm_stream_t stream) {
  const char *who = "gemm_bias_act_grad";
  int rc = check_linear(who, dtype, transw, act, M, N, K);
  if (rc != TMM_OK) return rc;
  if (transdw != 0 && transdw != 1)
    return fail(TMM_ERR_INVALID_ARG, "%s: transdw must be 0 or 1", who);
  if (act != TMM_ACT_NONE && pre == nullptr && M > 0 && N > 0)
    return fail(TMM_ERR_INVALID_ARG, "%s: pre is NULL", who);
  const tmm::LinearGradProblem p =
      linear_grad_problem(dtype, transw, act, M, N, K, dy, lddy, x, ldx, w, ldw, pre, ldpre, dx,
                          lddx, dw, lddw, transdw, dbias);
  const int size = element_size(dtype);
  const int64_t wr = transdw ? N : K, wc = transdw ? K : N;      // of dw
  if ((rc = check_stack(who, "dy", p.dy, size)) != TMM_OK ||
      (rc = check_optional(who, "pre", pre, M, N, ldpre, size)) != TMM_OK ||
      (rc = check_optional(who, "dx", dx, M, K, lddx, size)) != TMM_OK ||
      (rc = check_optional(who, "dw", dw, wr, wc, lddw, size)) != TMM_OK ||
      (rc = check_array(who, "dbias", dbias, 0)) != TMM_OK ||
      (dw && (rc = check_stack(who, "x", p.x, size)) != TMM_OK) ||
      (dx && (rc = check_stack(who, "w", p.w, size)) != TMM_OK))
    return rc;
  const size_t need = M == 0 || N == 0 ? 0 : tmm::linear_grad_workspace_bytes(p);
  if ((rc = check_workspace(who, need, workspace, workspace_bytes)) != TMM_OK) return rc;
  const Bytes all[8] = {{"dx", dx, matrix_bytes(dx, M, K, lddx, size)},
                        {"dw", dw, matrix_bytes(dw, wr, wc, lddw, size)},
                        {"dbias", dbias, dbias ? N * 4 : 0},
                        {"the workspace", need ? workspace : nullptr, int64_t(need)},
                        {"dy", dy, stack_span(p.dy) * size},
                        {"x", dw ? x : nullptr, stack_span(p.x) * size},
                        {"w", dx ? w : nullptr, stack_span(p.w) * size},
                        {"pre", pre, matrix_bytes(pre, M, N, ldpre, size)}};
  if ((rc = check_outputs(who, all, 4, 8)) != TMM_OK) return rc;
  if ((M == 0 || K == 0 || dx == nullptr) && (N == 0 || K == 0 || dw == nullptr) &&
      (N == 0 || dbias == nullptr))
    return TMM_OK;
  tmm::DeviceInfo dev;
  if ((rc = current_device(&dev)) != TMM_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0 || N == 0) {      // empty sums
    if (dx && M > 0 && K > 0 &&
        (rc = zero_output(who, dx, 1, M, K, lddx, 0, size, s)) != TMM_OK)
      return rc;
    if (dw && N > 0 && K > 0 &&
        (rc = zero_output(who, dw, 1, wr, wc, lddw, 0, size, s)) != TMM_OK)
      return rc;
    return dbias && N > 0 ? zero_output(who, dbias, 1, 1, N, N, 0, 4, s) : TMM_OK;
  }
  const cudaError_t e = tmm::launch_linear_grad(p, dev, workspace, s);
  if (e != cudaSuccess) return fail(TMM_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return TMM_OK;
}

const char *tmm_last_error_string(void) { return g_last_error; }

const char *gemm_last_error_string(void) { return g_last_error; }

int gemm_check_status(tmm_stream_t stream) { return tmm_check_device(stream); }

int tmm_version(void) { return 100; }

}  // extern "C"
