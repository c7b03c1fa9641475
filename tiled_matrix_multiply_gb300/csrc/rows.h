// rows.h -- declarations of the operators over rows of scores: routing to experts and log
// probabilities.  Not part of the public ABI (that is include/tmm_gemm.h).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "tmm_internal.h"

namespace tmm {

constexpr int kMaxExperts = 512, kMaxFan = 16, kMaxRouteGroups = 32, kMaxTop = 32;

// The experts of every token (see route_rows in tmm_gemm.h).
struct RouteProblem {
  int dtype;
  int64_t tokens;
  int experts, k;
  const void *logits;
  int64_t ld;
  const float *bias;            // experts, or NULL
  int sigmoid, renormalise;
  int groups, top_groups, best; // best: values of a group that are added to its own
  float scale;
  int32_t *chosen;              // tokens x k
  float *weights;               // tokens x k
  int group_size, lanes, lanes_log2, vec_bias;      // set by the launcher: lanes of a group, 16-byte loads
};
struct RouteGradProblem {
  int dtype;
  int64_t tokens;
  int experts, k;
  const float *dweights;        // tokens x k
  const void *logits;
  int64_t ld;
  const int32_t *chosen;        // tokens x k
  int sigmoid, renormalise;
  float scale;
  void *dlogits;
  int64_t ldd;
};
// Sizes reaching a launcher are > 0.
cudaError_t launch_route(const RouteProblem &p, cudaStream_t stream);
cudaError_t launch_route_grad(const RouteGradProblem &p, cudaStream_t stream);

// Log probabilities of given tokens (see logprob_rows in tmm_gemm.h).
struct LogprobProblem {
  int dtype;
  int64_t rows, cols;
  const void *logits;
  int64_t ld;
  const void *tokens;           // rows, 32- or 64-bit; NULL: none
  int token_bits;
  int top;
  float scale;
  float *logprob, *entropy, *lse;      // rows; logprob NULL without tokens
  int32_t *top_ids;             // rows x top
  float *top_logprobs;
};
struct LogprobGradProblem {
  int dtype;
  int64_t rows, cols;
  const void *logits;
  int64_t ld;
  const void *tokens;
  int token_bits;
  int top;
  float scale;
  const float *lse, *entropy;
  const float *dlogprob, *dentropy;    // rows, or NULL
  const int32_t *top_ids;              // rows x top
  const float *dtop;
  void *dlogits;
  int64_t ldd;
};
cudaError_t launch_logprob(const LogprobProblem &p, const DeviceInfo &dev, cudaStream_t stream);
cudaError_t launch_logprob_grad(const LogprobGradProblem &p, cudaStream_t stream);

}  // namespace tmm
