// route_rows.cu -- routing to experts: the k best experts of every token, and their weights.
//
//   s = softmax(l) or sigmoid(l) over a row's logits l,  c = s + bias,
//   the groups' values: the sum of a group's one or two best c,
//   the k best c among the experts of the best groups (ties: the lower number),
//   w_j = scale s_j / sum of the chosen s, or scale s_j.
// The choice is that of the scores in 64 bits.  Without a bias the logits stand for the scores
// (both functions are increasing), which is exact.  Otherwise c is computed in 32 bits with an
// error below `tol`, and a row in which two values that decide something are closer than that is
// done again in 64 bits: one row in a hundred at 256 experts, where 64 bits for all rows would take
// the FP64 units about 100 times the reading of the logits.
//
// A warp does a row, all of whose values stay in registers: with G groups rounded up to a power of
// two every group has 32 / G lanes, so that a group's best are a butterfly within its lanes.  The
// choice is k rounds of two warp reductions of the redux unit (the best value's bits in an order
// that unsigned numbers have, then the lowest number that has it).
// Gradient: w depends on the chosen logits alone, but for the softmax without renormalisation;
// rows are written whole, 16 bytes a lane.
#include <atomic>
#include <cstdint>

#include "rows.h"
#include "row_ops.cuh"
#include "tmm_gemm.h"

namespace tmm {
namespace {

constexpr int kWarps = 4;      // rows of a block
constexpr unsigned kAll = ~0u;

// Values as unsigned numbers in the same order, 0 for none; NaN is the largest, -0 equals 0.
__device__ __forceinline__ uint32_t key_of(float c) {
  const uint32_t b = __float_as_uint(c + 0.0f);
  return c != c ? ~0u : b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(double c) {
  const uint64_t b = uint64_t(__double_as_longlong(c + 0.0));
  return c != c ? ~uint64_t(0) : b >> 63 ? ~b : b | uint64_t(1) << 63;
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const uint64_t o = __shfl_xor_sync(kAll, v, d);
    v = o > v ? o : v;
  }
  return v;
}
template <typename C>
__device__ __forceinline__ C warp_sum(C v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
  return v;
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }
__device__ __forceinline__ double sigmoid(double l) { return 1.0 / (1.0 + exp(-l)); }
__device__ __forceinline__ float exp_of(float t) { return expf(t); }
__device__ __forceinline__ double exp_of(double t) { return exp(t); }

// A lane's experts: numbers first + v * step for v < V, where v * step + sub < size.
struct Lane {
  int first, step, sub, size, group;
  __device__ __forceinline__ bool has(int v) const { return v * step + sub < size; }
  __device__ __forceinline__ int expert(int v) const { return first + v * step; }
};
__device__ __forceinline__ Lane lane_of(const RouteProblem &p, int lane, bool vec) {
  Lane a;
  a.group = lane / p.lanes;
  const int sub = lane - a.group * p.lanes;
  if (vec) {       // every lane has V of them, one after another
    const int each = p.group_size / p.lanes;
    a.step = 1;
    a.sub = sub * each;
  } else {
    a.step = p.lanes;
    a.sub = sub;
  }
  a.first = a.group * p.group_size + a.sub;
  a.size = a.group < p.groups ? p.group_size : 0;
  return a;
}

// The choice of a row: lane j < k leaves with expert j, or -1.  `close`: two values that decide
// something are too close to tell (never in 64 bits).  l: this lane's logits, -inf where it has none.
template <typename T, typename C, int V>
__device__ __forceinline__ int choose(const RouteProblem &p, int64_t row, const Lane &a,
                                      const float (&l)[V], bool &close) {
  constexpr bool exact = sizeof(C) == 8;
  const int lane = threadIdx.x & 31;
  const float *const bias = p.bias;
  C c[V], m = 0;
  bool on[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    c[v] = C(l[v]);
    on[v] = l[v] != -INFINITY;
  }
  if (!p.sigmoid && (bias || p.best == 2)) {
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) top = fmaxf(top, l[v]);
    m = C(warp_max(top));
  }
  if (bias) {
    if (p.sigmoid) {
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = sigmoid(c[v]);
    } else {
      C sum = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        c[v] = on[v] ? exp_of(c[v] - m) : C(0);
        sum += c[v];
      }
      sum = warp_sum(sum);
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] /= sum;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float b = a.has(v) ? bias[a.expert(v)] : 0.0f;
      on[v] &= b != -INFINITY;
      c[v] += C(b);
    }
  }
  bool open = true;
  close = false;
  if (p.groups > 1) {
    C one = -INFINITY, two = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (on[v]) {
        const C low = c[v] < one ? c[v] : one;
        one = c[v] > one ? c[v] : one;
        two = low > two ? low : two;
      }
    for (int d = 1; d < p.lanes; d <<= 1) {
      const C o = __shfl_xor_sync(kAll, one, d), t = __shfl_xor_sync(kAll, two, d);
      const C low = o < one ? o : one;
      one = o > one ? o : one;
      two = t > two ? t : two;
      two = low > two ? low : two;
    }
    const bool any = one != C(-INFINITY);
    C value = one;
    if (p.best == 2 && any) {
      if (!bias && p.sigmoid)
        value = sigmoid(one) + sigmoid(two);
      else if (!bias)
        value = exp_of(one - m) + exp_of(two - m);
      else if (two != C(-INFINITY))
        value = one + two;
    }
    const auto key = any && a.size > 0 ? key_of(value) : key_of(C(0)) * 0;
    int rank = 0;
    for (int h = 0; h < p.groups; ++h) {
      const auto other = __shfl_sync(kAll, key, h * p.lanes);
      rank += other > key || (other == key && h < a.group);
    }
    open = key != 0 && rank < p.top_groups;
    if (!exact && (bias || p.best == 2)) {
      // The last group taken against the first that is not.
      float lo = open ? float(value) : INFINITY, hi = key != 0 && !open ? float(value) : -INFINITY;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(kAll, lo, d));
        hi = fmaxf(hi, __shfl_xor_sync(kAll, hi, d));
      }
      const float tol = bias ? 0x1p-17f + 0x1p-21f * fabsf(hi) : 0x1p-16f * hi + 1e-37f;
      close = hi != -INFINITY && lo - hi <= tol;
    }
  }
  decltype(key_of(C(0))) key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) key[v] = on[v] && open ? key_of(c[v]) : 0;
  // With a bias one round more, to see what the last one chosen was taken before.
  const bool check = !exact && bias;
  const int rounds = p.k + (check ? 1 : 0);
  int mine = -1;
  decltype(key_of(C(0))) mine_key = 0;
  for (int j = 0; j < rounds; ++j) {
    auto best = key[0];
    int at = 0;
#pragma unroll
    for (int v = 1; v < V; ++v)
      if (key[v] > best) {
        best = key[v];
        at = v;
      }
    const auto top = warp_max(best);
    if (top == 0) break;
    const int e = int(__reduce_min_sync(
        kAll, best == top ? unsigned(a.first + at * a.step) : unsigned(INT32_MAX)));
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (a.first + v * a.step == e && a.has(v)) key[v] = 0;
    if (lane == j) {
      mine = e;
      mine_key = top;
    }
  }
  if constexpr (!exact) {
    if (check) {
      const auto value = [](uint32_t k) {
        return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
      };
      const uint32_t next_key = __shfl_down_sync(kAll, mine_key, 1);
      const int next = __shfl_down_sync(kAll, mine, 1);
      const bool pair = lane < p.k && next >= 0 && lane < 31;
      const float x = value(mine_key), gap = x - value(next_key);
      bool near = pair && gap <= 0x1p-18f + 0x1p-22f * fabsf(x);
      if (__any_sync(kAll, near)) {
        if (near) {
          // Equal logits with equal biases are equal, and their numbers decide.
          const T *const at = static_cast<const T *>(p.logits) + row * p.ld;
          near = float(at[mine]) != float(at[next]) || bias[mine] != bias[next];
        }
        close |= __any_sync(kAll, near);
      }
    }
  }
  return lane < p.k ? mine : -1;
}

template <typename T, int V>
__device__ __forceinline__ void load_logits(const RouteProblem &p, int64_t row, const Lane &a,
                                            bool vec, float (&l)[V]) {
  const T *const from = static_cast<const T *>(p.logits) + row * p.ld;
  constexpr int kVec = Vec<T>::kCount;
  if constexpr (V >= kVec) {
    if (vec) {
      if (a.size == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) l[v] = -INFINITY;
        return;
      }
      Vec<T> w[V / kVec];
#pragma unroll
      for (int i = 0; i < V / kVec; ++i)
        w[i].w = *reinterpret_cast<const uint4 *>(from + a.first + i * kVec);
#pragma unroll
      for (int v = 0; v < V; ++v) l[v] = w[v / kVec].get(v % kVec);
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = a.has(v) ? as_float(from[a.expert(v)]) : -INFINITY;
}

// In 64 bits; apart from the kernel's usual way, whose registers it would take.
template <typename T, int V>
__device__ __noinline__ int choose_again(const RouteProblem &p, int64_t row, bool vec) {
  const Lane a = lane_of(p, threadIdx.x & 31, vec);
  float l[V];
  load_logits<T, V>(p, row, a, vec, l);
  bool close;
  return choose<T, double, V>(p, row, a, l, close);
}

// The chosen scores of a row over their sum, as lane j has logit x of slot j (-inf: none), 0 where
// every one is 0; or alone.  `m`, `sum`: of the softmax over all experts.
__device__ __forceinline__ float score_of(bool is_sigmoid, bool renormalise, float x, float m,
                                          float sum) {
  const bool none = x == -INFINITY;
  if (!renormalise) {
    if (none) return 0.0f;
    return is_sigmoid ? sigmoid(x) : expf(x - m) / sum;
  }
  // The sum is at least 1 for the softmax, and for a sigmoid below e^-60, which is e^x but for a
  // factor of 1 + e^-60, the same.
  const float top = warp_max(x != x ? INFINITY : x);
  float s = 0.0f;
  if (!none) s = is_sigmoid && !(top < -60.0f) ? sigmoid(x) : expf(x - top);
  const float total = warp_sum(s);
  return none ? 0.0f : s / total;
}

template <typename T, int V>
__global__ void __launch_bounds__(32 * kWarps)
route_kernel(const __grid_constant__ RouteProblem p) {
  wait_then_start_next();
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= p.tokens) return;
  const bool vec = p.vec;
  const Lane a = lane_of(p, lane, vec);
  float l[V];
  load_logits<T, V>(p, row, a, vec, l);
  bool close;
  int e = choose<T, float, V>(p, row, a, l, close);
  if (close) e = choose_again<T, V>(p, row, vec);
  float m = 0.0f, sum = 1.0f;
  if (!p.sigmoid && !p.renormalise) {
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) top = l[v] != l[v] ? l[v] : fmaxf(top, l[v]);
    m = warp_max(top);
    sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) sum += l[v] == -INFINITY ? 0.0f : expf(l[v] - m);
    sum = warp_sum(sum);
  }
  const float x =
      e >= 0 ? as_float(static_cast<const T *>(p.logits)[row * p.ld + e]) : -INFINITY;
  const float w = score_of(p.sigmoid, p.renormalise, x, m, sum);
  if (lane < p.k) {
    p.chosen[row * p.k + lane] = e;
    p.weights[row * p.k + lane] = e >= 0 ? p.scale * w : 0.0f;
  }
}

// ---- gradient ------------------------------------------------------------------------------

// Lane l has experts (32 i + l) W .. + W of piece i, W a vector's values or one.
template <typename T, int V, bool VEC>
__global__ void __launch_bounds__(32 * kWarps)
route_grad_kernel(const __grid_constant__ RouteGradProblem p) {
  constexpr int W = VEC ? Vec<T>::kCount : 1;
  constexpr int kPieces = (V + W - 1) / W;
  wait_then_start_next();
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= p.tokens) return;
  const T *const from = static_cast<const T *>(p.logits) + row * p.ld;
  T *const to = static_cast<T *>(p.dlogits) + row * p.ldd;
  int e = lane < p.k ? p.chosen[row * p.k + lane] : -1;
  if (e >= p.experts) e = -1;
  const float x = e >= 0 ? as_float(from[e]) : -INFINITY;
  const float g = e >= 0 ? p.scale * p.dweights[row * p.k + lane] : 0.0f;
  const bool dense = !p.sigmoid && !p.renormalise;

  float l[kPieces][W], m = 0.0f, sum = 1.0f;
  if (dense) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int first = (32 * i + lane) * W;
      if constexpr (VEC) {
        Vec<T> w;
        if (first < p.experts) w.w = *reinterpret_cast<const uint4 *>(from + first);
#pragma unroll
        for (int c = 0; c < W; ++c) l[i][c] = first < p.experts ? w.get(c) : -INFINITY;
      } else {
        l[i][0] = first < p.experts ? as_float(from[first]) : -INFINITY;
      }
#pragma unroll
      for (int c = 0; c < W; ++c) top = fmaxf(top, l[i][c]);
    }
    m = warp_max(top);
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
#pragma unroll
      for (int c = 0; c < W; ++c) {
        l[i][c] = l[i][c] == -INFINITY ? 0.0f : expf(l[i][c] - m);
        sum += l[i][c];
      }
    sum = warp_sum(sum);
  }
  const float s = score_of(p.sigmoid, p.renormalise, x, m, sum);
  // The slots' part, and (softmax over all) the sum that every expert's score takes.
  const float dot = dense || p.renormalise ? warp_sum(s * g) : 0.0f;
  float d;
  if (dense)
    d = s * g;
  else
    d = s * (g - dot) * (p.sigmoid ? sigmoid(-x) : 1.0f);
  const float r = dense ? -dot / sum : 0.0f;
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
#pragma unroll
    for (int c = 0; c < W; ++c) l[i][c] = dense && l[i][c] != 0.0f ? l[i][c] * r : 0.0f;
  for (int j = 0; j < p.k; ++j) {
    const int at = __shfl_sync(kAll, e, j);
    const float add = __shfl_sync(kAll, d, j);
    if (at < 0) continue;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
#pragma unroll
      for (int c = 0; c < W; ++c)
        if ((32 * i + lane) * W + c == at) l[i][c] += add;
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int first = (32 * i + lane) * W;
    if (first >= p.experts) continue;
    if constexpr (VEC) {
      Vec<T> w;
#pragma unroll
      for (int c = 0; c < W; ++c) w.set(c, l[i][c]);
      *reinterpret_cast<uint4 *>(to + first) = w.w;
    } else {
      to[first] = rounded<T>(l[i][0]);
    }
  }
}

template <typename P>
cudaError_t launch_rows(void (*kernel)(P), const P &p, int64_t tokens, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(unsigned((tokens + kWarps - 1) / kWarps), 1, 1);
  cfg.blockDim = dim3(32 * kWarps, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T>
cudaError_t launch_route_as(RouteProblem p, cudaStream_t stream) {
  // Every group on 32 / G lanes, G rounded up to a power of two; all groups taken is no grouping.
  if (p.top_groups == p.groups) p.groups = 1;
  int across = 1;
  while (across < p.groups) across *= 2;
  p.group_size = p.experts / p.groups;
  p.lanes = 32 / across;
  const int need = (p.group_size + p.lanes - 1) / p.lanes;      // at most 32
  int V = 1;
  while (V < need) V *= 2;
  p.vec = p.group_size == V * p.lanes && V * sizeof(T) % 16 == 0 &&
          (reinterpret_cast<uintptr_t>(p.logits) & 15u) == 0 && p.ld * sizeof(T) % 16 == 0;
  switch (V) {
    case 1: return launch_rows(route_kernel<T, 1>, p, p.tokens, stream);
    case 2: return launch_rows(route_kernel<T, 2>, p, p.tokens, stream);
    case 4: return launch_rows(route_kernel<T, 4>, p, p.tokens, stream);
    case 8: return launch_rows(route_kernel<T, 8>, p, p.tokens, stream);
    case 16: return launch_rows(route_kernel<T, 16>, p, p.tokens, stream);
    default: return launch_rows(route_kernel<T, 32>, p, p.tokens, stream);
  }
}

template <typename T>
cudaError_t launch_grad_as(const RouteGradProblem &p, cudaStream_t stream) {
  const bool vec = p.experts * sizeof(T) % 16 == 0 && p.ld * sizeof(T) % 16 == 0 &&
                   p.ldd * sizeof(T) % 16 == 0 &&
                   ((reinterpret_cast<uintptr_t>(p.logits) | reinterpret_cast<uintptr_t>(p.dlogits)) &
                    15u) == 0;
  if (vec) {
    if (p.experts <= 128) return launch_rows(route_grad_kernel<T, 4, true>, p, p.tokens, stream);
    if (p.experts <= 256) return launch_rows(route_grad_kernel<T, 8, true>, p, p.tokens, stream);
    return launch_rows(route_grad_kernel<T, 16, true>, p, p.tokens, stream);
  }
  if (p.experts <= 128) return launch_rows(route_grad_kernel<T, 4, false>, p, p.tokens, stream);
  return launch_rows(route_grad_kernel<T, 16, false>, p, p.tokens, stream);
}

}  // namespace

cudaError_t launch_route(const RouteProblem &p, cudaStream_t stream) {
  if (p.dtype == TMM_BF16) return launch_route_as<__nv_bfloat16>(p, stream);
  if (p.dtype == TMM_F16) return launch_route_as<__half>(p, stream);
  return launch_route_as<float>(p, stream);
}

cudaError_t launch_route_grad(const RouteGradProblem &p, cudaStream_t stream) {
  if (p.dtype == TMM_BF16) return launch_grad_as<__nv_bfloat16>(p, stream);
  if (p.dtype == TMM_F16) return launch_grad_as<__half>(p, stream);
  return launch_grad_as<float>(p, stream);
}

}  // namespace tmm
