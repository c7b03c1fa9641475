// logprob_rows.cu -- log probabilities of given tokens, with the rows' entropies and most probable
// tokens, and their gradient.
//
//   x = scale l,  lse = log sum_v e^(x_v),  logprob = x_t - lse,
//   entropy = -sum_v p_v log p_v = log S - (sum_v e^(x_v - M) (x_v - M)) / S,  S = sum_v e^(x_v - M),
// with M the row's maximum: one pass over the logits with a running (M, S, W), W the sum of
// e^(x - M) (x - M).  When the maximum rises by D = M' - M both are scaled by e^-D, and W becomes
// e^-D (W - D S).  Exponents are those of two, t = (l - M) c, c = scale log2(e): the difference first,
// which no logits overflow (rows masked by the type's lowest value) and which keeps log S apart from
// M until the end.
//
// Reading the logits is the bound: each value costs about eight instructions.  A block does a row; where rows are few
// a cluster of up to eight does, and its first block adds up what the others have in their shared
// memory.  Sums are added in a fixed order.
//
// The most probable: every warp keeps a sorted list of 32 keys, a lane each (a key: the value's
// bits in the order of unsigned numbers, then the number's complement, so that the larger key is
// the larger value or the lower number).  Its n-th is a threshold that a vector's maximum, which is
// needed anyway, is compared with, and so is, for all of the block's warps, what the lanes' running
// maxima imply: of each of w warps ceil(n / w) lanes have reached the least of the warps' ceil(n / w)-th
// largest.  Few values of a row are then ever inserted (131072 columns, 20 listed: about 20 a warp;
// with thresholds of the warps' own lists alone, 32 rows took 21 us in place of TOP_US).  Lists are
// merged pair by pair (half-cleaner and five exchange steps).
//
// Gradient: dl_v = scale (g ([v = t] - p_v) - h p_v (log p_v + entropy) + sum_j e_j ([v = id_j] - p_v))
// for the gradients g, h and e_j of the row's log probability, entropy and alternatives: one read and
// one write.
#include <atomic>
#include <cstdint>

#include "row_ops.cuh"
#include "rows.h"
#include "tmm_gemm.h"

namespace tmm {
namespace {

constexpr int kMaxThreads = 256, kMaxCluster = 8;
constexpr int kAhead = 4;          // vectors of a thread in flight
constexpr unsigned kAll = ~0u;
constexpr uint64_t kNoKey = 0;

__device__ __forceinline__ uint32_t order_of(float v) {      // v is not NaN
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float v, uint32_t at) {
  return uint64_t(order_of(v)) << 32 | uint32_t(~at);
}
__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }

template <typename T>
__device__ __forceinline__ uint32_t lowest_bits();      // -inf, in every value of a word
template <>
__device__ __forceinline__ uint32_t lowest_bits<float>() { return 0xFF800000u; }
template <>
__device__ __forceinline__ uint32_t lowest_bits<__nv_bfloat16>() { return 0xFF80FF80u; }
template <>
__device__ __forceinline__ uint32_t lowest_bits<__half>() { return 0xFC00FC00u; }

// The largest of a vector's values, NaN left out.
__device__ __forceinline__ float max_of(const Vec<float> &v) {
  return fmaxf(fmaxf(v.get(0), v.get(1)), fmaxf(v.get(2), v.get(3)));
}
__device__ __forceinline__ float max_of(const Vec<__nv_bfloat16> &v) {
  const __nv_bfloat162 *const w = reinterpret_cast<const __nv_bfloat162 *>(&v.w);
  const __nv_bfloat162 a = __hmax2(__hmax2(w[0], w[1]), __hmax2(w[2], w[3]));
  return fmaxf(float(a.x), float(a.y));
}
__device__ __forceinline__ float max_of(const Vec<__half> &v) {
  const __half2 *const w = reinterpret_cast<const __half2 *>(&v.w);
  const __half2 a = __hmax2(__hmax2(w[0], w[1]), __hmax2(w[2], w[3]));
  return fmaxf(float(a.x), float(a.y));
}

// The running statistics, in exponents of two.
struct Stats {
  float m, s, w;
  __device__ __forceinline__ float base() const { return m == -INFINITY ? 0.0f : m; }
  // To the maximum `to` >= m.
  __device__ __forceinline__ void raise(float to, float c) {
    const float d = m == -INFINITY ? 0.0f : fmaxf((m - to) * c, -1000.0f);
    const float f = exp2_approx(d);
    w = f * fmaf(d, s, w);
    s *= f;
    m = to;
  }
  __device__ __forceinline__ void join(Stats o, float c) {
    const float to = fmaxf(m, o.m);
    raise(to, c);
    o.raise(to, c);
    s += o.s;
    w += o.w;
  }
  __device__ __forceinline__ void join_warp(float c) {
    float to = m;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) to = fmaxf(to, __shfl_xor_sync(kAll, to, d));
    raise(to, c);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      s += __shfl_xor_sync(kAll, s, d);
      w += __shfl_xor_sync(kAll, w, d);
    }
  }
};
// One value's terms (of -inf: 0).
__device__ __forceinline__ void add_term(float x, float base, float c, float &s, float &w) {
  const float t = (x - base) * c, e = exp2_approx(t);
  s += e;
  w = fmaf(e, fmaxf(t, -1000.0f), w);
}

// A warp's n best keys so far, sorted, a lane each.
struct Best {
  uint64_t key;        // of this lane
  uint64_t low;        // keys up to it need not be looked at
  float low_value;
  int n;
  __device__ __forceinline__ void raise_low(uint64_t to) {
    if (to > low) {
      low = to;
      low_value = value_of(uint32_t(low >> 32));
    }
  }
  // One lane's value, every lane's in turn.
  __device__ __forceinline__ void offer(float v, uint32_t at) {
    const int lane = threadIdx.x & 31;
    const uint64_t mine = v >= low_value ? key_of(v, at) : kNoKey;      // (NaN: no key)
    unsigned want = __ballot_sync(kAll, mine > low);
    if (want == 0) return;
    do {
      const int from = __ffs(int(want)) - 1;
      want &= want - 1;
      const uint64_t k = __shfl_sync(kAll, mine, from);
      if (k <= low) continue;
      const int place = __popc(__ballot_sync(kAll, key > k));
      const uint64_t above = __shfl_up_sync(kAll, key, 1);
      key = lane < place ? key : lane == place ? k : above;
      raise_low(__shfl_sync(kAll, key, n - 1));
    } while (want);
  }
  // The each-th largest of the lanes' values (in their order's numbers, 0: none), each the warps' equal
  // share of n: the least of the warps' is one that at least n values of the row reach.
  __device__ __forceinline__ uint32_t share(float v, int each) const {
    uint32_t mine = v > -INFINITY ? order_of(v) : 0, top = 0;
    for (int j = 0; j < each; ++j) {
      top = __reduce_max_sync(kAll, mine);
      if ((threadIdx.x & 31) == unsigned(__ffs(int(__ballot_sync(kAll, mine == top))) - 1)) mine = 0;
    }
    return top;
  }
  // With another sorted list, given as its key 31 - lane.
  __device__ __forceinline__ void merge(uint64_t reversed) {
    const int lane = threadIdx.x & 31;
    key = larger(key, reversed);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const uint64_t other = __shfl_xor_sync(kAll, key, d);
      const bool first = (lane & d) == 0;
      key = first == (key > other) ? key : other;
    }
  }
};

__device__ __forceinline__ uint32_t shared_address(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint32_t in_block(uint32_t addr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float cluster_float(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t cluster_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ int64_t token_of(const void *tokens, int bits, int64_t row) {
  return bits == 64 ? static_cast<const int64_t *>(tokens)[row]
                    : int64_t(static_cast<const int32_t *>(tokens)[row]);
}

// Elements before the first 16-byte boundary of a row of `cols`.
template <typename T>
__device__ __forceinline__ int head_of(const T *row, int64_t cols) {
  const int n = int((16 - (reinterpret_cast<uintptr_t>(row) & 15u)) & 15u) / int(sizeof(T));
  return int(min(int64_t(n), cols));
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kMaxThreads)
logprob_kernel(const __grid_constant__ LogprobProblem p, int cluster) {
  constexpr int W = Vec<T>::kCount;
  constexpr int kWarps = kMaxThreads / 32;
  __shared__ float part[3][kWarps];
  __shared__ uint64_t lists[TOP ? kWarps : 1][32];
  __shared__ uint32_t reached[kWarps];      // by the lanes of each warp, see Best::share
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int threads = blockDim.x, warps = threads >> 5;
  const int64_t row = blockIdx.x / cluster;
  const int rank = int(blockIdx.x - row * cluster);
  wait_then_start_next();

  const T *const from = static_cast<const T *>(p.logits) + row * p.ld;
  const int cols = int(p.cols);
  const float c = p.scale * kLog2e;
  // The given token's logit, early.
  float at_token = 0.0f;
  bool given = false;
  if (rank == 0 && tid == 0 && p.tokens) {
    const int64_t t = token_of(p.tokens, p.token_bits, row);
    given = t >= 0 && t < p.cols;
    if (given) at_token = as_float(from[t]);
  }
  const int head = head_of(from, p.cols), vectors = (cols - head) / W;
  const int v0 = int(int64_t(vectors) * rank / cluster);
  const int v1 = int(int64_t(vectors) * (rank + 1) / cluster);
  const uint4 *const body = reinterpret_cast<const uint4 *>(from + head);

  Stats st = {-INFINITY, 0.0f, 0.0f};
  Best best;
  if (TOP) {
    best.key = kNoKey;
    best.low = uint64_t(order_of(-3.402823466e38f)) << 32;      // values of -inf are not listed
    best.low_value = -3.402823466e38f;
    best.n = p.top;
  }
  const auto fetch = [&](int first, Vec<T> (&v)[kAhead]) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = first + u * threads + tid;
      const uint32_t b = lowest_bits<T>();
      v[u].w = make_uint4(b, b, b, b);
      if (i < v1) v[u].w = __ldg(body + i);
    }
  };
  const int step = kAhead * threads;
  const int each = TOP ? (p.top + warps - 1) / warps : 0;
  bool first_batch = true;
  Vec<T> next[kAhead];
  fetch(v0, next);
  // Every warp makes the same number of rounds, so that its lanes stay together.
  for (int i0 = v0; i0 < v1; i0 += step) {
    Vec<T> v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) v[u] = next[u];
    fetch(i0 + step, next);
    float top[kAhead], most = -INFINITY;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      top[u] = max_of(v[u]);
      most = fmaxf(most, top[u]);
    }
    if (TOP) {
      const uint32_t mine = best.share(fmaxf(st.m, most), each);
      if (lane == 0) *const_cast<volatile uint32_t *>(&reached[warp]) = mine;
      if (first_batch) __syncthreads();
      first_batch = false;
      // (What another warp has reached by now is reached for good: an older value will do.)
      const uint32_t all = __reduce_min_sync(
          kAll, lane < warps ? *const_cast<volatile uint32_t *>(&reached[lane]) : ~0u);
      best.raise_low(uint64_t(all) << 32);
      if (__any_sync(kAll, most >= best.low_value)) {
#pragma unroll 1
        for (int u = 0; u < kAhead; ++u) {
          float t = top[0];
          Vec<T> x = v[0];
#pragma unroll
          for (int k = 1; k < kAhead; ++k)
            if (u == k) {
              t = top[k];
              x = v[k];
            }
          if (!__any_sync(kAll, t >= best.low_value)) continue;
          const uint32_t at = uint32_t(head + (i0 + u * threads + tid) * W);
#pragma unroll
          for (int k = 0; k < W; ++k) best.offer(x.get(k), at + k);
        }
      }
    }
    st.raise(fmaxf(st.m, most), c);
    const float base = st.base();
    float s2 = 0.0f, w2 = 0.0f;      // half of the terms, for shorter chains
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int k = 0; k < W; k += 2) {
        add_term(v[u].get(k), base, c, st.s, st.w);
        add_term(v[u].get(k + 1), base, c, s2, w2);
      }
    st.s += s2;
    st.w += w2;
  }
  if (rank == 0 && warp == 0) {
    // The elements before the first vector and after the last, fewer than two vectors' worth.
    const int tail = head + vectors * W, ends = head + cols - tail;
    const int i = lane < head ? lane : tail + lane - head;
    const float x = lane < ends ? as_float(from[i]) : -INFINITY;
    if (TOP) best.offer(x, uint32_t(i));
    st.raise(fmaxf(st.m, x), c);
    add_term(x, st.base(), c, st.s, st.w);
  }
  st.join_warp(c);
  if (lane == 0) {
    part[0][warp] = st.m;
    part[1][warp] = st.s;
    part[2][warp] = st.w;
  }
  if (TOP) lists[warp][lane] = best.key;
  __syncthreads();
  if (TOP) {
    // Pairs of warps, then pairs of those.
    for (int d = 1; d < warps; d *= 2) {
      const bool on = warp % (2 * d) == 0 && warp + d < warps;
      if (on) {
        best.merge(lists[warp + d][31 - lane]);
        lists[warp][lane] = best.key;
      }
      __syncthreads();
    }
  }
  if (cluster > 1) {
    cluster_barrier();
    if (TOP && rank == 0) {
      // Warp w takes the lists of blocks w, w + warps, ...; then as above.
      best.key = kNoKey;
      for (int r = warp; r < cluster; r += warps)
        best.merge(cluster_u64(in_block(shared_address(&lists[0][31 - lane]), r)));
      __syncthreads();      // lists[0] has been read
      lists[warp][lane] = best.key;
      __syncthreads();
      for (int d = 1; d < warps; d *= 2) {
        if (warp % (2 * d) == 0 && warp + d < warps) {
          best.merge(lists[warp + d][31 - lane]);
          lists[warp][lane] = best.key;
        }
        __syncthreads();
      }
    }
  }
  if (rank == 0 && warp == 0) {
    Stats all = {-INFINITY, 0.0f, 0.0f};
    for (int i = lane; i < cluster * warps; i += 32) {
      const int r = i / warps, w = i - r * warps;
      Stats o;
      if (cluster == 1) {
        o = {part[0][w], part[1][w], part[2][w]};
      } else {
        o.m = cluster_float(in_block(shared_address(&part[0][w]), r));
        o.s = cluster_float(in_block(shared_address(&part[1][w]), r));
        o.w = cluster_float(in_block(shared_address(&part[2][w]), r));
      }
      all.join(o, c);
    }
    all.join_warp(c);
    const float log_s = logf(all.s);
    const bool bad = !(all.s == all.s), nothing = all.s == 0.0f;
    const float nan = __uint_as_float(0x7FFFFFFFu);
    const float lse = bad ? nan : nothing ? -INFINITY : fmaf(all.m, p.scale, log_s);
    if (lane == 0) {
      p.lse[row] = lse;
      p.entropy[row] =
          bad ? nan : nothing ? 0.0f : fmaxf(0.0f, log_s - kLn2 * (all.w / all.s));
      if (p.logprob) {
        float lp = 0.0f;
        if (given) lp = bad ? nan : nothing ? -INFINITY : (at_token - all.m) * p.scale - log_s;
        p.logprob[row] = lp;
      }
    }
    if (TOP && lane < p.top) {
      const bool have = best.key != kNoKey && !bad;
      const float v = value_of(uint32_t(best.key >> 32));
      p.top_ids[row * p.top + lane] = have ? int(~uint32_t(best.key)) : -1;
      p.top_logprobs[row * p.top + lane] =
          bad ? nan : have ? (v - all.m) * p.scale - log_s : -INFINITY;
    }
  }
  if (cluster > 1) cluster_barrier();      // the others' shared memory has been read
}

// ---- gradient ------------------------------------------------------------------------------

// A block does `threads` x kAhead vectors of a row (`pieces` of them make a row).
template <typename T, bool TOP, bool VEC>
__global__ void __launch_bounds__(kMaxThreads)
logprob_grad_kernel(const __grid_constant__ LogprobGradProblem p, int pieces) {
  constexpr int W = VEC ? Vec<T>::kCount : 1;
  __shared__ int ids[kMaxTop];
  __shared__ float adds[kMaxTop];
  __shared__ int listed;
  wait_then_start_next();
  const int tid = threadIdx.x, lane = tid & 31, threads = blockDim.x;
  const int64_t row = blockIdx.x / pieces;
  const int piece = int(blockIdx.x - row * pieces);
  const T *const from = static_cast<const T *>(p.logits) + row * p.ld;
  T *const to = static_cast<T *>(p.dlogits) + row * p.ldd;
  const int cols = int(p.cols);
  // Element i of the row is at vector (i - head) / W; the vectors start at a 16-byte boundary of
  // both rows, and what is left at the row's ends is done one by one by the first piece.
  const int head = VEC ? head_of(from, p.cols) : 0, vectors = (cols - head) / W;
  const int first = piece * threads * kAhead;

  const float lse = p.lse[row];
  const float h = p.dentropy ? p.dentropy[row] : 0.0f;
  const float entropy = p.dentropy ? p.entropy[row] : 0.0f;
  int token = -1;
  float g = 0.0f;
  if (p.dlogprob) {
    const int64_t t = token_of(p.tokens, p.token_bits, row);
    if (t >= 0 && t < p.cols) {
      token = int(t);
      g = p.dlogprob[row];
    }
  }
  float sum = g;
  if (TOP) {
    int id = -1;
    float e = 0.0f;
    if (lane < p.top) {
      id = p.top_ids[row * p.top + lane];
      if (id >= cols) id = -1;
      if (id >= 0) e = p.dtop[row * p.top + lane];
    }
    float all = e;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) all += __shfl_xor_sync(kAll, all, d);
    sum += all;
    if (tid < 32) {
      // Those of this block's vectors, or at the ends.
      const int v = (id - head) / W - first;
      const bool ends = id < head || id >= head + vectors * W;
      const bool here = id >= 0 && (ends ? piece == 0 : v >= 0 && v < threads * kAhead);
      const unsigned mask = __ballot_sync(kAll, here);
      if (here) {
        const int at = __popc(mask & ((1u << lane) - 1));
        ids[at] = id;
        adds[at] = e;
      }
      if (lane == 0) listed = __popc(mask);
    }
    __syncthreads();
  }
  const int count = TOP ? listed : 0;
  const bool nothing = lse == -INFINITY;                   // no value of the row is visible
  const bool dense = !nothing && (sum != 0.0f || h != 0.0f);
  if (nothing) token = -1;
  const auto slope = [&](float x) {
    const float lp = fmaf(x, p.scale, -lse), e = exp2_approx(lp * kLog2e);
    return -e * fmaf(h, fmaxf(lp, -1000.0f) + entropy, sum);
  };
  const auto finish = [&](float d, int i) {
    if (i == token) d += g;
    if (TOP && !nothing)
      for (int k = 0; k < count; ++k) d += ids[k] == i ? adds[k] : 0.0f;
    return d * p.scale;
  };
  if (VEC) {
    Vec<T> v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = first + u * threads + tid;
      if (dense && i < vectors) v[u].w = *reinterpret_cast<const uint4 *>(from + head + i * W);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = first + u * threads + tid, at = head + i * W;
      if (i >= vectors) continue;
      float d[W];
#pragma unroll
      for (int k = 0; k < W; ++k) d[k] = dense ? slope(v[u].get(k)) : 0.0f;
      bool special = unsigned(token - at) < unsigned(W);
      for (int k = 0; k < count; ++k) special |= unsigned(ids[k] - at) < unsigned(W);
      if (special) {
#pragma unroll
        for (int k = 0; k < W; ++k) d[k] = finish(d[k], at + k);
      } else {
#pragma unroll
        for (int k = 0; k < W; ++k) d[k] *= p.scale;
      }
      Vec<T> out;
#pragma unroll
      for (int k = 0; k < W; ++k) out.set(k, d[k]);
      *reinterpret_cast<uint4 *>(to + at) = out.w;
    }
    if (piece == 0) {
      const int tail = head + vectors * W, ends = head + cols - tail;
      if (tid < ends) {
        const int i = tid < head ? tid : tail + tid - head;
        to[i] = rounded<T>(finish(dense ? slope(as_float(from[i])) : 0.0f, i));
      }
    }
  } else {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = first + u * threads + tid;
      if (i < cols) to[i] = rounded<T>(finish(dense ? slope(as_float(from[i])) : 0.0f, i));
    }
  }
}

int round_threads(int64_t want) {
  return int(std::min<int64_t>(kMaxThreads, std::max<int64_t>(32, (want + 31) / 32 * 32)));
}

template <typename T>
cudaError_t launch_logprob_as(const LogprobProblem &p, const DeviceInfo &dev, cudaStream_t stream) {
  const int64_t rounds = (p.cols / Vec<T>::kCount + kAhead - 1) / kAhead;     // of one thread
  const int threads = round_threads(rounds);
  // Blocks of a row: twice as many blocks as there are SMs, a round of loads each at least.
  int cluster = 1;
  while (cluster < kMaxCluster && p.rows * cluster < 2 * dev.sm_count &&
         rounds >= 2 * cluster * threads)
    cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(unsigned(p.rows * cluster), 1, 1);
  cfg.blockDim = dim3(unsigned(threads), 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return p.top ? cudaLaunchKernelEx(&cfg, logprob_kernel<T, true>, p, cluster)
               : cudaLaunchKernelEx(&cfg, logprob_kernel<T, false>, p, cluster);
}

template <typename T>
cudaError_t launch_logprob_grad_as(const LogprobGradProblem &p, cudaStream_t stream) {
  // Vectors where the rows of both matrices are equally far from a 16-byte boundary.
  const bool vec = ((reinterpret_cast<uintptr_t>(p.logits) ^ reinterpret_cast<uintptr_t>(p.dlogits)) &
                    15u) == 0 && (p.ld - p.ldd) * int64_t(sizeof(T)) % 16 == 0;
  const int64_t units = vec ? p.cols / Vec<T>::kCount : p.cols;
  const int threads = round_threads((units + kAhead - 1) / kAhead);
  const int64_t pieces = std::max<int64_t>(1, (units + threads * kAhead - 1) / (threads * kAhead));
  if (p.rows * pieces > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(unsigned(p.rows * pieces), 1, 1);
  cfg.blockDim = dim3(unsigned(threads), 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kernel = p.dtop ? (vec ? logprob_grad_kernel<T, true, true>
                                    : logprob_grad_kernel<T, true, false>)
                             : (vec ? logprob_grad_kernel<T, false, true>
                                    : logprob_grad_kernel<T, false, false>);
  return cudaLaunchKernelEx(&cfg, kernel, p, int(pieces));
}

}  // namespace

cudaError_t launch_logprob(const LogprobProblem &p, const DeviceInfo &dev, cudaStream_t stream) {
  if (p.dtype == TMM_BF16) return launch_logprob_as<__nv_bfloat16>(p, dev, stream);
  if (p.dtype == TMM_F16) return launch_logprob_as<__half>(p, dev, stream);
  return launch_logprob_as<float>(p, dev, stream);
}

cudaError_t launch_logprob_grad(const LogprobGradProblem &p, const DeviceInfo &,
                                cudaStream_t stream) {
  if (p.dtype == TMM_BF16) return launch_logprob_grad_as<__nv_bfloat16>(p, stream);
  if (p.dtype == TMM_F16) return launch_logprob_grad_as<__half>(p, stream);
  return launch_logprob_grad_as<float>(p, stream);
}

}  // namespace tmm
