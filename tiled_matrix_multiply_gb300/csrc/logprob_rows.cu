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
// Reading the logits is the bound, each value costs about eight instructions (4096 x 131072, bf16: 161 us,
// 6.65 TB/s).  A block does a row; where rows are many and short a warp does, and where they are few a
// cluster of up to eight blocks, whose first adds up what the others have in their shared memory (32 x
// 131072: 4.9 us, with 20 listed 11.1).  Sums are added in a fixed order.
//
// The most probable: the pass keeps the largest value of every thread, and of each of up to 16 pieces of
// what it reads.  Of w warps, ceil(n / w) threads each reach the least of the warps' ceil(n / w)-th
// largest; not many more values do than are listed, and only the pieces that do are read again.  What
// reaches that bound there (as keys: the value's bits in the order of unsigned numbers, then the number's
// complement, so that the larger key is the larger value or the lower number) is put in order by counting
// for each how many are larger.  So the pass is the one without alternatives, and the selection comes
// after it.  Rows of which too many values reach the bound (thousands of equal ones) are read again
// whole, by lists that are kept sorted: rows of equal logits (4096 x 131072 with 20 listed 2140 us, 32 rows 28),
// and those whose visible values lie in fewer threads' vectors than the bound is made of, the rest the type's
// lowest value (40 values far apart: as equal ones; a run of 2 % of the row: 214 and 28; with -inf in place
// of the lowest value 215 and 10).  (With such lists in the pass itself, under thresholds of various
// kinds, 4096 rows of 131072 with 20 listed took 320 to 520 us, 213 now; the pass alone takes 161, the
// memory's time.)
//
// Gradient: dl_v = scale (g ([v = t] - p_v) - h p_v (log p_v + entropy) + sum_j e_j ([v = id_j] - p_v))
// for the gradients g, h and e_j of the row's log probability, entropy and alternatives: one read and
// one write are the bound (4096 x 65536, bf16, a tenth of the rows without gradients, which are not read:
// 150 us, 6.80 TB/s; 515 x 50001, FP32: 32 us, 6.4 TB/s).
#include <algorithm>
#include <cstdint>

#include "row_ops.cuh"
#include "rows.h"
#include "tmm_gemm.h"

namespace tmm {
namespace {

constexpr int kMaxThreads = 256, kMaxCluster = 8;
constexpr int kAhead = 4;          // vectors of a thread in flight
constexpr int kPieces = 16;        // of what a thread reads, see the most probable
constexpr int kFound = 1024;       // keys that may be listed, of a block's rows
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

// A warp's best keys, sorted, a lane each.
struct Best {
  uint64_t key;
  // Exchanges with the lane `d` away: the larger key to the first of the two, or (not `down`) the other.
  __device__ __forceinline__ static uint64_t exchanged(uint64_t k, int d, bool down) {
    const uint64_t other = __shfl_xor_sync(kAll, k, d);
    const bool first = ((threadIdx.x & d) == 0) == down;
    return first == (k > other) ? k : other;
  }
  // With another sorted list, given as its key 31 - lane.
  __device__ __forceinline__ void merge(uint64_t reversed) {
    key = larger(key, reversed);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) key = exchanged(key, d, true);
  }
  // With a key of every lane (bitonic, upwards: a list's key 31 - lane).
  __device__ __forceinline__ void add(uint64_t k) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
      for (int d = size / 2; d > 0; d >>= 1) k = exchanged(k, d, (lane & size) != 0 && size < 32);
    merge(k);
  }
};

// The values, the largest in lane 0.
__device__ __forceinline__ float sorted_down(float v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int d = size / 2; d > 0; d >>= 1) {
      const float o = __shfl_xor_sync(kAll, v, d);
      v = ((lane & d) == 0) == ((lane & size) == 0) ? fmaxf(v, o) : fminf(v, o);
    }
  return v;
}

// Puts the 32 largest of `count` keys (none twice, but kNoKey) where their order says; thread `tid` of
// `threads`.
__device__ __forceinline__ void place(const uint64_t *keys, int count, uint64_t *list, int tid,
                                      int threads) {
  for (int i = tid; i < count; i += threads) {
    const uint64_t k = keys[i];
    int before = 0;
#pragma unroll 4
    for (int j = 0; j < count; ++j) before += keys[j] > k;
    if (k != kNoKey && before < 32) list[before] = k;
  }
}

// The n best keys of elements [begin, end) of a row, those of `stride` warps' turn: any values.
template <typename T>
__device__ __noinline__ uint64_t scan_whole(const T *row, int64_t begin, int64_t end, int stride,
                                            int n) {
  const int lane = threadIdx.x & 31;
  Best best = {kNoKey};
  uint64_t low = kNoKey;
  for (int64_t i = begin; i < end; i += 32 * stride) {
    const float x = i + lane < end ? as_float(row[i + lane]) : -INFINITY;
    const uint64_t k = x > -INFINITY ? key_of(x, uint32_t(i + lane)) : kNoKey;
    if (!__any_sync(kAll, k > low)) continue;
    best.add(k);
    low = __shfl_sync(kAll, best.key, n - 1);
  }
  return best.key;
}

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

// ONE: a warp does a row, eight a block.
template <typename T, bool TOP, bool ONE>
__global__ void __launch_bounds__(kMaxThreads)
logprob_kernel(const __grid_constant__ LogprobProblem p, int cluster) {
  constexpr int W = Vec<T>::kCount;
  constexpr int kWarps = kMaxThreads / 32;
  __shared__ float part[3][kWarps];
  __shared__ uint64_t lists[TOP ? kWarps : 1][32];
  // What every warp has reached, the largest value of each of a thread's pieces, and what may be listed.
  __shared__ float most_of[kWarps];
  __shared__ float piece_of[TOP ? kPieces : 1][kMaxThreads];
  __shared__ uint64_t found[TOP ? kFound : 1];
  __shared__ int founds[kWarps];
  // ONE: of the row's only warp, from here on.
  const int lane = threadIdx.x & 31, warp = ONE ? 0 : threadIdx.x >> 5;
  const int tid = ONE ? lane : threadIdx.x;
  const int threads = ONE ? 32 : blockDim.x, warps = ONE ? 1 : threads >> 5;
  const int64_t row = ONE ? int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5)
                          : int64_t(blockIdx.x / cluster);
  const int rank = ONE ? 0 : int(blockIdx.x - row * cluster);
  wait_then_start_next();
  if (ONE && row >= p.rows) return;

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
  const auto fetch = [&](int first, Vec<T> (&v)[kAhead]) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = first + u * threads + tid;
      const uint32_t b = lowest_bits<T>();
      v[u].w = make_uint4(b, b, b, b);
      if (i < v1) v[u].w = body[i];
    }
  };
  const int step = kAhead * threads;
  // Rounds of loads in a piece, and the piece so far.
  const int rounds = TOP ? (v1 - v0 + step - 1) / step : 0;
  const int in_piece = TOP ? max(1, (rounds + kPieces - 1) / kPieces) : 1;
  int piece = 0, left = in_piece;
  float piece_most = -INFINITY, even = -INFINITY, odd = -INFINITY;      // (of every other vector)
  Vec<T> next[kAhead];
  fetch(v0, next);
  // Every warp makes the same number of rounds, so that its lanes stay together.
  for (int i0 = v0; i0 < v1; i0 += step) {
    Vec<T> v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) v[u] = next[u];
    fetch(i0 + step, next);
    float most = -INFINITY;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) most = fmaxf(most, max_of(v[u]));
    if (TOP && ONE) {
#pragma unroll
      for (int u = 0; u < kAhead; u += 2) {
        even = fmaxf(even, max_of(v[u]));
        odd = fmaxf(odd, max_of(v[u + 1]));
      }
    }
    if (TOP) {
      piece_most = fmaxf(piece_most, most);
      piece_of[piece][threadIdx.x] = piece_most;
      if (--left == 0) {
        left = in_piece;
        piece_most = -INFINITY;
        ++piece;
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
  // The elements before the first vector and after the last, fewer than two vectors' worth.
  const int tail = head + vectors * W, ends = rank == 0 && warp == 0 ? head + cols - tail : 0;
  const int end_at = lane < head ? lane : tail + lane - head;
  const float x = lane < ends ? as_float(from[end_at]) : -INFINITY;
  const float thread_most = st.m;      // of the vectors
  if (ends > 0) {
    st.raise(fmaxf(st.m, x), c);
    add_term(x, st.base(), c, st.s, st.w);
  }
  if constexpr (TOP) {
    const auto together = [] {
      if (ONE) __syncwarp();
      else __syncthreads();
    };
    const int own = ONE ? threadIdx.x >> 5 : 0, base = threadIdx.x - lane;
    const int room = ONE ? kFound / kWarps : kFound;
    uint64_t *const mine = found + own * room, *const list = lists[own];
    if (tid == 0) founds[own] = 0;
    if (tid < 32) list[tid] = kNoKey;
    // ceil(n / w) threads of every one of w warps reach the least of the warps' ceil(n / w)-th largest.
    const int each = (p.top + warps - 1) / warps;
    const float reached = __shfl_sync(kAll, sorted_down(thread_most), each - 1);
    float bound = reached;
    if (ONE && p.top > 20) {
      // Many values reach the least of nearly all of a warp's maxima: 130 of any row that of 32, on the
      // mean, and 128 have room.  Half as many of each of two maxima a thread: 50 do (8192 x 1000, 32
      // listed, 61 and 20 us).
      const int half = (p.top + 1) / 2;
      bound = fminf(__shfl_sync(kAll, sorted_down(even), half - 1),
                    __shfl_sync(kAll, sorted_down(odd), half - 1));
    }
    if constexpr (!ONE) {
      if (lane == 0) most_of[warp] = reached;
      __syncthreads();
      for (int w = 0; w < warps; ++w) bound = fminf(bound, most_of[w]);
    }
    bound = fmaxf(bound, -3.402823466e38f);      // values of -inf are not listed
    together();
    const auto note = [&](float v, int at) {
      if (!(v >= bound)) return;
      const int to = atomicAdd(&founds[own], 1);
      if (to < room) mine[to] = key_of(v, uint32_t(at));
    };
    const bool some = thread_most >= bound;
    if constexpr (ONE) {
      // Most lanes have something: each its own.
      for (int r0 = 0, piece = 0; some && r0 < rounds; r0 += in_piece, ++piece) {
        if (!(piece_of[piece][base + lane] >= bound)) continue;
        for (int r = r0; r < min(r0 + in_piece, rounds); ++r) {
          Vec<T> w[kAhead];
          fetch(v0 + r * step, w);
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            if (!(max_of(w[u]) >= bound)) continue;
            const int at = head + (v0 + r * step + u * threads + tid) * W;
#pragma unroll
            for (int k = 0; k < W; ++k) note(w[u].get(k), at + k);
          }
        }
      }
    } else {
      // Few have: the warp lists their pieces (where the pieces' maxima were, as they have been looked
      // at), and reads eight threads' at a time, four lanes a thread's loads in a round.
      // (Little code: it is run once a row, and has to be fetched.)
      unsigned pieces = 0;
#pragma unroll 1
      for (int i = 0; some && i * in_piece < rounds; ++i)
        if (piece_of[i][threadIdx.x] >= bound) pieces |= 1u << i;
      int to = __popc(pieces);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int before = __shfl_up_sync(kAll, to, d);
        if (lane >= d) to += before;
      }
      const int listed = __shfl_sync(kAll, to, 31);
      to -= __popc(pieces);
      const auto entry = [&](int i) -> float & { return piece_of[i >> 5][base + (i & 31)]; };
      for (; pieces; pieces &= pieces - 1)
        entry(to++) = __int_as_float(lane | (__ffs(int(pieces)) - 1) << 5);
      __syncwarp();
#pragma unroll 1
      for (int e = lane / kAhead; e < listed; e += 32 / kAhead) {
        const int which = __float_as_int(entry(e)), r0 = (which >> 5) * in_piece;
        const int first = v0 + lane % kAhead * threads + (tid - lane) + (which & 31);
#pragma unroll 1
        for (int r = r0; r < min(r0 + in_piece, rounds); ++r) {
          const int i = first + r * step;
          if (i >= v1) break;
          Vec<T> w;
          w.w = body[i];
          if (!(max_of(w) >= bound)) continue;
#pragma unroll
          for (int k = 0; k < W; ++k) note(w.get(k), head + i * W + k);
        }
      }
    }
    if (lane < ends) note(x, end_at);
    together();
    int count = founds[own];
    if (count > room) {
      // Too many alike: all of the block's part of the row again, and the ends, a list a warp.
      together();
      Best best = {scan_whole(from, head + int64_t(v0) * W + 32 * warp, head + int64_t(v1) * W, warps,
                              p.top)};
      if (ends > 0) best.add(lane < ends && x > -INFINITY ? key_of(x, uint32_t(end_at)) : kNoKey);
      mine[32 * warp + lane] = best.key;
      count = 32 * warps;
      together();
    }
    place(mine, count, list, tid, threads);
    together();
  }
  st.join_warp(c);
  Stats all = st;
  if constexpr (!ONE) {
    if (lane == 0) {
      part[0][warp] = st.m;
      part[1][warp] = st.s;
      part[2][warp] = st.w;
    }
    __syncthreads();
    if (cluster > 1) {
      cluster_barrier();
      if (TOP && rank == 0) {
        // Warp w takes the lists of blocks w, w + warps, ...
        for (int r = warp; r < cluster; r += warps)
          if (lane < p.top)
            found[p.top * r + lane] = cluster_u64(in_block(shared_address(&lists[0][lane]), r));
        __syncthreads();
        place(found, p.top * cluster, lists[0], tid, threads);   // (the same or larger keys, and as many)
        __syncthreads();
      }
    }
    if (rank == 0 && warp == 0) {
      all = {-INFINITY, 0.0f, 0.0f};
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
    }
  }
  if (rank == 0 && warp == 0) {
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
      const uint64_t key = lists[ONE ? threadIdx.x >> 5 : 0][lane];
      const bool have = key != kNoKey && !bad;
      const float v = value_of(uint32_t(key >> 32));
      p.top_ids[row * p.top + lane] = have ? int(~uint32_t(key)) : -1;
      p.top_logprobs[row * p.top + lane] =
          bad ? nan : have ? (v - all.m) * p.scale - log_s : -INFINITY;
    }
  }
  if (!ONE && cluster > 1) cluster_barrier();      // the others' shared memory has been read
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
  // Short rows in numbers: a warp each (8192 rows of 1000, bf16: a block of a warp each 19 us, eight
  // rows a block 6.4 us; of 8000, no or 5 listed: 38 and 56 by blocks, 27 and 40 by warps, but 2000 rows
  // with 20 listed 19 and 22).
  const bool one = rounds <= (p.top <= 16 ? 256 : 128) && p.rows >= 8 * dev.sm_count;
  // With alternatives smaller blocks, whose selections come more evenly (20 listed: 2000 x 8000, bf16, 25
  // and 20 us, 4096 x 32768 81 and 72, but 4096 x 131072 213 and 228).
  const bool small = p.top && rounds <= 4 * kMaxThreads && p.rows >= 4 * dev.sm_count;
  const int threads = one ? kMaxThreads : std::min(small ? 128 : kMaxThreads, round_threads(rounds));
  // Blocks of a row: twice as many blocks as there are SMs, a round of loads each at least.
  int cluster = 1;
  while (!one && cluster < kMaxCluster && p.rows * cluster < 2 * dev.sm_count &&
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
  const int64_t per = kMaxThreads / 32;
  cfg.gridDim = dim3(unsigned(one ? (p.rows + per - 1) / per : p.rows * cluster), 1, 1);
  cfg.blockDim = dim3(unsigned(threads), 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const auto kernel = p.top ? (one ? logprob_kernel<T, true, true> : logprob_kernel<T, true, false>)
                            : (one ? logprob_kernel<T, false, true>
                                   : logprob_kernel<T, false, false>);
  return cudaLaunchKernelEx(&cfg, kernel, p, cluster);
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

cudaError_t launch_logprob_grad(const LogprobGradProblem &p, cudaStream_t stream) {
  if (p.dtype == TMM_BF16) return launch_logprob_grad_as<__nv_bfloat16>(p, stream);
  if (p.dtype == TMM_F16) return launch_logprob_grad_as<__half>(p, stream);
  return launch_logprob_grad_as<float>(p, stream);
}

}  // namespace tmm
