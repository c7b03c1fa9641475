// route_rows.cu -- routing to experts: the k best experts of every token, and their weights.
//
//   s = softmax(l) or sigmoid(l) over a row's logits l,  c = s + bias,
//   the groups' values: the sum of a group's one or two best c,
//   the k best c among the experts of the best groups (ties: the lower number),
//   w_j = scale s_j / sum of the chosen s, or scale s_j.
// The choice is that of the scores to 43 bits (without a bias the logits stand for the scores, as both
// functions are increasing).  It is made in 32 bits, whose errors are bounded, and a row in which two
// values that decide something are closer than that is done again in pairs of FP32 values: one row in
// a thousand at 256 experts.
//
// A warp does a row, all of whose values stay in registers: with G groups rounded up to a power of
// two every group has 32 / G lanes, so that a group's best are a butterfly within its lanes.  The
// choice is k + 1 rounds of one warp reduction over keys that hold a value and its number.  A row's
// instructions (930 at 256 experts in 8 groups: 13 us of issue slots) and the chains of reductions and
// shuffles that they stand in, at 43 % of the warps that an SM holds, take the time (16384 rows of 256 FP32
// logits, k = 8, by replays of a graph: plain 14 us, sigmoids and a bias 17, in 8 groups 21 to 23; reading
// takes 2.7).  Neither more rows in flight (40 or 48 warps an SM: within 2 us, either way)
// nor blocks of another size help (one or two rows a block: 8 experts 17 and 9 us in place of 7; eight:
// the same).
// Gradient: w depends on the chosen logits alone, but for the softmax without renormalisation;
// rows are written whole, 16 bytes a lane, and the chosen few again (16384 x 256: 6.6 us; writing and
// reading take 2.8, a block every four rows most of the rest).
#include <cstdint>
#include <type_traits>

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
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}
// (NaN left out, unless all are.)
__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }
// For the choice, which allows for errors of 2^-20: the hardware's power of two and reciprocal.
__device__ __forceinline__ float near_exp(float t) { return exp2_approx(t * kLog2e); }
__device__ __forceinline__ float near_sigmoid(float l) {
  float s;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + near_exp(-l)));
  return s;
}

// ---- pairs of FP32 values --------------------------------------------------------------------
//
// A value is the sum of two FP32 values that do not overlap, 47 bits (Dekker's and Knuth's exact sums and
// products).  The FP64 units of this GPU are few and far: a row of 256 sigmoids took them 16 us, with
// nothing else to do.

struct Two {
  float h, l;
};
__device__ __forceinline__ Two sum_of(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two renewed(float h, float l) {      // |h| >= |l|
  const float s = __fadd_rn(h, l);
  return {s, __fsub_rn(l, __fsub_rn(s, h))};
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
  const Two s = sum_of(a.h, b.h), t = sum_of(a.l, b.l);
  const Two u = renewed(s.h, __fadd_rn(s.l, t.h));
  return renewed(u.h, __fadd_rn(u.l, t.l));
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
  const float p = __fmul_rn(a.h, b.h);
  return renewed(p, __fmaf_rn(a.h, b.l, __fmaf_rn(a.l, b.h, __fmaf_rn(a.h, b.h, -p))));
}
__device__ __forceinline__ Two one_over(Two b) {
  const float q = __frcp_rn(b.h);
  // 1 - q b, exactly but for its last bits.
  const float r = __fmaf_rn(-q, b.l, __fmaf_rn(-q, b.h, 1.0f));
  return renewed(q, __fmul_rn(q, r));
}
// e^y for y.h from -87 to 88.  y = n ln 2 + r, the first part of ln 2 of nine bits, so that n times it is
// exact; Taylor's series, whose terms from the seventh on are below 2^-22 of the sum and made in FP32.
__device__ __forceinline__ Two exp_of(Two y) {
  const float n = rintf(y.h * 1.44269504f);
  const float c = -0.00021219444f, p = __fmul_rn(n, c);      // the rest of ln 2
  const Two tail = {p, __fmaf_rn(n, 1.6465949697480609e-12f, __fmaf_rn(n, c, -p))};
  const Two r = Two{__fmaf_rn(-n, 0.693359375f, y.h), y.l} + Two{-tail.h, -tail.l};
  const float x = r.h;
  float t = 1.0f / 6227020800.0f;
  t = fmaf(t, x, 1.0f / 479001600.0f);
  t = fmaf(t, x, 1.0f / 39916800.0f);
  t = fmaf(t, x, 1.0f / 3628800.0f);
  t = fmaf(t, x, 1.0f / 362880.0f);
  t = fmaf(t, x, 1.0f / 40320.0f);
  t = fmaf(t, x, 1.0f / 5040.0f);
  Two q = {t, 0.0f};      // 1/6!, 1/5!, ...: their nearest FP32 values, and what these leave
  q = q * r + Two{1.0f / 720.0f, -3.3631094437103215e-11f};
  q = q * r + Two{1.0f / 120.0f, -4.34617203337595e-10f};
  q = q * r + Two{1.0f / 24.0f, -1.2417634698280722e-09f};
  q = q * r + Two{1.0f / 6.0f, -4.967053879312289e-09f};
  q = q * r + Two{0.5f, 0.0f};
  q = q * r + Two{1.0f, 0.0f};
  q = q * r + Two{1.0f, 0.0f};
  const float scale = __int_as_float((int(n) + 127) << 23);
  return {q.h * scale, q.l * scale};
}
__device__ __forceinline__ uint64_t key_of(Two v) {
  return uint64_t(key_of(v.h)) << 32 | key_of(v.l);
}
__device__ __forceinline__ Two value_of(uint64_t key) {
  return {value_of(uint32_t(key >> 32)), value_of(uint32_t(key))};
}
// To 44 bits, so that sums which are equal in the mathematics (of s(l) and s(-l)) are equal.
__device__ __forceinline__ Two shortened(Two v) {
  const float c = 1.5f * 0x1p-20f * __uint_as_float(__float_as_uint(v.h) & 0x7F800000u);
  return {v.h, __fsub_rn(__fadd_rn(v.l, c), c)};
}
__device__ __forceinline__ uint64_t more(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t less(uint64_t a, uint64_t b) { return a > b ? b : a; }

// The scores of up to four logits, a call: seldom run, and has to be fetched when it is.
struct Four {
  Two v[4];
};
__device__ __noinline__ Four scores_of(float l0, float l1, float l2, float l3, float m,
                                       bool is_sigmoid) {
  const float l[4] = {l0, l1, l2, l3};
  Four f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // 1 / (1 + e^-l) of the smaller of e^-l and e^l; e^(l - m).  0 below -87, where FP32 ends.
    Two y = is_sigmoid ? Two{-fabsf(l[i]), 0.0f} : sum_of(l[i], -m);
    const bool tiny = y.h < -87.0f;      // (NaN stays)
    if (tiny) y = {0.0f, 0.0f};
    Two e = exp_of(y);
    if (is_sigmoid) {
      const Two s = one_over(e + Two{1.0f, 0.0f});
      e = l[i] < 0.0f ? e * s : s;
    }
    const float end = is_sigmoid && l[i] > 0.0f ? 1.0f : 0.0f;
    f.v[i] = tiny ? Two{end, 0.0f} : e;
  }
  return f;
}

// A lane's keys, the largest first (a network of exchanges: Batcher's odd-even merge sort).
template <int V>
__device__ __forceinline__ void sort_down(uint32_t (&k)[V]) {
#pragma unroll
  for (int run = 1; run < V; run *= 2)
#pragma unroll
    for (int d = run; d > 0; d /= 2)
#pragma unroll
      for (int j = d % run; j + d < V; j += 2 * d)
#pragma unroll
        for (int i = 0; i < d; ++i)
          if (i + j + d < V && (i + j) / (2 * run) == (i + j + d) / (2 * run)) {
            const uint32_t x = k[i + j], y = k[i + j + d];
            k[i + j] = max(x, y);
            k[i + j + d] = min(x, y);
          }
}

// A lane's experts: numbers first + v * step for v < V, where v * step + sub < size.  VEC: every lane of
// a group has V of them, one after another.
template <bool VEC>
struct Lane {
  int first, stride, sub, size, group;
  __device__ __forceinline__ bool has(int v) const {
    return VEC ? size > 0 : v * stride + sub < size;
  }
  __device__ __forceinline__ int expert(int v) const { return first + (VEC ? v : v * stride); }
};
template <bool VEC, int V>
__device__ __forceinline__ Lane<VEC> lane_of(const RouteProblem &p, int lane) {
  Lane<VEC> a;
  a.group = lane >> p.lanes_log2;
  const int sub = lane & (p.lanes - 1);
  a.stride = p.lanes;
  a.sub = VEC ? sub * V : sub;
  a.first = a.group * p.group_size + a.sub;
  a.size = a.group < p.groups ? p.group_size : 0;
  return a;
}

// The biases of this lane's experts, 0 where it has none.
template <bool VEC, int V>
__device__ __forceinline__ void load_bias(const RouteProblem &p, const Lane<VEC> &a, float (&b)[V]) {
  if constexpr (VEC && V >= 4) {
    if (p.vec_bias) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (a.size > 0) w = *reinterpret_cast<const float4 *>(p.bias + a.first + 4 * i);
        b[4 * i] = w.x;
        b[4 * i + 1] = w.y;
        b[4 * i + 2] = w.z;
        b[4 * i + 3] = w.w;
      }
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) b[v] = a.has(v) ? p.bias[a.expert(v)] : 0.0f;
}

// In 32 bits, the scores c of this lane's experts (the logits without a bias) and which of them may be
// chosen; m: the row's maximum, where the scores are the softmax's.  Returns what two scores may be off
// by together: of the sigmoids, e^-l by 2^-22.5 and |l| 2^-23.4 of itself (times s (1 - s), and
// |l| s (1 - s) < 0.225), 1 + e^-l by 2^-24 and the reciprocal by 2^-23, in all 2.4e-7 each; of the
// softmax, every term by 2^-21, their sum by as many half steps as it has additions (at most 37), in all
// 2^-18 of the two scores, which are 1 / sum at most each.
template <bool VEC, int V>
__device__ __forceinline__ float make_scores(const RouteProblem &p, const Lane<VEC> &a,
                                             const float (&l)[V], float (&c)[V], bool (&on)[V],
                                             float &m) {
  const float *const bias = p.bias;
  float error = 0x1.2p-21f;
  m = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    c[v] = l[v];
    on[v] = l[v] != -INFINITY;
  }
  if (!p.sigmoid && (bias || p.best == 2)) {
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) top = fmaxf(top, l[v]);
    m = warp_max(top);
  }
  if (bias == nullptr) return 0.0f;
  if (p.sigmoid) {
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = near_sigmoid(c[v]);
  } else {
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      c[v] = on[v] ? near_exp(c[v] - m) : 0.0f;
      sum += c[v];
    }
    sum = 1.0f / warp_sum(sum);
    error = 0x1p-17f * sum;
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] *= sum;
  }
  float b[V];
  load_bias(p, a, b);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    on[v] &= b[v] != -INFINITY;
    c[v] += b[v];
  }
  return error;
}

// Whether this lane's group is one of the best.  `close`: the last one taken and the first that is not
// are too close to tell.
// one, two: this lane's two largest values.
template <bool VEC>
__device__ __forceinline__ bool group_open(const RouteProblem &p, const Lane<VEC> &a, float one,
                                           float two, float m, float error, bool &close) {
  const bool bias = p.bias != nullptr;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int d = 1; d < p.lanes; d <<= 1) {
    const float o = __shfl_xor_sync(kAll, one, d), t = __shfl_xor_sync(kAll, two, d);
    two = fmaxf(fmaxf(two, t), fminf(one, o));
    one = fmaxf(one, o);
  }
  const bool any = one != -INFINITY && a.size > 0;
  float value = one;
  if (p.best == 2 && any) {
    if (!bias && p.sigmoid)
      value = near_sigmoid(one) + near_sigmoid(two);
    else if (!bias)
      value = near_exp(one - m) + near_exp(two - m);
    else if (two != -INFINITY)
      value = one + two;
  }
  const uint32_t key = any ? key_of(value) : 0u;
  // A group's lanes compare it with every lanes-th group each.
  int rank = 0;
  for (int h = lane & (p.lanes - 1); h - (lane & (p.lanes - 1)) < p.groups; h += p.lanes) {
    const uint32_t other = __shfl_sync(kAll, key, h * p.lanes);
    rank += h < p.groups && (other > key || (other == key && h < a.group));
  }
#pragma unroll 1
  for (int d = 1; d < p.lanes; d <<= 1) rank += __shfl_xor_sync(kAll, rank, d);
  const bool open = key != 0 && rank < p.top_groups;
  if (bias || p.best == 2) {
    // (Values are in the order of their keys.)
    const uint32_t lo = __reduce_min_sync(kAll, open ? key : ~0u);
    const uint32_t hi = __reduce_max_sync(kAll, open ? 0u : key);
    const float x = value_of(lo), y = value_of(hi);
    // With a bias: the scores' errors, and half a step of each of four c and of two sums of them, which
    // may be far smaller than the c.  Without, a score of e^-87 is off by 87 2^-23.4 of itself.
    const float size = any && bias ? fabsf(one) + (fabsf(two) < INFINITY ? fabsf(two) : 0.0f) : 0.0f;
    const float tol = bias ? 2.0f * error + 0x1p-22f * warp_max(size) : 0x1p-15f * y + 1e-37f;
    close |= hi != 0 && x - y <= tol;
  }
  return open;
}

// The choice of a row in 32 bits: lane j < k leaves with expert j, or -1.  A key is 23 bits of where a
// value lies between the lowest and the highest that may be chosen, and 9 bits of the expert's number's
// complement, so that one reduction finds the best and, of equal ones, the lower number; every lane's
// keys are sorted first, and the lane that had the best shows its next.  `close`: two values that
// decide something are within the error of the scores and of a key, and not made from equal inputs, or
// one is not finite.  Two sigmoids alone that are close to each other, by far the most of these, are put
// in order here (again: 7 us; 16384 x 256, 8 groups: 27.5 us without this, 23.6 with it).
// l: this lane's logits, -inf where it has none.
template <typename T, bool VEC, int V>
__device__ __forceinline__ int choose(const RouteProblem &p, int64_t row, const Lane<VEC> &a,
                                      const float (&l)[V], bool &close) {
  const int lane = threadIdx.x & 31;
  float c[V], m;
  bool on[V], open = true;
  const float error = make_scores(p, a, l, c, on, m);
  float odd = 0.0f;      // NaN where a score is infinite or NaN
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (on[v]) odd += c[v] * 0.0f;
  close = __any_sync(kAll, odd != 0.0f);
  if (p.groups > 1) {
    float one = -INFINITY, two = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float x = on[v] ? c[v] : -INFINITY;
      two = fmaxf(two, fminf(one, x));
      one = fmaxf(one, x);
    }
    open = group_open(p, a, one, two, m, error, close);
  }
  float hi = -INFINITY, below = -INFINITY;      // below: the lowest, negated
#pragma unroll
  for (int v = 0; v < V; ++v) {
    on[v] &= open;
    if (on[v]) {
      hi = fmaxf(hi, c[v]);
      below = fmaxf(below, -c[v]);
    }
  }
  hi = warp_max(hi);
  const float lo = fmaxf(-warp_max(below), hi - 32.0f);      // (values further down share a key)
  const float range = hi - lo, step = range > 1e-30f ? 8388600.0f / range : 0.0f;
  const bool some = hi > -INFINITY;
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    // 2^23 + 1 to 2^24 - 7, whose lower 23 bits the key takes.
    const float at = fmaf(fmaxf(c[v], lo) - lo, step, 8388609.0f);
    key[v] = on[v] && some ? __float_as_uint(at) * 512u + uint32_t(511 - a.expert(v)) : 0u;
  }
  sort_down(key);
  // One round more than are chosen, to see what the last one was taken before.
  uint32_t mine = 0;
  for (int j = 0; j <= p.k; ++j) {
    const uint32_t top = __reduce_max_sync(kAll, key[0]);
    if (lane == j) mine = top;
    const bool pop = key[0] == top;
#pragma unroll
    for (int v = 0; v + 1 < V; ++v) key[v] = pop ? key[v + 1] : key[v];
    key[V - 1] = pop ? 0u : key[V - 1];
  }
  const uint32_t next = __shfl_down_sync(kAll, mine, 1);
  // (Keys are made of steps that do not decrease: without a bias only equal ones are in doubt.)
  const float tol =
      p.bias ? (error + 0x1p-22f * fmaxf(fabsf(hi), fabsf(lo))) * step + 1.5f : 0.5f;
  const bool near = lane < p.k && next != 0 && float((mine >> 9) - (next >> 9)) <= tol;
  const unsigned pairs = __ballot_sync(kAll, near);
  if (pairs) {
    const T *const at = static_cast<const T *>(p.logits) + row * p.ld;
    const int x = 511 - int(mine & 511), y = 511 - int(next & 511);
    // Equal logits with equal biases are equal, and their numbers decide.
    const bool doubt = near && (as_float(at[x]) != as_float(at[y]) ||
                                (p.bias && p.bias[x] != p.bias[y]));
    // The last one and the one before it are no pair alone if a third is close, which is shown next.
    const uint32_t third = __reduce_max_sync(kAll, key[0]), last = __shfl_sync(kAll, mine, p.k);
    const bool three = third != 0 && float((last >> 9) - (third >> 9)) <= tol;
    if (!p.bias || !p.sigmoid || (pairs & pairs << 1) || (three && (pairs >> (p.k - 1) & 1))) {
      close |= __any_sync(kAll, doubt);
    } else {
      bool swap = false;
      if (doubt) {
        const Four f = scores_of(as_float(at[x]), as_float(at[y]), 0.0f, 0.0f, 0.0f, true);
        const uint64_t a2 = key_of(f.v[0] + Two{p.bias[x], 0.0f});
        const uint64_t b2 = key_of(f.v[1] + Two{p.bias[y], 0.0f});
        swap = b2 > a2 || (b2 == a2 && y < x);
      }
      const unsigned swaps = __ballot_sync(kAll, swap);
      const uint32_t before = __shfl_up_sync(kAll, mine, 1);
      if (swap)
        mine = next;
      else if (swaps << 1 >> lane & 1)
        mine = before;
    }
  }
  return lane < p.k && mine != 0 ? 511 - int(mine & 511) : -1;
}

template <typename T, bool VEC, int V>
__device__ __forceinline__ void load_logits(const RouteProblem &p, int64_t row, const Lane<VEC> &a,
                                            float (&l)[V]) {
  const T *const from = static_cast<const T *>(p.logits) + row * p.ld;
  constexpr int kVec = Vec<T>::kCount;
  if constexpr (VEC) {
    Vec<T> w[V / kVec];
    if (a.size > 0) {
#pragma unroll
      for (int i = 0; i < V / kVec; ++i)
        w[i].w = *reinterpret_cast<const uint4 *>(from + a.first + i * kVec);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = a.size > 0 ? w[v / kVec].get(v % kVec) : -INFINITY;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = a.has(v) ? as_float(from[a.expert(v)]) : -INFINITY;
  }
}

// ---- the choice again ----------------------------------------------------------------------

// `choose` in pairs of values: the expert, or -1, plus 1, and kNaN for a row whose weights are NaN.
constexpr int kNaN = 1 << 16;
template <typename T, bool VEC, int V>
__device__ __noinline__ int choose_again(const RouteProblem &p, int64_t row) {
  const int lane = threadIdx.x & 31;
  const Lane<VEC> a = lane_of<VEC, V>(p, lane);
  float l[V], b[V], m = -INFINITY;      // -inf for an expert that may not be chosen
  load_logits<T>(p, row, a, l);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    b[v] = 0.0f;
    m = fmaxf(m, l[v]);
  }
  m = warp_max(m);
  Two c[V], sum = {0.0f, 0.0f};
#pragma unroll
  for (int v = 0; v < V; ++v) c[v] = {l[v], 0.0f};
  if (p.bias) {
    load_bias(p, a, b);
#pragma unroll
    for (int v = 0; v < V; v += 4) {
      const Four f = scores_of(l[v], v + 1 < V ? l[v + 1] : 0.0f, v + 2 < V ? l[v + 2] : 0.0f,
                               v + 3 < V ? l[v + 3] : 0.0f, m, p.sigmoid);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (v + i < V) c[v + i] = f.v[i];
    }
    Two scale = {1.0f, 0.0f};
    if (!p.sigmoid) {
#pragma unroll
      for (int v = 0; v < V; ++v) sum = sum + c[v];
#pragma unroll 1
      for (int d = 16; d > 0; d >>= 1)
        sum = sum + Two{__shfl_xor_sync(kAll, sum.h, d), __shfl_xor_sync(kAll, sum.l, d)};
      scale = one_over(sum);
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      c[v] = fabsf(b[v]) < INFINITY ? c[v] * scale + Two{b[v], 0.0f} : Two{b[v], 0.0f};
  }
  uint64_t key[V], best = 0, second = 0;
  bool bad = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    // (Of the softmax any expert's logit makes every score NaN, whatever its bias.)
    bad |= p.sigmoid ? l[v] != l[v] && b[v] != -INFINITY : l[v] != l[v] || l[v] == INFINITY;
    key[v] = l[v] == -INFINITY || b[v] == -INFINITY ? 0 : key_of(c[v]);
    second = more(second, less(best, key[v]));
    best = more(best, key[v]);
  }
  if (p.groups > 1) {
    uint64_t one = best, two = second;
#pragma unroll 1
    for (int d = 1; d < p.lanes; d <<= 1) {
      const uint64_t o = __shfl_xor_sync(kAll, one, d), t = __shfl_xor_sync(kAll, two, d);
      two = more(more(two, t), less(one, o));
      one = more(one, o);
    }
    uint64_t value = one;
    if (p.best == 2 && two != 0) {
      Two x = value_of(one), y = value_of(two);
      if (!p.bias) {
        const Four f = scores_of(x.h, y.h, 0.0f, 0.0f, m, p.sigmoid);
        x = f.v[0];
        y = f.v[1];
      }
      const Two s = shortened(x + y);
      value = key_of(fabsf(x.h + y.h) < INFINITY ? s : Two{x.h + y.h, 0.0f});
    } else if (p.best == 2 && one != 0 && !p.bias) {
      value = key_of(scores_of(value_of(one).h, 0.0f, 0.0f, 0.0f, m, p.sigmoid).v[0]);
    }
    int rank = 0;
#pragma unroll 1
    for (int h = 0; h < p.groups; ++h) {
      const uint64_t other = __shfl_sync(kAll, value, h * p.lanes);
      rank += other > value || (other == value && h < a.group);
    }
    if (value == 0 || rank >= p.top_groups)
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = 0;
  }
  int mine = -1;
#pragma unroll 1
  for (int j = 0; j < p.k; ++j) {
    best = key[0];
    int at = 0;
#pragma unroll
    for (int v = 1; v < V; ++v)
      if (key[v] > best) {
        best = key[v];
        at = v;
      }
    const uint32_t high = __reduce_max_sync(kAll, uint32_t(best >> 32));
    const uint32_t low =
        __reduce_max_sync(kAll, uint32_t(best >> 32) == high ? uint32_t(best) : 0u);
    const uint64_t most = uint64_t(high) << 32 | low;
    if (most == 0) break;
    const int e = int(__reduce_min_sync(
        kAll, best == most ? unsigned(a.expert(at)) : unsigned(INT32_MAX)));
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (a.has(v) && a.expert(v) == e) key[v] = 0;
    if (lane == j) mine = e;
  }
  return mine + 1 + (__any_sync(kAll, bad) ? kNaN : 0);
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

// (64 registers a thread for up to 8 values a lane: the choice in pairs would take 96 and leave fewer rows in
// flight.  As it is it keeps some in memory, 28 to 56 bytes a thread at 8 values and up to 340 at 32, in a row in a
// thousand.)
template <typename T, bool VEC, int V>
__global__ void __launch_bounds__(32 * kWarps, V <= 8 ? 8 : V <= 16 ? 5 : 3)
route_kernel(const __grid_constant__ RouteProblem p) {
  wait_then_start_next();
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= p.tokens) return;
  const Lane<VEC> a = lane_of<VEC, V>(p, lane);
  float l[V];
  load_logits<T>(p, row, a, l);
  bool close;
  int e = choose<T>(p, row, a, l, close);
  bool bad = false;
  if (close) {
    const int again = choose_again<T, VEC, V>(p, row);
    bad = again >= kNaN;
    e = (again & (kNaN - 1)) - 1;
  }
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
  float w = score_of(p.sigmoid, p.renormalise, x, m, sum);
  if (bad) w = __uint_as_float(0x7FFFFFFFu);
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
  // The same expert in several slots: the first of them adds them up.
  const unsigned same = __match_any_sync(kAll, e);
  const bool writes = e >= 0 && (same & ((1u << lane) - 1)) == 0;
  if (__any_sync(kAll, e >= 0 && !writes)) {
    float all = 0.0f;
    for (int j = 0; j < p.k; ++j) {
      const float add = __shfl_sync(kAll, d, j);
      if (same >> j & 1) all += add;
    }
    d = all;
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int first = (32 * i + lane) * W;
    if (first >= p.experts) continue;
    if constexpr (VEC) {
      Vec<T> w;
      w.w = make_uint4(0, 0, 0, 0);
      if (dense)
#pragma unroll
        for (int c = 0; c < W; ++c) w.set(c, l[i][c] != 0.0f ? l[i][c] * r : 0.0f);
      *reinterpret_cast<uint4 *>(to + first) = w.w;
    } else {
      to[first] = rounded<T>(dense && l[i][0] != 0.0f ? l[i][0] * r : 0.0f);
    }
  }
  __syncwarp();      // orders the row's stores before those of the slots
  if (writes) {
    // (What the row has there, once more: e^(x - m), and the slots' part.)
    const float part = dense && x != -INFINITY ? expf(x - m) : 0.0f;
    to[e] = rounded<T>((part != 0.0f ? part * r : 0.0f) + d);
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
  p.lanes_log2 = 0;
  while (1 << p.lanes_log2 < p.lanes) ++p.lanes_log2;
  const int need = (p.group_size + p.lanes - 1) / p.lanes;      // at most 32
  int V = 1;
  while (V < need) V *= 2;
  const bool vec = p.group_size == V * p.lanes && V * sizeof(T) % 16 == 0 &&
                   (reinterpret_cast<uintptr_t>(p.logits) & 15u) == 0 && p.ld * sizeof(T) % 16 == 0;
  p.vec_bias = (reinterpret_cast<uintptr_t>(p.bias) & 15u) == 0;
  const auto launch = [&](auto few) {
    constexpr int N = decltype(few)::value;
    if constexpr (N * sizeof(T) % 16 == 0)
      if (vec) return launch_rows(route_kernel<T, true, N>, p, p.tokens, stream);
    return launch_rows(route_kernel<T, false, N>, p, p.tokens, stream);
  };
  switch (V) {
    case 1: return launch(std::integral_constant<int, 1>());
    case 2: return launch(std::integral_constant<int, 2>());
    case 4: return launch(std::integral_constant<int, 4>());
    case 8: return launch(std::integral_constant<int, 8>());
    case 16: return launch(std::integral_constant<int, 16>());
    default: return launch(std::integral_constant<int, 32>());
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
