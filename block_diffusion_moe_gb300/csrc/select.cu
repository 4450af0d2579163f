// Expert selection and grouping (clover_route) and the weighted sum of expert
// rows (clover_moe_combine).
#include <math.h>

#include "launch.cuh"
#include "moe_ops.cuh"
#include "routing.cuh"
#include "sm100.cuh"

namespace clover {

namespace {

constexpr int kWarps = plan::kRouteWarps;  // one token each at a time
constexpr int kThreads = kWarps * 32;
constexpr int kPerThread = kRouteOpMaxExperts / kThreads;  // experts a thread counts for, at most
constexpr uint32_t kAll = 0xffffffffu;
// Largest K + 1 that is selected by counting (select_token): beyond it the
// keys above the bound no longer fit 32 lanes as a rule.
constexpr int kCountedMax = 17;
constexpr int kNoGroup = 64;  // rank of a lane that holds no group
constexpr int kListBytes = 512;  // a warp's list of 32 keys and ids, or exact keys and scores

// +inf counts as the largest finite value, NaN as -inf (fmaxf takes the operand
// that is a number).
__device__ __forceinline__ float clean_logit(float v) { return fminf(fmaxf(v, -INFINITY), 3.402823466e+38f); }

__device__ __forceinline__ float load_logit(const RouteOpArgs& a, int64_t row, int e) {
  const float v = a.bf16_logits ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[row + e])
                                : static_cast<const float*>(a.logits)[row + e];
  return clean_logit(v);
}

// The token's logits: expert lane * VPL + i in slot i (so that a lower lane
// holds lower ids), -inf past E. One vector per lane where the rows allow it
// (a.vec: E % VPL == 0 and every lane's part aligned to its size or 16 bytes).
template <int VPL>
__device__ __forceinline__ void load_row(const RouteOpArgs& a, int64_t row, int lane, float (&x)[VPL]) {
  const int e0 = lane * VPL;
  if (a.vec) {
    uint32_t wd[VPL];  // the lane's part
    const int words = a.bf16_logits ? VPL / 2 : VPL;
#pragma unroll
    for (int i = 0; i < VPL; ++i) wd[i] = a.bf16_logits ? 0xFF80FF80u : 0xFF800000u;  // -inf
    if (e0 < a.E) {
      const uint8_t* p = static_cast<const uint8_t*>(a.logits) + (row + e0) * (a.bf16_logits ? 2 : 4);
      if (VPL >= 4 && words >= 4) {
#pragma unroll
        for (int v = 0; v < VPL / 4; ++v)
          if (4 * v < words) {
            const uint4 u = *reinterpret_cast<const uint4*>(p + 16 * v);
            wd[4 * v] = u.x, wd[4 * v + 1] = u.y, wd[4 * v + 2] = u.z, wd[4 * v + 3] = u.w;
          }
      } else if (words == 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        wd[0] = u.x, wd[1] = u.y;
      } else {
        wd[0] = *reinterpret_cast<const uint32_t*>(p);
      }
    }
    if (a.bf16_logits) {
#pragma unroll
      for (int i = VPL - 1; i >= 0; --i)
        x[i] = __uint_as_float(i % 2 == 0 ? wd[i / 2] << 16 : wd[i / 2] & 0xFFFF0000u);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) x[i] = __uint_as_float(wd[i]);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) x[i] = clean_logit(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) x[i] = e0 + i < a.E ? load_logit(a, row, e0 + i) : -INFINITY;
  }
}

// The biases in shared memory, by the whole CTA: 0 without any and past E, -inf
// for NaN.
template <int VPL>
__device__ __forceinline__ void load_bias(const RouteOpArgs& a, float* s_bias) {
  for (int e = threadIdx.x; e < 32 * VPL; e += kThreads) {
    const float b = (a.bias != nullptr && e < a.E) ? a.bias[e] : 0.f;
    s_bias[e] = b > -INFINITY ? b : -INFINITY;
  }
  __syncthreads();
}

// How far below key k another has to lie for their order to be certain, where a
// score is off by up to err: the error of both keys. The rounding of the sum with
// the bias, half a unit of the key, comes on top of the score's (twice that here,
// which covers the comparison's own). It goes by the key, not by the largest bias,
// so that an expert masked by -1e9 puts no other in doubt (32,768 tokens with one
// such expert: 490 us by the largest bias, 45 so). The lower key's unit can only
// be the larger one where both are negative or far apart, and then by less than a
// 2^-23rd of their distance. k -+ key_gap(k) grows with k, so where the order of
// two keys is certain, all above the one lie above all below the other.
__device__ __forceinline__ float key_gap(float err, float k) {
  return fmaf(fminf(fabsf(k), 3.402823466e+38f), 0x1p-22f, 2.f * err);
}

// Keys whose signed order is the order of the floats (with +0 above -0).
__device__ __forceinline__ int order_int(float v) {
  const int b = __float_as_int(v);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float order_float(int m) { return __int_as_float(m ^ ((m >> 31) & 0x7fffffff)); }

__device__ __forceinline__ float warp_max_fast(float v) { return order_float(__reduce_max_sync(kAll, order_int(v))); }

// The same for doubles (-0 first made 0, so that the two tie).
__device__ __forceinline__ int64_t order_int64(double v) {
  const int64_t b = __double_as_longlong(v + 0.0);
  return b ^ ((b >> 63) & 0x7fffffffffffffffLL);
}
__device__ __forceinline__ double order_double(int64_t m) {
  return __longlong_as_double(m ^ ((m >> 63) & 0x7fffffffffffffffLL));
}

// Error: see token_keys. Values below 2^-126 count as 0 (.ftz; with the steps
// that keep them 32,768 tokens took 35.2 instead of 34.2 us).
__device__ __forceinline__ float fast_sigmoid(float v) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return s;
}

// (b1, b2): the two largest of a set, kept up to date with v
__device__ __forceinline__ void two_best(float& b1, float& b2, float v) {
  b2 = fmaxf(b2, fminf(b1, v));
  b1 = fmaxf(b1, v);
}

// Lists this warp's keys at or above the lane's bound (and above -inf) in shared
// memory, lower lanes first: (key, id). Returns their number; a number above 32
// and no list where they do not fit.
template <int VPL>
__device__ __forceinline__ int list_above(const float (&key)[VPL], float bound, uint2* list, int lane) {
  bound = fmaxf(bound, -3.402823466e+38f);
  int c = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) c += key[i] >= bound ? 1 : 0;
  // places by lane: the sum of the lower lanes' counts, bit by bit
  const uint32_t lower = (1u << lane) - 1u;
  int at = 0, n = 0;
#pragma unroll
  for (int bit = 0; (1 << bit) <= VPL; ++bit) {
    const uint32_t v = __ballot_sync(kAll, (c >> bit) & 1);
    at += __popc(v & lower) << bit;
    n += __popc(v) << bit;
  }
  if (n > 32) return n;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (key[i] >= bound) list[at++] = make_uint2(__float_as_uint(key[i]), lane * VPL + i);
  __syncwarp();
  return n;
}

// ---- The order in exact arithmetic: in double, as the definition has it. Rare
// (about one token in a thousand) and written for few registers: what these
// functions need is taken from the loop over tokens that calls them (with four
// exponentials at a time 32,768 tokens took 51 instead of 47 us).

struct SoftmaxSum {
  double max, sum;
};

__device__ __noinline__ SoftmaxSum softmax_sum(const RouteOpArgs& a, int64_t row, int lane) {
  float m = -INFINITY;
  for (int e = lane; e < a.E; e += 32) m = fmaxf(m, load_logit(a, row, e));
  SoftmaxSum r;
  r.max = warp_max_f(m);
  r.sum = 0;
#pragma unroll 1
  for (int e = lane; e < a.E; e += 32) r.sum += exp(static_cast<double>(load_logit(a, row, e)) - r.max);
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) r.sum += __shfl_xor_sync(kAll, r.sum, o);
  return r;
}

// The same with a sum in float, off by less than 2^-19 of it.
__device__ __noinline__ SoftmaxSum softmax_sum_near(const RouteOpArgs& a, int64_t row, int lane) {
  float m = -INFINITY, sum = 0.f;
  for (int e = lane; e < a.E; e += 32) m = fmaxf(m, load_logit(a, row, e));
  m = warp_max_f(m);
  for (int e = lane; e < a.E; e += 32) sum += expf(load_logit(a, row, e) - m);
  SoftmaxSum r;
  r.max = m;
  r.sum = warp_sum_f(sum);
  return r;
}

// Score + bias of expert e, -inf where dead; the score in *score.
__device__ __forceinline__ double exact_total(const RouteOpArgs& a, int64_t row, int e, SoftmaxSum s,
                                              double* score = nullptr) {
  const float z = load_logit(a, row, e);
  const float b = a.bias != nullptr ? a.bias[e] : 0.f;
  if (!(z > -INFINITY && b > -INFINITY)) return -static_cast<double>(INFINITY);
  double t = exp(a.softmax ? static_cast<double>(z) - s.max : -static_cast<double>(z));
  t = a.softmax ? t / s.sum : 1.0 / (1.0 + t);
  if (score != nullptr) *score = t;
  return t + static_cast<double>(b);
}

// Lane k < n holds candidate id; returns the candidate of rank k by exact key,
// the lower id first on ties.
//
// A softmax's sum is what costs (E exponentials in double, 8 us; the candidates'
// own take 1.5). An error of the sum moves all scores in proportion, so the
// difference of two keys by as much of the difference of their scores: with the
// sum in float the order stands unless two neighbours are that close, and only
// then the sum is worked out in double.
__device__ __noinline__ int rank_exact(const RouteOpArgs& a, int64_t row, int id, int n, int lane, int64_t* smem) {
  struct Entry {
    double key, score;
  };
  Entry* sorted = reinterpret_cast<Entry*>(smem);  // [32]
  int32_t* order = reinterpret_cast<int32_t*>(smem);
  SoftmaxSum s = {0, 1};
  if (a.softmax) s = softmax_sum_near(a, row, lane);
  int before;
#pragma unroll 1
  for (bool near = a.softmax != 0;; near = false) {
    double score = 0;
    const double key = lane < n ? exact_total(a, row, id, s, &score) : 0.0;
    const int64_t own = order_int64(key);
    smem[lane] = own;
    __syncwarp();
    before = 0;
    for (int j = 0; j < n; ++j) {
      const int64_t o = smem[j];
      const int f = __shfl_sync(kAll, id, j);
      before += (o > own || (o == own && f < id)) ? 1 : 0;
    }
    __syncwarp();
    if (!near) break;
    if (lane < n) sorted[before] = Entry{key, score};
    __syncwarp();
    bool close = false;
    if (lane + 1 < n) {
      const Entry u = sorted[lane], v = sorted[lane + 1];
      const double apart = fabs(u.score - v.score);
      close = apart > 0 && !(u.key - v.key > apart * 0x1p-18 + fabs(u.key) * 0x1p-50);
    }
    __syncwarp();
    if (!__any_sync(kAll, close)) break;
    s = softmax_sum(a, row, lane);
  }
  if (lane < n) order[before] = id;
  __syncwarp();
  const int r = lane < n ? order[lane] : -1;
  __syncwarp();
  return r;
}

// The whole selection: lane k < K returns the k-th expert (-1: none left).
// smem: E numbers.
__device__ __noinline__ int select_exact(const RouteOpArgs& a, int64_t row, int lane, int64_t* smem) {
  const int64_t ninf = order_int64(-static_cast<double>(INFINITY));
  SoftmaxSum s = {0, 1};
  if (a.softmax) s = softmax_sum(a, row, lane);
#pragma unroll 1
  for (int e = lane; e < a.E; e += 32) smem[e] = order_int64(exact_total(a, row, e, s));
  __syncwarp();
  uint32_t mask = kAll;
  if (a.n_groups > 1) {
    int64_t b1 = ninf, b2 = ninf;
    if (lane < a.n_groups)
#pragma unroll 1
      for (int n = 0; n < a.group_size; ++n) {
        const int64_t v = smem[lane * a.group_size + n];
        b2 = max(b2, min(b1, v));
        b1 = max(b1, v);
      }
    const int64_t rank = (a.group_rank == 2 && b2 > ninf) ? order_int64(order_double(b1) + order_double(b2)) : b1;
    int before = 0;
#pragma unroll 1
    for (int j = 0; j < a.n_groups; ++j) {
      const int64_t r = __shfl_sync(kAll, rank, j);
      before += (r > rank || (r == rank && j < lane)) ? 1 : 0;
    }
    mask = __ballot_sync(kAll, before < a.top_groups);
    __syncwarp();
  }
#pragma unroll 1
  for (int e = lane; e < a.E; e += 32) {
    if (a.bias == nullptr) smem[e] = order_int64(static_cast<double>(load_logit(a, row, e)));
    if (a.n_groups > 1 && ((mask >> (e / a.group_size)) & 1u) == 0) smem[e] = ninf;
  }
  __syncwarp();
  int mine = -1;
#pragma unroll 1
  for (int k = 0; k < a.K; ++k) {
    int64_t best = ninf;
    int at = 0x7fffffff;
#pragma unroll 1
    for (int e = lane; e < a.E; e += 32)
      if (smem[e] > best) {
        best = smem[e];
        at = e;
      }
    int64_t top = best;
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) top = max(top, static_cast<int64_t>(__shfl_xor_sync(kAll, top, o)));
    if (top == ninf) break;  // uniform: no live expert left
    const int id = __reduce_min_sync(kAll, best == top ? at : 0x7fffffff);
    if (lane == k) mine = id;
    if (lane == (id & 31)) smem[id] = ninf;
    __syncwarp();
  }
  return mine;
}

// Groups before this lane's, by exact ranks: lane k < n holds one of the
// candidates (the experts that can be among the one or two best of their
// group). g: this lane's group.
__device__ __noinline__ int rank_groups_exact(const RouteOpArgs& a, int64_t row, int id, int n, int g, int lane,
                                              int64_t* smem) {
  const int64_t ninf = order_int64(-static_cast<double>(INFINITY));
  SoftmaxSum s = {0, 1};
  if (a.softmax) s = softmax_sum(a, row, lane);
  if (lane < n) smem[lane] = order_int64(exact_total(a, row, id, s));
  __syncwarp();
  int64_t b1 = ninf, b2 = ninf;  // of group `lane`
  for (int j = 0; j < n; ++j) {
    const int64_t v = __shfl_sync(kAll, id, j) / a.group_size == lane ? smem[j] : ninf;
    b2 = max(b2, min(b1, v));
    b1 = max(b1, v);
  }
  __syncwarp();
  const int64_t rank = (a.group_rank == 2 && b2 > ninf) ? order_int64(order_double(b1) + order_double(b2)) : b1;
  const int64_t mine = __shfl_sync(kAll, rank, g & 31);
  int before = 0;
  for (int j = 0; j < a.n_groups; ++j) {
    const int64_t r = __shfl_sync(kAll, rank, j);
    before += (r > mine || (r == mine && j < g)) ? 1 : 0;
  }
  return before;
}

// Turns the token's logits in key (-inf where dead) into what experts are
// ordered by: -inf for a dead expert and for one in a group that does not stay.
// False where the token has no live expert (every lane alike).
//
// *err bounds the error of a score (key_gap: that of two keys), and *doubt is
// set (in every lane) where the ranks on either side of the group border are
// closer than the errors they can have and are not settled here. With m the
// largest score: a softmax score is off by less than 2^-19 m (exp and quotient a
// few roundings each, the sum up to 21). A sigmoid: exp(-x) is off by (2 + |x|)
// 2^-23 of its value (2^-22 by the documented bound of ex2.approx, the rest by
// the rounding of its argument and of log2 e), which changes s by (1 - s) s of
// that; s (1 - s) |x| is below 0.23, and below m |x of m| where all logits are
// low, so with the 2^-22 of the sum and the reciprocal less than (2^-20 + 2^-22
// max(-x of m, 0)) m. Scores that count as 0 add less than 1e-37. Logits used as
// keys are exact.
template <int VPL>
__device__ __forceinline__ bool token_keys(const RouteOpArgs& a, const float* bias, int64_t row, int64_t* smem, int lane,
                                           float (&key)[VPL], float* err, bool* doubt) {
  *err = 0.f;
  const bool sums = a.n_groups > 1 && a.group_rank == 2;  // ranks are sums of scores
  if (a.bias != nullptr || sums) {
    float xm = key[0], xl = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) xm = fmaxf(xm, key[i]), xl = fminf(xl, key[i]);
    xm = warp_max_fast(xm);
    if (xm == -INFINITY) return false;
    uint32_t dead = 0;  // bit i: slot i holds no live expert
    if (__any_sync(kAll, xl == -INFINITY)) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) dead |= (key[i] > -INFINITY ? 0u : 1u) << i;
    }
    float s_max;
    if (a.softmax) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        key[i] = expf(key[i] - xm);
        sum += key[i];
      }
      s_max = 1.f / warp_sum_f(sum);  // the sum is at least 1
      *err = s_max * 0x1p-19f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] *= s_max;
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = fast_sigmoid(key[i]);
      s_max = fast_sigmoid(xm);
      *err = s_max * (0x1p-20f + 0x1p-22f * fmaxf(-xm, 0.f));
    }
    if (a.bias != nullptr) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] += bias[lane * VPL + i];
    }
    if (__any_sync(kAll, dead != 0)) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = (dead >> i) & 1u ? -INFINITY : key[i];
    }
    *err += 1e-37f;
  }
  if (a.n_groups == 1) return true;

  // Group ranks. Without a bias experts go by their logits, whatever the
  // groups go by.
  float b1 = -INFINITY, b2 = -INFINITY;
  int g = lane, shift = 0;  // this lane's group; groups lie 2^shift lanes apart
  if (a.group_shift >= 0) {
    // a group is all slots of a power of two of neighbouring lanes
#pragma unroll
    for (int i = 0; i < VPL; ++i) two_best(b1, b2, key[i]);
    shift = a.group_shift;
    g = lane >> shift;
    for (int o = 1; o < (1 << shift); o <<= 1) {
      const float c1 = __shfl_xor_sync(kAll, b1, o), c2 = __shfl_xor_sync(kAll, b2, o);
      two_best(b1, b2, c1);
      b2 = fmaxf(b2, c2);
    }
  } else {
    // any other size: keys in shared memory, lane g scans group g
    float* s_keys = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane * VPL + i < a.E) s_keys[lane * VPL + i] = key[i];
    __syncwarp();
    if (g < a.n_groups)
      for (int n = 0; n < a.group_size; ++n) two_best(b1, b2, s_keys[g * a.group_size + n]);
    __syncwarp();
  }
  const bool two = a.group_rank == 2 && b2 > -INFINITY;
  const float sum = two ? b1 + b2 : b1;
  // below fp32's range a live group still comes before one without a live expert
  const float rank = two ? fmaxf(sum, -3.402823466e+38f) : sum;
  // the groups before this one; a group's lanes share the comparisons
  const int step = 1 << shift;
  int before = 0;
  for (int j0 = 0; j0 < a.n_groups; j0 += step) {
    const int j = j0 + (lane & (step - 1));
    const float r = __shfl_sync(kAll, rank, (j << shift) & 31);
    before += (j < a.n_groups && (r > rank || (r == rank && j < g))) ? 1 : 0;
  }
  for (int o = 1; o < step; o <<= 1) before += __shfl_xor_sync(kAll, before, o);
  if (g >= a.n_groups) before = kNoGroup;
  if (*err > 0.f) {
    // the lowest that a group that stays can rank and the highest that another
    // live one can (a sum's own rounding: the other half of the keys' units)
    float off = 0.5f * key_gap(*err, b1);
    if (two) off += fmaf(fminf(fabsf(rank), 3.402823466e+38f), 0x1p-24f, 0.5f * key_gap(*err, b2));
    // (sums outside fp32's range are bounded on one side only)
    const float in = -warp_max_fast(before < a.top_groups ? off - fminf(sum, 3.402823466e+38f) : -INFINITY);
    const float out = warp_max_fast(before < a.top_groups || b1 == -INFINITY ? -INFINITY : rank + off);
    *doubt = out > -INFINITY && !(in > out);
    if (*doubt && a.group_shift >= 0) {
      // the ranks again, from the exact scores of the few that can matter
      uint2* list = reinterpret_cast<uint2*>(smem);
      const float last = a.group_rank == 2 ? b2 : b1;
      const int n = list_above<VPL>(key, last - key_gap(*err, last), list, lane);
      if (n <= 32) {
        const int id = lane < n ? static_cast<int>(list[lane].y) : 0;
        __syncwarp();
        before = rank_groups_exact(a, row, id, n, g, lane, smem);
        if (g >= a.n_groups) before = kNoGroup;
        *doubt = false;
      }
    }
  }
  if (a.bias == nullptr && sums) {
    load_row<VPL>(a, row, lane, key);
    *err = 0.f;
  }
  if (a.group_shift >= 0) {
    if (before >= a.top_groups) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = -INFINITY;
    }
  } else {
    const uint32_t mask = __ballot_sync(kAll, before < a.top_groups);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      if (e < a.E && ((mask >> (e / a.group_size)) & 1u) == 0) key[i] = -INFINITY;
    }
  }
  return true;
}

// Whether two experts' keys, closer than their errors, are a true tie: the
// same logit and the same bias.
__device__ __forceinline__ bool same_key(const RouteOpArgs& a, int64_t row, int e, int f) {
  return load_logit(a, row, e) == load_logit(a, row, f) && (a.bias == nullptr || a.bias[e] == a.bias[f]);
}

// The first `want` experts by descending key, ties to the lower id: lane k
// returns the k-th (-1: none left). Each round takes the largest key and the
// lowest lane, so the lowest id, that holds it. *doubt is set where two
// successive keys are closer than their errors. The last pair's order has to be
// certain: behind a true tie there the rounds go on to the first one that is
// not, as a key further down could still belong before both.
template <int VPL>
__device__ __forceinline__ int pick_by_rounds(const RouteOpArgs& a, int64_t row, float (&key)[VPL], int want, float err,
                                              int lane, bool* doubt) {
  int mine = -1, last_id = -1;
  float last = 0.f, gap = 0.f;  // the last key, key_gap(last)
  bool tied = false;            // the last pair is a true tie
  for (int k = 0; k < want || tied; ++k) {
    float best = -INFINITY;
    int at = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    const float top = warp_max_fast(best);
    if (!(top > -INFINITY)) break;  // uniform: no live expert left
    const int from = __ffs(__ballot_sync(kAll, best == top)) - 1;
    const int id = __shfl_sync(kAll, lane * VPL + at, from);
    tied = k > 0 && err > 0.f && !(last - top > gap);
    if (tied && !same_key(a, row, last_id, id)) {
      *doubt = true;
      break;
    }
    last = top;
    gap = key_gap(err, top);
    last_id = id;
    if (lane == k) mine = id;
    if (lane == from) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i == at) key[i] = -INFINITY;
    }
  }
  return mine;
}

// The same by counting: the want-th largest of the 32 lanes' maxima is a lower
// bound of the want-th largest key; the few keys at or above it (as a rule
// want to want + 4) are listed in shared memory, one per lane, and each lane
// counts how many come before its own. With inexact keys the bound is lowered
// by twice its error, so that the list holds the first want - 1 of the exact
// order too; where two successive ones are in doubt the list is ranked again
// by exact keys. False where more than 32 keys qualify.
template <int VPL>
__device__ __forceinline__ bool pick_by_count(const RouteOpArgs& a, int64_t row, const float (&key)[VPL], int want,
                                              float err, int64_t* smem, int lane, int* mine) {
  float best = key[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) best = fmaxf(best, key[i]);
  // (equal maxima leave together, which can only lower the bound)
  constexpr int kNone = static_cast<int>(0x80000000u);
  int m = order_int(best), bound_int = kNone;
  for (int k = 0; k < want; ++k) {
    bound_int = __reduce_max_sync(kAll, m);
    m = m == bound_int ? kNone : m;
  }
  const float bound = bound_int == kNone ? -INFINITY : order_float(bound_int);
  uint2* list = reinterpret_cast<uint2*>(smem);  // [32]
  const int n = list_above<VPL>(key, err > 0.f ? bound - key_gap(err, bound) : bound, list, lane);
  if (n > 32) return false;
  // (key, lower id first) as one unsigned number; 0 for no entry
  uint64_t own = 0;
  if (lane < n) {
    const uint2 u = list[lane];
    const float k0 = __uint_as_float(u.x) + 0.0f;  // -0 ties with 0
    own = (static_cast<uint64_t>(static_cast<uint32_t>(order_int(k0)) ^ 0x80000000u) << 32) | (0xffffu - u.y);
  }
  uint64_t* sorted = reinterpret_cast<uint64_t*>(smem);
  __syncwarp();
  sorted[lane] = own;
  __syncwarp();
  int before = 0;
  for (int j = 0; j < n; j += 2) {
    const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(sorted + j);
    before += (o.x > own ? 1 : 0) + (o.y > own ? 1 : 0);
  }
  __syncwarp();
  if (lane >= n) before = lane;  // entries of 0 stay behind
  sorted[before] = own;
  __syncwarp();
  own = sorted[lane];
  __syncwarp();
  int id = own != 0 ? static_cast<int>(0xffffu - static_cast<uint32_t>(own & 0xffffu)) : -1;
  if (err > 0.f) {
    const float k0 = order_float(static_cast<int>(static_cast<uint32_t>(own >> 32) ^ 0x80000000u));
    const float next = __shfl_down_sync(kAll, k0, 1);
    const int next_id = __shfl_down_sync(kAll, id, 1);
    // the first certain step at the K-th key or behind it; no pair before it may
    // be in doubt (behind true ties a key further down could belong before them)
    const bool sure = lane + 1 >= n || k0 - next > key_gap(err, k0);
    const int end = __ffs(__ballot_sync(kAll, sure) & (kAll << (want - 2))) - 1;
    const bool close = lane < end && !sure && !same_key(a, row, id, next_id);
    if (__any_sync(kAll, close)) id = rank_exact(a, row, id, n, lane, smem);
  }
  *mine = id;
  return true;
}

// One token's selection by one warp: lane k < K returns the k-th selected
// expert (-1: none left). Worked out in float; where some comparison is closer
// than the errors allow, again in double, whose order is the definition's.
template <int VPL>
__device__ __forceinline__ int select_token(const RouteOpArgs& a, int64_t row, const float* bias, int64_t* smem,
                                            int lane) {
  float key[VPL], err;
  bool doubt = false;
  load_row<VPL>(a, row, lane, key);
  if (!token_keys<VPL>(a, bias, row, smem, lane, key, &err, &doubt)) return -1;
  // with inexact keys one more than K, to see the key that just missed
  const int want = err > 0.f ? a.K + 1 : a.K;
  int mine = -1;
  if (!doubt && (want > kCountedMax || !pick_by_count<VPL>(a, row, key, want, err, smem, lane, &mine)))
    mine = pick_by_rounds<VPL>(a, row, key, want, err, lane, &doubt);
  if (doubt) mine = select_exact(a, row, lane, smem);
  return lane < a.K ? mine : -1;
}

// Weight of the expert lane k holds (id < 0: 0), among the selected ones. Sums
// are shifted by the largest exponent where that matters, so that renormalised
// weights keep their ratio where every score is below the smallest float.
template <int VPL>
__device__ __forceinline__ float token_weight(const RouteOpArgs& a, int64_t row, int id, int lane) {
  const bool on = id >= 0;
  const float z = on ? load_logit(a, row, id) : -INFINITY;
  float num, sum = 1.f;
  if (a.softmax && a.renormalise) {
    const float m = warp_max_fast(z);
    num = on ? expf(z - m) : 0.f;
  } else if (a.softmax) {
    float x[VPL];
    load_row<VPL>(a, row, lane, x);
    float m = x[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, x[i]);
    m = warp_max_fast(m);
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) sum += x[i] > -INFINITY ? expf(x[i] - m) : 0.f;
    sum = warp_sum_f(sum);
    num = on ? expf(z - m) : 0.f;
  } else {
    float t = fminf(z, 0.f);
    if (a.renormalise && __any_sync(kAll, on && t < -60.f)) t -= warp_max_fast(on ? t : -INFINITY);
    num = on ? __fdividef(expf(t), 1.f + expf(-fabsf(z))) : 0.f;
  }
  if (a.renormalise) sum = warp_sum_f(num);
  return on ? __fdividef(num, sum) * a.scale : 0.f;
}

// A warp's scratch: the list of the largest keys, or every key in double where
// keys can be inexact.
__host__ __device__ __forceinline__ size_t select_scratch(const RouteOpArgs& a) {
  const size_t keys = (a.n_groups > 1 || a.bias != nullptr) ? static_cast<size_t>(a.E + 1) / 2 * 16 : 0;
  return keys > kListBytes ? keys : kListBytes;
}

// The places of this CTA's selected slots: an expert's slots are ordered by
// token, so a slot's place is the expert's first place for this CTA plus the
// number of the CTA's earlier tokens that selected it (a bit count).
__device__ __forceinline__ void place_slots(const RouteOpArgs& a, const uint32_t* s_mask, const int* s_first, int t0,
                                            int nt) {
  const int64_t base = static_cast<int64_t>(t0) * a.K;
  for (int i = threadIdx.x; i < nt * a.K; i += blockDim.x) {
    const int t = i / a.K;
    const int e = a.idx[base + i];
    int p = -1;
    if (e >= 0) {
      const uint32_t lo = s_mask[2 * e], hi = s_mask[2 * e + 1];
      p = s_first[e] + (t < 32 ? __popc(lo & ((1u << t) - 1u)) : __popc(lo) + __popc(hi & ((1u << (t - 32)) - 1u)));
      a.rows[p] = static_cast<int>(base) + i;
    }
    a.pos[base + i] = p;
  }
}

// Exclusive scan of s_cnt[E] into s_first, the total in s_first[E], by the
// whole CTA. s_tmp: a word per warp.
__device__ __forceinline__ void scan_counts(const int* s_cnt, int* s_first, int* s_tmp, int E) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    const int v = e < E ? s_cnt[e] : 0;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 31) s_tmp[warp] = incl;
    __syncthreads();
    const int w = lane < warps ? s_tmp[lane] : 0;
    const int before = __reduce_add_sync(kAll, lane < warp ? w : 0);
    if (e < E) s_first[e] = carry + before + incl - v;
    carry += __reduce_add_sync(kAll, w);
    __syncthreads();
  }
  if (threadIdx.x == 0) s_first[E] = carry;
  __syncthreads();
}

}  // namespace

// Selection: one warp per token, cta_tokens tokens per CTA. Bound by the issue
// of a token's ~900 instructions and the latency between them (70% of issue slots
// busy), not by its logits: 32,768 tokens x 256 experts, sigmoid with bias, 4 of 8
// groups, 8 experts 34 us (33.6 MB at 1 TB/s), softmax alone 20 us; one token
// 2.6-3.6 us. A thread per token instead would leave 7 warps per SM at that size.
// 64 registers and 4 CTAs per SM: 3 or 5 CTAs were slower (60 and 66 against 51
// us). Where tokens can be in doubt, which takes several times as long, a CTA's
// warps take its tokens in common (35.2 us; each its own eighth of them 36.4);
// where they cannot, that costs more than it gives (softmax alone 21.4 against
// 20.2). Where the slots are to be grouped, a call that one cluster takes groups
// them too (each CTA reads the others' counts in their shared memory); otherwise
// each CTA leaves its counts per expert to the kernels below.
template <int VPL>
__global__ void __launch_bounds__(kThreads, VPL <= 8 ? 4 : 2) k_select(const __grid_constant__ RouteOpArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  const size_t scratch = select_scratch(a);
  uint32_t* s_mask = reinterpret_cast<uint32_t*>(raw + kWarps * scratch);  // [E][2]
  int* s_cnt = reinterpret_cast<int*>(s_mask + 2 * a.E);                      // [E]
  int* s_first = s_cnt + a.E;                                                 // [E + 1]
  __shared__ int s_tmp[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * a.cta_tokens;
  const int nt = min(a.cta_tokens, a.M - t0);  // below 1 in a cluster's last CTAs
  const bool grouping = a.offsets != nullptr;
  const bool take = nt > kWarps && (a.bias != nullptr || a.n_groups > 1);
  __shared__ int s_next;  // the next token that no warp has taken
  if (threadIdx.x == 0) s_next = kWarps;
  if (grouping) {
    for (int e = threadIdx.x; e < 2 * a.E; e += kThreads) s_mask[e] = 0;
    __syncthreads();
  }
  pdl_wait();
  pdl_trigger();
  int64_t* keys = reinterpret_cast<int64_t*>(raw + warp * scratch);
  __shared__ __align__(16) float s_bias[32 * VPL];
  load_bias<VPL>(a, s_bias);
  for (int t = warp, next; t < nt; t = next) {
    next = t + kWarps;
    if (take) {
      if (lane == 0) next = atomicAdd(&s_next, 1);
      next = __shfl_sync(kAll, next, 0);
    }
    const int64_t row = static_cast<int64_t>(t0 + t) * a.ld;
    const int id = select_token<VPL>(a, row, s_bias, keys, lane);
    const float w = token_weight<VPL>(a, row, id, lane);
    if (lane < a.K) {
      const int64_t o = static_cast<int64_t>(t0 + t) * a.K + lane;
      a.idx[o] = id;
      a.w[o] = w;
      if (grouping && id >= 0) atomicOr(&s_mask[2 * id + (t >> 5)], 1u << (t & 31));
    }
  }
  if (!grouping) return;
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    const int c = __popc(s_mask[2 * e]) + __popc(s_mask[2 * e + 1]);
    if (a.shape.cluster)
      s_cnt[e] = c;
    else
      a.hist[static_cast<int64_t>(e) * a.n_ctas + blockIdx.x] = c;
  }
  if (!a.shape.cluster) return;
  const int ctas = a.n_ctas, rank = blockIdx.x;
  int before[kPerThread];  // the expert's slots in earlier CTAs
  if (ctas > 1) {
    cluster_sync();  // every CTA's counts are there
    int total[kPerThread];
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const int e = threadIdx.x + j * kThreads;
      before[j] = total[j] = 0;
      for (int r = 0; e < a.E && r < ctas; ++r) {
        const int v = cluster_load(cluster_map(smem_u32(&s_cnt[e]), r));
        total[j] += v;
        before[j] += r < rank ? v : 0;
      }
    }
    cluster_sync();  // and read, so they may become the totals
#pragma unroll
    for (int j = 0; j < kPerThread; ++j)
      if (threadIdx.x + j * kThreads < a.E) s_cnt[threadIdx.x + j * kThreads] = total[j];
  }
  __syncthreads();
  scan_counts(s_cnt, s_first, s_tmp, a.E);
  if (rank == 0)
    for (int e = threadIdx.x; e <= a.E; e += kThreads) a.offsets[e] = s_first[e];
  if (ctas > 1) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPerThread; ++j)
      if (threadIdx.x + j * kThreads < a.E) s_first[threadIdx.x + j * kThreads] += before[j];
    __syncthreads();
  }
  place_slots(a, s_mask, s_first, t0, nt);
}

// One warp per expert: the exclusive scan of its counts over the CTAs (607 CTAs
// x 256 experts: with k_place 8 us, both latency).
__global__ void __launch_bounds__(kThreads) k_scan_hist(const RouteOpArgs a) {
  pdl_wait();
  pdl_trigger();
  const int e = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (e >= a.E) return;
  int32_t* h = a.hist + static_cast<int64_t>(e) * a.n_ctas;
  // Counts a lane loads before the first is added (all of 640 CTAs), and how many
  // scans of 32 run side by side (32,768 tokens: one at a time 45.4 us per call, four
  // 44.1; 257 tokens, which have 33 CTAs, 7.9 and 8.0).
  constexpr int kAhead = 20, kSide = 4;
  int run = 0;
  for (int c0 = 0; c0 < a.n_ctas; c0 += 32 * kAhead) {
    int v[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int c = c0 + 32 * j + lane;
      v[j] = c < a.n_ctas ? h[c] : 0;
    }
#pragma unroll
    for (int j0 = 0; j0 < kAhead; j0 += kSide) {
      if (c0 + 32 * j0 >= a.n_ctas) break;
      int incl[kSide];
#pragma unroll
      for (int j = 0; j < kSide; ++j) incl[j] = v[j0 + j];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int j = 0; j < kSide; ++j) {
          const int n = __shfl_up_sync(kAll, incl[j], o);
          if (lane >= o) incl[j] += n;
        }
      }
#pragma unroll
      for (int j = 0; j < kSide; ++j) {
        const int c = c0 + 32 * (j0 + j) + lane;
        if (c < a.n_ctas) h[c] = run + incl[j] - v[j0 + j];
        run += __shfl_sync(kAll, incl[j], 31);
      }
    }
  }
  if (lane == 0) a.totals[e] = run;
}

// Places the slots of the tokens that this CTA had in k_select, from the
// scanned counts.
__global__ void __launch_bounds__(kThreads) k_place(const RouteOpArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  uint32_t* s_mask = reinterpret_cast<uint32_t*>(raw);
  int* s_cnt = reinterpret_cast<int*>(s_mask + 2 * a.E);
  int* s_first = s_cnt + a.E;
  __shared__ int s_tmp[kWarps];
  const int t0 = blockIdx.x * a.cta_tokens;
  const int nt = min(a.cta_tokens, a.M - t0);
  for (int e = threadIdx.x; e < 2 * a.E; e += kThreads) s_mask[e] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const int64_t base = static_cast<int64_t>(t0) * a.K;
  int before[kPerThread];
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int e = threadIdx.x + j * kThreads;
    before[j] = 0;
    if (e < a.E) {
      before[j] = a.hist[static_cast<int64_t>(e) * a.n_ctas + blockIdx.x];
      s_cnt[e] = a.totals[e];
    }
  }
  for (int i = threadIdx.x; i < nt * a.K; i += kThreads) {
    const int t = i / a.K, e = a.idx[base + i];
    if (e >= 0) atomicOr(&s_mask[2 * e + (t >> 5)], 1u << (t & 31));
  }
  __syncthreads();
  scan_counts(s_cnt, s_first, s_tmp, a.E);
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= a.E; e += kThreads) a.offsets[e] = s_first[e];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPerThread; ++j)
    if (threadIdx.x + j * kThreads < a.E) s_first[threadIdx.x + j * kThreads] += before[j];
  __syncthreads();
  place_slots(a, s_mask, s_first, t0, nt);
}

cudaError_t launch_route_op(const RouteOpArgs& args, cudaStream_t s) {
  RouteOpArgs a = args;
  const size_t tail = static_cast<size_t>(4 * a.E + 1) * 4;
  const size_t smem = kWarps * select_scratch(a) + tail;
  const int vpl = a.E <= 64 ? 2 : a.E <= 128 ? 4 : a.E <= 256 ? 8 : 16;
  void (*k)(const RouteOpArgs) = vpl == 2   ? k_select<2>
                                 : vpl == 4 ? k_select<4>
                                 : vpl == 8 ? k_select<8>
                                            : k_select<16>;
  const int size = a.bf16_logits ? 2 : 4;
  const int part = vpl * size < 16 ? vpl * size : 16;
  a.vec = a.E % vpl == 0 && reinterpret_cast<uintptr_t>(a.logits) % part == 0 && a.ld * size % part == 0;
  a.group_size = a.E / a.n_groups;
  a.group_shift = -1;
  for (int b = 0; b <= 5; ++b)
    if (a.group_size == vpl << b) a.group_shift = b;
  cudaError_t e =
      launch_kernel<RouteOpArgs>(k, dim3(a.n_ctas), dim3(kThreads), smem, s, true, a, a.shape.cluster ? a.n_ctas : 1);
  if (e != cudaSuccess || a.offsets == nullptr || a.shape.cluster) return e;
  e = launch_kernel<RouteOpArgs>(k_scan_hist, dim3((a.E + kWarps - 1) / kWarps), dim3(kThreads), 0, s, true, a);
  if (e != cudaSuccess) return e;
  return launch_kernel<RouteOpArgs>(k_place, dim3(a.n_ctas), dim3(kThreads), tail, s, true, a);
}

// ---------------------------------------------------------------- combine

namespace {

__device__ __forceinline__ void add_row8(float (&acc)[8], float w, uint4 u) {
  const uint32_t wd[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    acc[2 * j] = fmaf(w, __uint_as_float(wd[j] << 16), acc[2 * j]);
    acc[2 * j + 1] = fmaf(w, __uint_as_float(wd[j] & 0xFFFF0000u), acc[2 * j + 1]);
  }
}

}  // namespace

// One thread per token and 8 columns; up to 8 rows' loads are in flight
// before the first is added. Bound by HBM: every y row is read once (16,384
// tokens x 8 rows of 2,048: 119 us, 7.0 TB/s of DRAM traffic).
__global__ void __launch_bounds__(kThreads) k_combine_rows(const CombineOpArgs a) {
  pdl_wait();
  pdl_trigger();
  const int chunks = a.H / 8;
  const int64_t gid = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t t = gid / chunks;
  if (t >= a.M) return;
  const int c = static_cast<int>(gid - t * chunks) * 8;
  float acc[8] = {};
  if (a.x != nullptr) {
    const float4* px = reinterpret_cast<const float4*>(a.x + t * a.H + c);
    const float4 u = px[0], v = px[1];
    acc[0] = u.x, acc[1] = u.y, acc[2] = u.z, acc[3] = u.w;
    acc[4] = v.x, acc[5] = v.y, acc[6] = v.z, acc[7] = v.w;
  }
  uint4 sh = make_uint4(0, 0, 0, 0);
  if (a.shared != nullptr) sh = *reinterpret_cast<const uint4*>(a.shared + t * a.H + c);
  for (int k0 = 0; k0 < a.K; k0 += 8) {
    uint4 r[8];
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] = 0.f;
      r[j] = make_uint4(0, 0, 0, 0);
      if (k0 + j < a.K) {
        const int p = a.pos[t * a.K + k0 + j];
        if (p >= 0 && p < a.n_rows) {
          w[j] = a.w[t * a.K + k0 + j];
          r[j] = *reinterpret_cast<const uint4*>(a.y + static_cast<int64_t>(p) * a.H + c);
        } else {
          w[j] = 0.f;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) add_row8(acc, w[j], r[j]);
  }
  if (a.shared != nullptr) add_row8(acc, 1.f, sh);
  float4* po = reinterpret_cast<float4*>(a.out + t * a.H + c);
  po[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  po[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
}

cudaError_t launch_combine_op(const CombineOpArgs& a, cudaStream_t s) {
  const int64_t n = static_cast<int64_t>(a.M) * (a.H / 8);
  const int64_t blocks = (n + kThreads - 1) / kThreads;
  return launch_kernel(k_combine_rows, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s, true, a);
}

}  // namespace clover
