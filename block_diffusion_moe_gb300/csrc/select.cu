// Expert selection and grouping (clover_route) and the weighted sum of expert
// rows (clover_moe_combine).
#include <math.h>

#include "launch.cuh"
#include "moe_ops.cuh"
#include "routing.cuh"
#include "sm100.cuh"

namespace clover {

namespace {

constexpr int kThreads = 256;  // 8 warps, one token each at a time
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float load_logit(const RouteOpArgs& a, int64_t row, int e) {
  float v = a.bf16_logits
                ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[row + e])
                : static_cast<const float*>(a.logits)[row + e];
  // +inf counts as the largest finite value, -0 as 0; NaN stays NaN
  return (v > 3.402823466e+38f ? 3.402823466e+38f : v) + 0.0f;
}

// The token's logits, expert lane + 32 i in slot i; -inf for NaN and past E.
template <int VPL>
__device__ __forceinline__ void load_row(const RouteOpArgs& a, int64_t row, int lane, float (&x)[VPL]) {
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    const float v = e < a.E ? load_logit(a, row, e) : -INFINITY;
    x[i] = v > -INFINITY ? v : -INFINITY;
  }
}

__device__ __forceinline__ double warp_max_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max_t(float v) { return warp_max_f(v); }
__device__ __forceinline__ double warp_max_t(double v) { return warp_max_d(v); }
__device__ __forceinline__ float warp_sum_t(float v) { return warp_sum_f(v); }
__device__ __forceinline__ double warp_sum_t(double v) { return warp_sum_d(v); }
__device__ __forceinline__ float exp_t(float v) { return expf(v); }
__device__ __forceinline__ double exp_t(double v) { return exp(v); }

// One token's selection by one warp, in T. Expert lane + 32 i sits in slot i;
// x holds the logits, -inf where the expert is not live. Lane k < K returns
// the k-th selected expert (-1: none left).
//
// In float, *unsure is set where the order could be another one in exact
// arithmetic: two keys (or the ranks on either side of the group border)
// closer than twice the largest error a key can have. A score's error is
// below 2^-19 of the largest score (exp and quotient a few roundings each, the
// softmax's sum up to 21), the sum with the bias adds half a unit of the key.
// Logits used as keys are exact. The caller then repeats the token in double, whose order is the
// definition's.
template <int VPL, typename T>
__device__ __forceinline__ int select_token(const RouteOpArgs& a, const float (&x)[VPL], T* s_keys, int lane,
                                            bool* unsure) {
  constexpr bool kExact = sizeof(T) == 8;
  const T ninf = -static_cast<T>(INFINITY);
  const bool need_scores = a.bias != nullptr || (a.n_groups > 1 && a.group_rank == 2);
  T key[VPL];   // what experts are ordered by
  T total[VPL]; // score + bias, what group ranks sum
  T err = 0;    // bound on the error of a key or half a rank
  if (need_scores) {
    T m = ninf;
    if (a.softmax) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) m = fmax(m, static_cast<T>(x[i]));
      m = warp_max_t(m);
      T sum = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        total[i] = x[i] > -INFINITY ? exp_t(static_cast<T>(x[i]) - m) : static_cast<T>(0);
        sum += total[i];
      }
      sum = warp_sum_t(sum);
      const T inv = static_cast<T>(1) / sum;  // sum >= 1 where any expert is live
#pragma unroll
      for (int i = 0; i < VPL; ++i) total[i] = kExact ? total[i] / sum : total[i] * inv;
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        total[i] = static_cast<T>(1) / (static_cast<T>(1) + exp_t(-static_cast<T>(x[i])));
    }
    T s_max = 0, k_max = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      const bool on = x[i] > -INFINITY;
      if (!kExact && on) s_max = fmax(s_max, total[i]);
      const float b = (a.bias != nullptr && e < a.E) ? a.bias[e] : 0.f;
      const bool live = on && b > -INFINITY;  // false for NaN too
      total[i] = live ? total[i] + static_cast<T>(b) : ninf;
      if (!kExact && live) k_max = fmax(k_max, fabs(total[i]));
    }
    if (!kExact) err = warp_max_t(s_max) * static_cast<T>(1.9e-6) + warp_max_t(k_max) * static_cast<T>(1.2e-7) + static_cast<T>(1e-37);
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) key[i] = a.bias != nullptr ? total[i] : static_cast<T>(x[i]);
  bool doubt = false;

  if (a.n_groups > 1) {
    // keys in shared memory, one lane per group
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 32 * i < a.E) s_keys[lane + 32 * i] = a.group_rank == 2 ? total[i] : key[i];
    __syncwarp();
    const int size = a.E / a.n_groups;
    T b1 = ninf, b2 = ninf;
    if (lane < a.n_groups) {
      int j = lane % size;  // each lane starts elsewhere in its group: other banks
      for (int n = 0; n < size; ++n) {
        const T v = s_keys[lane * size + j];
        if (v > b1) {
          b2 = b1;
          b1 = v;
        } else if (v > b2) {
          b2 = v;
        }
        if (++j == size) j = 0;
      }
    }
    __syncwarp();
    const T rank = (a.group_rank == 2 && b2 > ninf) ? b1 + b2 : b1;
    int before = 0;
    for (int g = 0; g < a.n_groups; ++g) {
      const T r = __shfl_sync(0xffffffffu, rank, g);
      before += (r > rank || (r == rank && g < lane)) ? 1 : 0;
    }
    const bool stays = lane < a.n_groups && before < a.top_groups;
    const uint32_t mask = __ballot_sync(0xffffffffu, stays);
    if (!kExact && err > 0) {
      const T low = -warp_max_t(stays ? -rank : ninf);
      const T high = warp_max_t(lane < a.n_groups && !stays ? rank : ninf);
      doubt = high > ninf && !(low - high > (a.group_rank == 2 ? 4 : 2) * err);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      if (e < a.E && ((mask >> (e / size)) & 1u) == 0) key[i] = ninf;
    }
  }

  // K rounds: the largest key, the lowest id holding it; one more round in
  // float to see the key that just missed
  const bool check = !kExact && a.bias != nullptr;
  const int rounds = check ? a.K + 1 : a.K;
  int mine = -1;
  T last = 0, last_x = 0, last_b = 0;
  for (int k = 0; k < rounds; ++k) {
    T best = ninf;
    int at = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    const T top = warp_max_t(best);
    if (!(top > ninf)) break;  // uniform: no live expert left
    const int id = (best == top) ? lane + 32 * at : 0x7fffffff;
    const int win = __reduce_min_sync(0xffffffffu, id);
    if (check) {
      float wx = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i == win / 32) wx = x[i];
      wx = __shfl_sync(0xffffffffu, wx, win & 31);
      const float wb = a.bias[win];
      // the same logit and bias give the same key: a real tie, by id
      if (k > 0 && !(last - top > 2 * err) && !(wx == last_x && wb == last_b)) doubt = true;
      last = top;
      last_x = wx;
      last_b = wb;
    }
    if (k < a.K && lane == k) mine = win;
    if ((win & 31) == lane) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i == win / 32) key[i] = ninf;
    }
  }
  if (!kExact) *unsure = doubt;
  return mine;
}

template <int VPL>
__device__ __noinline__ int select_token_exact(const RouteOpArgs& a, int64_t row, double* s_keys, int lane) {
  float x[VPL];
  load_row<VPL>(a, row, lane, x);
  return select_token<VPL, double>(a, x, s_keys, lane, nullptr);
}

// Weight of the expert lane k holds (id < 0: 0), among the selected ones.
// Shifted by the largest exponent, so that renormalised weights keep their
// ratio where every score is below the smallest float.
template <int VPL>
__device__ __forceinline__ float token_weight(const RouteOpArgs& a, const float (&x)[VPL], int64_t row, int id) {
  const bool on = id >= 0;
  const float z = on ? load_logit(a, row, id) : -INFINITY;
  float num, e;
  if (a.softmax) {
    float m = z;
    if (!a.renormalise) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) m = fmaxf(m, x[i]);
    }
    m = warp_max_f(m);
    num = on ? expf(z - m) : 0.f;
    if (!a.renormalise) {
      e = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) e += x[i] > -INFINITY ? expf(x[i] - m) : 0.f;
      e = warp_sum_f(e);
    } else {
      e = warp_sum_f(num);
    }
  } else {
    const float t = fminf(z, 0.f);
    const float shift = a.renormalise ? warp_max_f(on ? t : -INFINITY) : 0.f;
    num = on ? expf(t - shift) / (1.f + expf(-fabsf(z))) : 0.f;
    e = a.renormalise ? warp_sum_f(num) : 1.f;
  }
  return on ? num / e * a.scale : 0.f;
}

// The places of this CTA's selected slots: an expert's slots are ordered by
// token, so a slot's place is the expert's first place for this CTA plus the
// number of the CTA's earlier tokens that selected it (a bit count).
__device__ __forceinline__ void place_slots(const RouteOpArgs& a, const uint32_t* s_mask, const int* s_first, int t0,
                                            int nt) {
  const int64_t base = static_cast<int64_t>(t0) * a.K;
  for (int i = threadIdx.x; i < nt * a.K; i += kThreads) {
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

// Exclusive scan of s_cnt[E] (E <= 2 kThreads) into s_first, the total in
// s_first[E].
__device__ __forceinline__ void scan_counts(const int* s_cnt, int* s_first, int* s_tmp, int E) {
  const int e = 2 * threadIdx.x;
  const int c0 = e < E ? s_cnt[e] : 0, c1 = e + 1 < E ? s_cnt[e + 1] : 0;
  int total;
  const int x = block_excl_scan(c0 + c1, s_tmp, &total);
  if (e < E) s_first[e] = x;
  if (e + 1 < E) s_first[e + 1] = x + c0;
  if (threadIdx.x == 0) s_first[E] = total;
  __syncthreads();
}

}  // namespace

// Selection: one warp per token, cta_tokens tokens per CTA. Where the slots
// are to be grouped, each CTA also leaves its counts per expert; a call that
// one CTA takes groups them itself.
template <int VPL>
__global__ void __launch_bounds__(kThreads) k_select(const RouteOpArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  double* s_keys = reinterpret_cast<double*>(raw);  // [kWarps][E], only with groups
  uint32_t* s_mask = reinterpret_cast<uint32_t*>(s_keys + (a.n_groups > 1 ? kWarps * a.E : 0));  // [E][2]
  int* s_cnt = reinterpret_cast<int*>(s_mask + 2 * a.E);                                          // [E]
  int* s_first = s_cnt + a.E;                                                                     // [E + 1]
  __shared__ int s_tmp[17];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * a.cta_tokens;
  const int nt = min(a.cta_tokens, a.M - t0);
  const bool grouping = a.offsets != nullptr;
  if (grouping) {
    for (int e = threadIdx.x; e < 2 * a.E; e += kThreads) s_mask[e] = 0;
    __syncthreads();
  }
  pdl_wait();
  pdl_trigger();
  double* keys = s_keys + static_cast<size_t>(warp) * a.E;
  for (int t = warp; t < nt; t += kWarps) {
    const int64_t row = static_cast<int64_t>(t0 + t) * a.ld;
    float x[VPL];
    load_row<VPL>(a, row, lane, x);
    bool unsure = false;
    int id = select_token<VPL, float>(a, x, reinterpret_cast<float*>(keys), lane, &unsure);
    if (unsure) id = select_token_exact<VPL>(a, row, keys, lane);
    const float w = token_weight<VPL>(a, x, row, id);
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
    if (a.n_ctas == 1)
      s_cnt[e] = c;
    else
      a.hist[static_cast<int64_t>(e) * a.n_ctas + blockIdx.x] = c;
  }
  if (a.n_ctas > 1) return;
  __syncthreads();
  scan_counts(s_cnt, s_first, s_tmp, a.E);
  for (int e = threadIdx.x; e <= a.E; e += kThreads) a.offsets[e] = s_first[e];
  place_slots(a, s_mask, s_first, t0, nt);
}

// One warp per expert: the exclusive scan of its counts over the CTAs.
__global__ void __launch_bounds__(kThreads) k_scan_hist(const RouteOpArgs a) {
  pdl_wait();
  pdl_trigger();
  const int e = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (e >= a.E) return;
  int32_t* h = a.hist + static_cast<int64_t>(e) * a.n_ctas;
  int run = 0;
  for (int c0 = 0; c0 < a.n_ctas; c0 += 32) {
    const int c = c0 + lane;
    const int v = c < a.n_ctas ? h[c] : 0;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    if (c < a.n_ctas) h[c] = run + incl - v;
    run += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) a.totals[e] = run;
}

// Each CTA takes the tokens it had in k_select and places their slots.
__global__ void __launch_bounds__(kThreads) k_place(const RouteOpArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  uint32_t* s_mask = reinterpret_cast<uint32_t*>(raw);
  int* s_cnt = reinterpret_cast<int*>(s_mask + 2 * a.E);
  int* s_first = s_cnt + a.E;
  __shared__ int s_tmp[17];
  const int t0 = blockIdx.x * a.cta_tokens;
  const int nt = min(a.cta_tokens, a.M - t0);
  for (int e = threadIdx.x; e < 2 * a.E; e += kThreads) s_mask[e] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const int64_t base = static_cast<int64_t>(t0) * a.K;
  for (int i = threadIdx.x; i < nt * a.K; i += kThreads) {
    const int t = i / a.K, e = a.idx[base + i];
    if (e >= 0) atomicOr(&s_mask[2 * e + (t >> 5)], 1u << (t & 31));
  }
  for (int e = threadIdx.x; e < a.E; e += kThreads) s_cnt[e] = a.totals[e];
  __syncthreads();
  scan_counts(s_cnt, s_first, s_tmp, a.E);
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= a.E; e += kThreads) a.offsets[e] = s_first[e];
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kThreads)
    s_first[e] += a.hist[static_cast<int64_t>(e) * a.n_ctas + blockIdx.x];
  __syncthreads();
  place_slots(a, s_mask, s_first, t0, nt);
}

cudaError_t launch_route_op(const RouteOpArgs& a, cudaStream_t s) {
  const size_t tail = static_cast<size_t>(4 * a.E + 1) * 4;
  const size_t smem = (a.n_groups > 1 ? static_cast<size_t>(kWarps) * a.E * 8 : 0) + tail;
  void (*k)(const RouteOpArgs) = a.E <= 64 ? k_select<2> : a.E <= 128 ? k_select<4> : a.E <= 256 ? k_select<8>
                                                                                                  : k_select<16>;
  cudaError_t e = launch_kernel(k, dim3(a.n_ctas), dim3(kThreads), smem, s, true, a);
  if (e != cudaSuccess || a.offsets == nullptr || a.n_ctas == 1) return e;
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
// before the first is added. Bound by HBM: every y row is read once.
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
