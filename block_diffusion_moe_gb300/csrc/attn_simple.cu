// Attention, one warp per query row and head: the running maximum and sum of a
// softmax over one key at a time, all in fp32.
#include <math.h>

#include "attn_ops.cuh"
#include "launch.cuh"
#include "sm100.cuh"

namespace clover {

namespace {

constexpr int kWarps = 8;

// kPer consecutive elements of a 4-bit row, from element e.
template <int kPer>
__device__ __forceinline__ void row4(const uint8_t* codes, const uint8_t* scales, int row, int dim, int e, float (&x)[kPer]) {
  const float s = e4m3_to_float(scales[row * (dim / 16) + e / 16]);
#pragma unroll
  for (int i = 0; i < kPer / 2; ++i) {
    const float2 v = e2m1_values(codes[row * (dim / 2) + e / 2 + i]);
    x[2 * i] = v.x * s;
    x[2 * i + 1] = v.y * s;
  }
}

template <int kPer>
__device__ __forceinline__ void row16(const AttnRows& r, int row, int head, int e, float (&x)[kPer]) {
  const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(r.data + row * r.row + head * r.head) + e;
#pragma unroll
  for (int i = 0; i < kPer; ++i) x[i] = __bfloat162float(p[i]);
}

}  // namespace

template <int kDim, bool kCached>
__global__ void __launch_bounds__(kWarps * 32) k_attention_simple(const AttnArgs a) {
  constexpr int kPer = kDim / 32;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (w >= static_cast<int64_t>(a.s.n_rows) * a.q_heads) return;
  const int row = static_cast<int>(w / a.q_heads), h = static_cast<int>(w - static_cast<int64_t>(row) * a.q_heads);
  const int i = seq_of_row(a.s, row);
  if (i < 0) return;
  const SeqSpan sp = seq_span(a.s, i);
  if (row >= sp.row0 + sp.rows) return;
  const int limit = seen(sp.len - sp.rows + row - sp.row0, sp.len, a.block);
  const int kh = h / a.group, e = lane * kPer;
  float q[kPer], acc[kPer] = {}, m = -INFINITY, l = 0.f;
  row16<kPer>(a.q, row, h, e, q);
  for (int j = 0; j < limit; ++j) {
    float k[kPer], v[kPer];
    if (kCached) {
      const uint8_t* six = kv_sixteen(a.c, a.s, i, kh, j);
      if (six == nullptr) continue;
      row4<kPer>(six, six + 8 * kDim, j % 16, kDim, e, k);
      row4<kPer>(six + 9 * kDim, six + 17 * kDim, j % 16, kDim, e, v);
    } else {
      row16<kPer>(a.k, sp.key0 + j, kh, e, k);
      row16<kPer>(a.v, sp.key0 + j, kh, e, v);
    }
    float z = 0.f;
#pragma unroll
    for (int d = 0; d < kPer; ++d) z += q[d] * k[d];
    z = warp_sum_f(z) * a.scale_log2;
    if (z == -INFINITY) continue;
    const float m1 = fmaxf(m, z), f = exp2f(m - m1), p = exp2f(z - m1);  // (a NaN z: p is NaN)
    l = l * f + p;
#pragma unroll
    for (int d = 0; d < kPer; ++d) acc[d] = acc[d] * f + p * v[d];
    m = m1;
  }
  const float inv = l == 0.f ? 0.f : a.c.v_mul / l;
  __nv_bfloat16* o = a.out + (static_cast<int64_t>(row) * a.q_heads + h) * kDim + e;
#pragma unroll
  for (int d = 0; d < kPer; ++d) o[d] = __float2bfloat16_rn(acc[d] * inv);
  if (a.lse != nullptr && lane == 0)
    a.lse[static_cast<int64_t>(row) * a.q_heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

cudaError_t launch_attention_simple(const AttnArgs& a, bool cached, cudaStream_t s) {
  void (*k)(const AttnArgs) = a.c.dim == 64 ? (cached ? k_attention_simple<64, true> : k_attention_simple<64, false>)
                                            : (cached ? k_attention_simple<128, true> : k_attention_simple<128, false>);
  const int64_t n = static_cast<int64_t>(a.s.n_rows) * a.q_heads;
  return launch_kernel(k, dim3(static_cast<unsigned>((n + kWarps - 1) / kWarps)), dim3(kWarps * 32), 0, s, true, a);
}

}  // namespace clover
