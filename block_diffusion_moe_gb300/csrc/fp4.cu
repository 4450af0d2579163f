// Microscaled 4-bit floating point: quantisation and what the codes stand for.
//
// Formats (include/clover.h): e2m1 codes with one scale per 16 columns (NV,
// e4m3) or 32 columns (MX, e8m0); scales in 512-byte tiles of 128 rows x 4
// blocks, the order the tensor core's scale copy reads.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "fp4.cuh"
#include "launch.cuh"
#include "moe_ops.cuh"
#include "sm100.cuh"

namespace clover {

namespace {

constexpr int kThreads = 256;  // 8 warps, one row each
constexpr int kWarps = kThreads / 32;

// Two values to two e2m1 codes (nearest, ties to the even code, at most 6),
// `lo` in the low nibble.
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The two e2m1 codes of a byte as two halves.
__device__ __forceinline__ float2 e2m1_values(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(byte));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// The row of the scale tiles that belongs to row i, by one warp. False for a
// grouped row behind the last group.
__device__ __forceinline__ bool scale_row(const Fp4QuantArgs& a, int64_t i, int lane, int64_t* r) {
  if (a.offsets == nullptr) {
    const int64_t m = i / a.mat_rows;
    *r = m * ((a.mat_rows + 127) / 128 * 128) + (i - m * a.mat_rows);
    return true;
  }
  // group of row i: the number of groups that end at or before it
  const int n = static_cast<int>(a.n_rows);
  int below = 0;
  for (int g = lane; g < a.n_groups; g += 32) below += group_offset(a.offsets, g + 1, n) <= i ? 1 : 0;
  const int g = warp_sum_i(below);
  if (g >= a.n_groups) return false;
  const int off = group_offset(a.offsets, g, n);
  if (off > i) return false;  // offsets that do not ascend
  *r = (off / 128 + static_cast<int64_t>(g)) * 128 + (i - off);
  return true;
}

template <bool kBf16>
struct Src;
template <>
struct Src<true> {
  using T = __nv_bfloat16;
};
template <>
struct Src<false> {
  using T = float;
};

}  // namespace

// One warp per row, one lane per block of columns: a block's values stay in
// registers between its maximum and its codes, so x is read once. Bound by
// HBM (2.56 bytes per bf16 element with NV scales).
//
// The codes are exact. MX: y / s is exact (s a power of two). NV with fp32
// input: the correctly rounded quotient lies on the same side of every border
// (or on it) as the exact one, as border * s has 7 significant bits. NV with
// bf16 input: a quotient that is not on a border is at least 2^-9 of it away,
// so y * (1 / s), which is off by at most 2^-23, is rounded to a multiple of
// 2^-14 (the borders are multiples of 2^-2): a tie becomes exactly a tie.
template <bool kMx, bool kBf16>
__global__ void __launch_bounds__(kThreads) k_quantize_fp4(const Fp4QuantArgs a) {
  constexpr int kBlock = kMx ? 32 : 16;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (i >= a.n_rows) return;
  int64_t sr;
  if (!scale_row(a, i, lane, &sr)) return;
  int64_t src = i;
  if (a.offsets != nullptr) {
    if (a.src_rows != nullptr) src = a.src_rows[i] < 0 ? -1 : a.src_rows[i] / a.src_div;
    if (src >= a.n_src) src = -1;
  }
  const typename Src<kBf16>::T* row = static_cast<const typename Src<kBf16>::T*>(a.x) + src * a.ldx;
  const int nb = a.cols / kBlock, ct = (nb + 3) / 4;
  uint8_t* tile = a.scales + (sr / 128) * ct * 512 + (sr % 32) * 16 + (sr % 128) / 32 * 4;
  uint8_t* codes = a.codes + i * (a.cols / 2);
  for (int b = lane; b < nb; b += 32) {
    float y[kBlock];
    uint32_t top = 0;  // largest |x| as bits: NaN above infinity above every number
    if (src < 0) {
#pragma unroll
      for (int j = 0; j < kBlock; ++j) y[j] = 0.f;
    } else if (kBf16) {
      const uint4* p = reinterpret_cast<const uint4*>(row + b * kBlock);
#pragma unroll
      for (int v = 0; v < kBlock / 8; ++v) {
        const uint4 u = p[v];
        const uint32_t wd[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[8 * v + 2 * j] = __uint_as_float(wd[j] << 16);
          y[8 * v + 2 * j + 1] = __uint_as_float(wd[j] & 0xFFFF0000u);
        }
      }
    } else {
      const float4* p = reinterpret_cast<const float4*>(row + b * kBlock);
#pragma unroll
      for (int v = 0; v < kBlock / 4; ++v) {
        const float4 u = p[v];
        y[4 * v] = u.x, y[4 * v + 1] = u.y, y[4 * v + 2] = u.z, y[4 * v + 3] = u.w;
      }
    }
#pragma unroll
    for (int j = 0; j < kBlock; ++j) {
      y[j] *= a.mul;
      top = max(top, __float_as_uint(y[j]) & 0x7FFFFFFFu);
    }
    const bool finite = top < 0x7F800000u;
    const float amax = __uint_as_float(top);
    uint32_t sb;
    float s, inv;
    if (kMx) {
      const int e = max(static_cast<int>(top >> 23) - 129, -127);  // floor(log2 amax) - 2 (subnormals: -127)
      sb = finite ? static_cast<uint32_t>(e + 127) : 0xFFu;
      inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      s = 0.f;
    } else {
      sb = finite ? __nv_cvt_float_to_fp8(__fdiv_rn(amax, 6.0f), __NV_SATFINITE, __NV_E4M3) : 0x7Fu;
      s = e4m3_to_float(sb);
      inv = s > 0.f ? __frcp_rn(s) : 0.f;
    }
    uint32_t words[kBlock / 8];
#pragma unroll
    for (int wd = 0; wd < kBlock / 8; ++wd) {
      uint32_t word = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float v = y[8 * wd + 2 * j + h];
          if (kMx) {
            q[h] = v * inv;
          } else if (kBf16) {
            // |v| first: the sum below would lose the sign of a small one
            const float m = __fadd_rn(__fmaf_rn(fabsf(v), inv, 768.0f), -768.0f);
            q[h] = copysignf(m, v);
          } else {
            q[h] = inv > 0.f ? __fdiv_rn(v, s) : 0.f;
          }
        }
        word |= e2m1_pair(q[0], q[1]) << (8 * j);
      }
      words[wd] = (finite && (kMx || inv > 0.f)) ? word : 0u;
    }
    if (kMx)
      *reinterpret_cast<uint4*>(codes + b * 16) = make_uint4(words[0], words[1], words[kMx ? 2 : 0], words[kMx ? 3 : 1]);
    else
      *reinterpret_cast<uint2*>(codes + b * 8) = make_uint2(words[0], words[1]);
    tile[(b / 4) * 512 + b % 4] = static_cast<uint8_t>(sb);
  }
}

// The other way: one warp per row, one lane per 16 columns.
template <bool kMx>
__global__ void __launch_bounds__(kThreads) k_dequantize_fp4(const Fp4QuantArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (i >= a.n_rows) return;
  int64_t sr;
  if (!scale_row(a, i, lane, &sr)) return;
  const int ct = ((kMx ? a.cols / 32 : a.cols / 16) + 3) / 4;
  const uint8_t* tile = a.scales + (sr / 128) * ct * 512 + (sr % 32) * 16 + (sr % 128) / 32 * 4;
  const uint8_t* codes = a.codes + i * (a.cols / 2);
  for (int c = lane; c < a.cols / 16; c += 32) {
    const int b = kMx ? c / 2 : c;
    const uint32_t sb = tile[(b / 4) * 512 + b % 4];
    const float s = kMx ? e8m0_to_float(sb) : e4m3_to_float(sb);
    const uint2 u = *reinterpret_cast<const uint2*>(codes + c * 8);
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 v = e2m1_values(((j < 4 ? u.x : u.y) >> (8 * (j & 3))) & 0xFFu);
      const __nv_bfloat162 p = __floats2bfloat162_rn(v.x * s * a.mul, v.y * s * a.mul);
      o[j] = *reinterpret_cast<const uint32_t*>(&p);
    }
    uint4* dst = reinterpret_cast<uint4*>(a.out + i * a.cols + c * 16);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

namespace {
dim3 row_grid(const Fp4QuantArgs& a) { return dim3(static_cast<unsigned>((a.n_rows + kWarps - 1) / kWarps)); }
}  // namespace

cudaError_t launch_quantize_fp4(const Fp4QuantArgs& a, bool mx, cudaStream_t s) {
  void (*k)(const Fp4QuantArgs) = mx ? (a.bf16_x ? k_quantize_fp4<true, true> : k_quantize_fp4<true, false>)
                                     : (a.bf16_x ? k_quantize_fp4<false, true> : k_quantize_fp4<false, false>);
  return launch_kernel(k, row_grid(a), dim3(kThreads), 0, s, true, a);
}

cudaError_t launch_dequantize_fp4(const Fp4QuantArgs& a, bool mx, cudaStream_t s) {
  void (*k)(const Fp4QuantArgs) = mx ? k_dequantize_fp4<true> : k_dequantize_fp4<false>;
  return launch_kernel(k, row_grid(a), dim3(kThreads), 0, s, true, a);
}

}  // namespace clover
