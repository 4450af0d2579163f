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

// The row of the scale tiles that belongs to row i, by one warp. False for a
// grouped row in no group: behind the last one, or in none by offsets that do
// not ascend.
__device__ __forceinline__ bool scale_row(const Fp4QuantArgs& a, int64_t i, int lane, int64_t* r) {
  if (a.offsets == nullptr) {
    const int64_t m = i / a.mat_rows;
    *r = m * ((a.mat_rows + 127) / 128 * 128) + (i - m * a.mat_rows);
    return true;
  }
  const int row = static_cast<int>(i);
  const int g = warp_search(a.n_groups, row, [&](int j) { return a.offsets[j]; });
  const int n = static_cast<int>(a.n_rows);
  const int off = group_offset(a.offsets, g, n);
  if (off > row || row >= group_offset(a.offsets, g + 1, n)) return false;
  *r = (off / 128 + static_cast<int64_t>(g)) * 128 + (i - off);
  return true;
}

}  // namespace

// One warp per row, one lane per block of columns: a block's values stay in
// registers between its maximum and its codes, so x is read once. Matrices are
// bound by HBM (64 x 1,024 x 2,048 bf16 to NV: 52 us, 343 MB at 6.6 TB/s); rows
// gathered eight times each, which come from L2, by the arithmetic (65,536 rows
// of 2,048 to MX: 43 us, the ALU pipe two thirds busy). A division per element
// instead of the products below: 62 us for the matrices.
// kUnit: scale_exp is 0.
template <bool kMx, bool kBf16, bool kUnit>
__global__ void __launch_bounds__(kThreads) k_quantize_fp4(const Fp4QuantArgs a) {
  constexpr int kBlock = kMx ? 32 : 16;
  constexpr int kWords = kBlock * (kBf16 ? 2 : 4) / 4;  // of a block's input
  // NV, bf16: 2^-scale_exp / s, rounded up, for each scale byte (0 for none)
  __shared__ float s_inv[128];
  if (!kMx && kBf16) {
    if (threadIdx.x < 128) s_inv[threadIdx.x] = scale_inverse(threadIdx.x, a.mul);
    __syncthreads();
  }
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (i >= a.n_rows) return;
  int64_t sr;
  if (!scale_row(a, i, lane, &sr)) return;
  int64_t src = i;
  if (a.offsets != nullptr) {
    if (a.src_rows != nullptr) {
      const int v = a.src_rows[i];
      src = v < 0 ? -1 : (a.src_shift >= 0 ? v >> a.src_shift : v / a.src_div);
    }
    if (src >= a.n_src) src = -1;
  }
  const uint8_t* row = static_cast<const uint8_t*>(a.x) + src * a.ldx * (kBf16 ? 2 : 4);
  const int nb = a.cols / kBlock, ct = (nb + 3) / 4;
  uint8_t* tile = a.scales + (sr / 128) * ct * 512 + (sr % 32) * 16 + (sr % 128) / 32 * 4;
  uint8_t* codes = a.codes + i * (a.cols / 2);
  const bool wide = a.wide;
#pragma unroll 2
  for (int b = lane; b < nb; b += 32) {
    uint32_t in[kWords];
    if (src >= 0) {
#pragma unroll
      for (int v = 0; v < kWords / 8; ++v)
        load32b(row + b * (kWords * 4) + v * 32, wide, *reinterpret_cast<uint32_t(*)[8]>(&in[8 * v]));
    } else {
#pragma unroll
      for (int v = 0; v < kWords; ++v) in[v] = 0;
    }
    uint32_t words[kBlock / 8];
    const uint32_t sb = quantize_block<kMx, kBf16, kUnit>(in, a.mul, s_inv, words);
    if (kMx)
      *reinterpret_cast<uint4*>(codes + b * 16) = make_uint4(words[0], words[1], words[kMx ? 2 : 0], words[kMx ? 3 : 1]);
    else
      *reinterpret_cast<uint2*>(codes + b * 8) = make_uint2(words[0], words[1]);
    tile[(b / 4) * 512 + b % 4] = static_cast<uint8_t>(sb);
  }
}

// The other way: one warp per row, one lane per 16 columns. Bound by HBM (the
// same sizes: 52 and 54 us, 6.6 TB/s).
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
#pragma unroll 2
  for (int c = lane; c < a.cols / 16; c += 32) {
    const int b = kMx ? c / 2 : c;
    const uint32_t sb = tile[(b / 4) * 512 + b % 4];
    const float s = kMx ? e8m0_to_float(sb) : e4m3_to_float(sb);
    // a 2^scale_exp below 1 first: either way both products are then exact unless
    // the result itself leaves bf16's range (6 x 2^126 x 2^-3 does not)
    const float f1 = a.mul < 1.f ? a.mul : s, f2 = a.mul < 1.f ? s : a.mul;
    const uint2 u = *reinterpret_cast<const uint2*>(codes + c * 8);
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 v = e2m1_values(((j < 4 ? u.x : u.y) >> (8 * (j & 3))) & 0xFFu);
      const __nv_bfloat162 p = __floats2bfloat162_rn(v.x * f1 * f2, v.y * f1 * f2);
      o[j] = *reinterpret_cast<const uint32_t*>(&p);
    }
    store32b(a.out + i * a.cols + c * 16, a.wide, o);
  }
}

namespace {
dim3 row_grid(const Fp4QuantArgs& a) { return dim3(static_cast<unsigned>((a.n_rows + kWarps - 1) / kWarps)); }
}  // namespace

cudaError_t launch_quantize_fp4(const Fp4QuantArgs& args, bool mx, cudaStream_t s) {
  Fp4QuantArgs a = args;
  a.src_shift = -1;
  for (int b = 0; b < 31; ++b)
    if (a.src_div == 1 << b) a.src_shift = b;
  a.wide = reinterpret_cast<uintptr_t>(a.x) % 32 == 0 && a.ldx * (a.bf16_x ? 2 : 4) % 32 == 0;
  void (*k)(const Fp4QuantArgs);
  if (a.mul == 1.f)
    k = mx ? (a.bf16_x ? k_quantize_fp4<true, true, true> : k_quantize_fp4<true, false, true>)
           : (a.bf16_x ? k_quantize_fp4<false, true, true> : k_quantize_fp4<false, false, true>);
  else
    k = mx ? (a.bf16_x ? k_quantize_fp4<true, true, false> : k_quantize_fp4<true, false, false>)
           : (a.bf16_x ? k_quantize_fp4<false, true, false> : k_quantize_fp4<false, false, false>);
  return launch_kernel(k, row_grid(a), dim3(kThreads), 0, s, true, a);
}

cudaError_t launch_dequantize_fp4(const Fp4QuantArgs& args, bool mx, cudaStream_t s) {
  Fp4QuantArgs a = args;
  a.wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
  void (*k)(const Fp4QuantArgs) = mx ? k_dequantize_fp4<true> : k_dequantize_fp4<false>;
  return launch_kernel(k, row_grid(a), dim3(kThreads), 0, s, true, a);
}

}  // namespace clover
