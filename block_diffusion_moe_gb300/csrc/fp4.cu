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

// Eight values to e2m1 codes (nearest, ties to the even code, at most 6), the
// first in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1_word(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The two e2m1 codes of a byte as floats.
__device__ __forceinline__ float2 e2m1_values(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(byte));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// 32 bytes per lane: one access where the address allows it (a whole sector per
// lane; two of 16 bytes touch every sector twice).
__device__ __forceinline__ void load32b(const void* p, bool wide, uint32_t (&w)[8]) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 u = static_cast<const uint4*>(p)[0], v = static_cast<const uint4*>(p)[1];
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w, w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
  }
}
__device__ __forceinline__ void store32b(void* p, bool wide, const uint32_t (&w)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "l"(p)
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

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
//
// The codes are exact. MX: y / s is exact (s a power of two). NV with fp32
// input: the correctly rounded quotient lies on the same side of every border
// (or on it) as the exact one, as border * s has 7 significant bits. NV with
// bf16 input: a quotient that is not on a border is at least 2^-9 of it away,
// far more than x * (1 / s) is off; on a border, with 1 / s rounded up and the
// product cut off, the product is the border itself (for each of the 8
// significands a scale can have and each border). The same holds for amax / 6
// and the midpoints between scales.
// kUnit: scale_exp is 0.
template <bool kMx, bool kBf16, bool kUnit>
__global__ void __launch_bounds__(kThreads) k_quantize_fp4(const Fp4QuantArgs a) {
  constexpr int kBlock = kMx ? 32 : 16;
  constexpr int kWords = kBlock * (kBf16 ? 2 : 4) / 4;  // of a block's input
  // NV, bf16: 2^-scale_exp / s, rounded up, for each scale byte (0 for none)
  __shared__ float s_inv[128];
  if (!kMx && kBf16) {
    if (threadIdx.x < 128) {
      const float s = e4m3_to_float(threadIdx.x);
      s_inv[threadIdx.x] = s > 0.f ? __frcp_ru(s) * a.mul : 0.f;
    }
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
    // largest |x| as bits: NaN above infinity above every number
    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < kWords; ++v)
      top = kBf16 ? __vmaxu2(top, in[v] & 0x7FFF7FFFu) : max(top, in[v] & 0x7FFFFFFFu);
    if (kBf16) top = max(top << 16, top & 0xFFFF0000u);
    const float amax = __uint_as_float(top) * a.mul;
    const bool finite = __float_as_uint(amax) < 0x7F800000u;
    uint32_t sb;
    float s = 0.f, inv = 0.f;
    if (kMx) {
      // floor(log2 amax) - 2; subnormals: -127
      const int e = max(static_cast<int>(__float_as_uint(amax) >> 23) - 129, -127);
      sb = finite ? static_cast<uint32_t>(e + 127) : 0xFFu;
      inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    } else {
      const float sixth = kBf16 ? __fmul_rz(amax, 0x1.555556p-3f) : __fdiv_rn(amax, 6.0f);
      sb = finite ? __nv_cvt_float_to_fp8(sixth, __NV_SATFINITE, __NV_E4M3) : 0x7Fu;
      if (kBf16)
        inv = s_inv[sb & 127u];
      else
        s = e4m3_to_float(sb);
    }
    const bool coded = finite && (kMx || sb != 0);
    uint32_t words[kBlock / 8];
#pragma unroll
    for (int wd = 0; wd < kBlock / 8; ++wd) {
      float q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = 8 * wd + j;
        const float v = kBf16 ? __uint_as_float(k % 2 == 0 ? in[k / 2] << 16 : in[k / 2] & 0xFFFF0000u)
                              : __uint_as_float(in[k]);
        if (kMx)
          q[j] = kUnit ? v * inv : v * a.mul * inv;
        else if (kBf16)
          q[j] = __fmul_rz(v, inv);
        else
          q[j] = s > 0.f ? __fdiv_rn(kUnit ? v : v * a.mul, s) : 0.f;
      }
      words[wd] = coded ? e2m1_word(q) : 0u;
    }
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
