// Device helpers of the microscaled 4-bit formats.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace clover {

// offsets[g] kept inside [0, n_rows], whatever the array holds.
__device__ __forceinline__ int group_offset(const int32_t* offsets, int g, int n_rows) {
  const int v = offsets[g];
  return v < 0 ? 0 : (v > n_rows ? n_rows : v);
}

// The last of n <= 1024 ascending values that is at most v, by a whole warp:
// among every per-th, then among the per from there. value(0) <= v.
template <typename F>
__device__ __forceinline__ int warp_search(int n, int v, F value) {
  const int lane = threadIdx.x & 31, per = (n + 31) / 32;
  const int a = lane * per;
  // (bit 0 stands even where the values do not ascend)
  const int lo = (31 - __clz(__ballot_sync(0xffffffffu, a < n && value(a) <= v) | 1u)) * per;
  const int b = lo + lane;
  return lo + 31 - __clz(__ballot_sync(0xffffffffu, lane < per && b < n && value(b) <= v) | 1u);
}

__device__ __forceinline__ float e4m3_to_float(uint32_t byte) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3)));
}

__device__ __forceinline__ float e8m0_to_float(uint32_t byte) {
  // 2^(byte - 127): byte 0 is the subnormal 2^-127, byte 255 NaN
  return __uint_as_float(byte == 0 ? 0x00400000u : (byte == 255 ? 0x7FC00000u : byte << 23));
}

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

// 2^-scale_exp / s, rounded up, of an e4m3 scale byte below 128 (0 for none):
// the factor by which quantize_block takes bf16 values to NV codes.
__device__ __forceinline__ float scale_inverse(uint32_t byte, float mul) {
  const float s = e4m3_to_float(byte);
  return s > 0.f ? __frcp_ru(s) * mul : 0.f;
}

// The codes (eight to a word) of one block of values and, returned, its scale
// byte. in: the block's bf16 or fp32 bits. mul: 2^-scale_exp (kUnit: 1). inv_of:
// scale_inverse of each byte (NV with bf16 values only).
//
// The codes are exact. MX: y / s is exact (s a power of two). NV with fp32
// input: the correctly rounded quotient lies on the same side of every border
// (or on it) as the exact one, as border * s has 7 significant bits. NV with
// bf16 input: a quotient that is not on a border is at least 2^-9 of it away,
// far more than x * (1 / s) is off; on a border, with 1 / s rounded up and the
// product cut off, the product is the border itself (for each of the 8
// significands a scale can have and each border). The same holds for amax / 6
// and the midpoints between scales.
template <bool kMx, bool kBf16, bool kUnit>
__device__ __forceinline__ uint32_t quantize_block(const uint32_t (&in)[(kMx ? 32 : 16) * (kBf16 ? 2 : 4) / 4], float mul,
                                                   const float* inv_of, uint32_t (&words)[(kMx ? 32 : 16) / 8]) {
  constexpr int kBlock = kMx ? 32 : 16;
  constexpr int kWords = kBlock * (kBf16 ? 2 : 4) / 4;
  // largest |x| as bits: NaN above infinity above every number
  uint32_t top = 0;
#pragma unroll
  for (int v = 0; v < kWords; ++v)
    top = kBf16 ? __vmaxu2(top, in[v] & 0x7FFF7FFFu) : max(top, in[v] & 0x7FFFFFFFu);
  if (kBf16) top = max(top << 16, top & 0xFFFF0000u);
  const float amax = __uint_as_float(top) * mul;
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
      inv = inv_of[sb & 127u];
    else
      s = e4m3_to_float(sb);
  }
  const bool coded = finite && (kMx || sb != 0);
#pragma unroll
  for (int wd = 0; wd < kBlock / 8; ++wd) {
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = 8 * wd + j;
      const float v = kBf16 ? __uint_as_float(k % 2 == 0 ? in[k / 2] << 16 : in[k / 2] & 0xFFFF0000u)
                            : __uint_as_float(in[k]);
      if (kMx)
        q[j] = kUnit ? v * inv : v * mul * inv;
      else if (kBf16)
        q[j] = __fmul_rz(v, inv);
      else
        q[j] = s > 0.f ? __fdiv_rn(kUnit ? v : v * mul, s) : 0.f;
    }
    words[wd] = coded ? e2m1_word(q) : 0u;
  }
  return sb;
}

// Four pairs of values of eight codes (one instruction each, whichever byte).
__device__ __forceinline__ void expand_word(uint32_t w, __half2 (&h)[4]) {
  uint32_t r[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = *reinterpret_cast<const __half2*>(&r[i]);
}

// The two scale bytes of a halfword in fp16.
__device__ __forceinline__ __half2 scales2(uint32_t bytes) {
  uint32_t r;
  asm("{\n\t.reg .b16 x;\n\tcvt.u16.u32 x, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}" : "=r"(r) : "r"(bytes));
  return *reinterpret_cast<const __half2*>(&r);
}

__device__ __forceinline__ uint32_t half2_word(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

}  // namespace clover
