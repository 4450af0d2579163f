// Device helpers of the microscaled 4-bit formats.
#pragma once

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

}  // namespace clover
