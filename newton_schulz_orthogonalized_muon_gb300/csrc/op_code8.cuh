// e4m3 codes and their power-of-two scales, as the operators that keep values
// in 8 bits share them.
#pragma once

#include <cuda_fp8.h>

#include "op_common.cuh"

namespace muon {

// The scale byte of a block whose largest magnitude has these fp32 bits (a
// finite a >= 0): e + 127 for the smallest e >= -111 with a 2^-e <= 448.
__device__ __forceinline__ int e4m3_scale_byte(int bits) {
  // a = m 2^k, 1 <= m < 2 (a below the normal range: k <= -127, clamped)
  const int k = (bits >> 23) - 127;
  const int e = (bits & 0x7FFFFF) <= 0x600000 ? k - 8 : k - 7;   // 448 = 1.75 * 2^8
  return max(e + 127, 16);
}

__device__ __forceinline__ uint32_t e4m3x4(const float* f) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0], f[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2], f[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// The four values of a word of codes, each times `unit`.
__device__ __forceinline__ void e4m3x4_values(uint32_t w, float unit, float* f) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * k)), __NV_E4M3));
    const float2 v = __half22float2(h);
    f[2 * k] = v.x * unit;
    f[2 * k + 1] = v.y * unit;
  }
}

}  // namespace muon
