// e2m1 codes (sign, two exponent bits, one fraction bit: 0, 0.5, 1, 1.5, 2, 3,
// 4, 6) to and from fp32, two per byte, the lower one first.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <stdint.h>

namespace moe {

// Rounded to nearest, ties to even.
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
  return __nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest);
}

__device__ __forceinline__ float2 e2m1_values(uint32_t byte) {
  const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(byte), __NV_E2M1);
  return __half22float2(__half2(h));
}

}  // namespace moe
