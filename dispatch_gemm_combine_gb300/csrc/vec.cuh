// Vectors of eight consecutive elements (bf16: one 16-byte access, fp32: two)
// as fp32 values, reductions over a block, and the power-of-two scale of a
// microscaled block: shared by the memory-bound operators.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
  v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
}
__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
  uint4 u;
  u.x = pack_bf16(v[0], v[1]), u.y = pack_bf16(v[2], v[3]);
  u.z = pack_bf16(v[4], v[5]), u.w = pack_bf16(v[6], v[7]);
  *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// Two fp32 products or fused products and sums in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// Sum over the block, the same value in every thread; the order of the sum is
// fixed by the block's size.  `part` holds 32 floats and may be reused after
// the next barrier.
__device__ __forceinline__ float block_sum(float v, float* part) {
  v = warp_sum(v);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < warps ? part[lane] : 0.f);
}

// Microscaled blocks: 32 values share the scale 2^q, the smallest power of two
// with amax <= top * 2^q (top: the largest value of the code), so nothing is
// clipped.  With amax = m * 2^x, 1 <= m < 2, and top = mt * 2^xt, q = x - xt,
// plus one where m > mt; both are read off the bits of amax.  q is kept in
// [-127, 127]; the scale byte is q + 127, and 255 stands for NaN: a block that
// holds an infinity or a NaN reads as NaN throughout.
//   top_mant, top_exp: the fraction bits and the exponent of `top`
//   e4m3: 448 = 1.75 * 2^8;  e2m1: 6 = 1.5 * 2^2
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits, uint32_t top_mant,
                                                  int top_exp) {
  if (amax_bits >= 0x7f800000u) return 255u;
  const int b = static_cast<int>(amax_bits >> 23) - top_exp +
                ((amax_bits & 0x7fffffu) > top_mant ? 1 : 0);
  return static_cast<uint32_t>(max(0, min(254, b)));
}

// 2^-q of a scale byte: an exact factor (2^-127 is a subnormal).  The byte 255
// gives 0, so that the codes of a NaN block are not undefined.
__device__ __forceinline__ float mx_inv_scale(uint32_t byte) {
  if (byte == 255u) return 0.f;
  return byte == 254u ? __uint_as_float(0x00400000u) : __uint_as_float((254u - byte) << 23);
}

// 2^q of a scale byte.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return byte == 0u ? __uint_as_float(0x00400000u)
                    : (byte == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23));
}

}  // namespace moe
