// What the kernels that walk rows share: rows ahead of their use through shared
// memory, and launch shapes.
#pragma once

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "vec.cuh"

namespace moe {
namespace {

constexpr int kMaxVec = 4;                       // 8-column vectors per thread
constexpr int kMaxH = 1024 * 8 * kMaxVec;

// Eight elements as they lie in memory.
template <typename E>
struct Raw8 {
  static constexpr int W = sizeof(E) / 2;   // 16-byte pieces
  uint4 u[W];
  __device__ __forceinline__ void load(const E* p) {
#pragma unroll
    for (int i = 0; i < W; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void ones() {
    const uint32_t w = sizeof(E) == 4 ? 0x3f800000u : 0x3f803f80u;
#pragma unroll
    for (int i = 0; i < W; ++i) u[i] = make_uint4(w, w, w, w);
  }
  __device__ __forceinline__ float get(int j) const {
    const uint32_t* w = &u[0].x;
    if (sizeof(E) == 4) return __uint_as_float(w[j]);
    return j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
  }
  __device__ __forceinline__ float2 pair(int j) const { return make_float2(get(2 * j), get(2 * j + 1)); }
};

// Four sums over the warp at once: two exchanges leave each lane one of the four
// (lane & 3: x, z, y, w), three butterflies add it up, six shuffles in place of twenty.
__device__ __forceinline__ float warp_sum4(const float4& v) {
  const int lane = threadIdx.x & 31;
  const bool odd = lane & 1, high = lane & 2;
  float a = odd ? v.z : v.x, b = odd ? v.w : v.y;
  a += __shfl_xor_sync(0xffffffffu, odd ? v.x : v.z, 1);
  b += __shfl_xor_sync(0xffffffffu, odd ? v.y : v.w, 1);
  float s = high ? b : a;
  s += __shfl_xor_sync(0xffffffffu, high ? a : b, 2);
#pragma unroll
  for (int d = 4; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  return s;
}

// Four sums over the block of at most MAXT threads, the same in every thread, in a fixed
// order.  `part` holds 128 floats and may be reused after the next barrier.
template <int MAXT>
__device__ __forceinline__ float4 block_sum4(const float4& v, float* part) {
  float s = warp_sum4(v);
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (warps > 1) {
    if (lane < 4) part[(threadIdx.x >> 5) * 4 + lane] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int i = 0; i < (MAXT + 255) / 256; ++i) {
      const float p = part[i * 32 + lane];      // (past the warps: not one of the sums)
      s += i * 32 + lane < warps * 4 ? p : 0.f;
    }
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  }
  return make_float4(__shfl_sync(0xffffffffu, s, 0), __shfl_sync(0xffffffffu, s, 2),
                     __shfl_sync(0xffffffffu, s, 1), __shfl_sync(0xffffffffu, s, 3));
}

// The largest of three, NaN if one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 16 bytes to global memory where `on`, without a branch.
__device__ __forceinline__ void store16_if(void* p, const uint4& u, bool on) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t@p st.global.v4.b32 [%0], {%1, %2, %3, %4};\n\t}" ::"l"(p),
               "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w), "r"(static_cast<int>(on))
               : "memory");
}
__device__ __forceinline__ void store8_if(__nv_bfloat16* p, const float2 (&v)[4], bool on) {
  store16_if(p, make_uint4(pack_bf16(v[0].x, v[0].y), pack_bf16(v[1].x, v[1].y), pack_bf16(v[2].x, v[2].y),
                           pack_bf16(v[3].x, v[3].y)), on);
}
__device__ __forceinline__ void store8_if(float* p, const float2 (&v)[4], bool on) {
  const uint4* u = reinterpret_cast<const uint4*>(&v[0]);
  store16_if(p, u[0], on);
  store16_if(p + 4, u[1], on);
}

// Eight of a row's values as e4m3 codes with their block's scale byte, which four
// neighbouring threads (32 columns, inside or outside the row together) find by two
// shuffles: all lanes of the warp call it, with zeros where the columns do not exist
// (`in` is false).
__device__ __forceinline__ void store_e4m3(const float2 (&o)[4], bool in, uint8_t* codes, uint8_t* scale) {
  float top = max3_nan(fabsf(o[0].x), fabsf(o[0].y), 0.f);
#pragma unroll
  for (int j = 1; j < 4; ++j) top = max3_nan(top, fabsf(o[j].x), fabsf(o[j].y));
  uint32_t amax = __float_as_uint(top) & 0x7fffffffu;
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const uint32_t sb = mx_scale_byte(amax, 0x600000u, 8);
  const float inv = mx_inv_scale(sb);
  const float2 inv2 = make_float2(inv, inv);
  uint32_t h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) h[j] = __nv_cvt_float2_to_fp8x2(mul2(o[j], inv2), __NV_SATFINITE, __NV_E4M3);
  uint2 code = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  if (sb == 255u) code = make_uint2(0u, 0u);      // a block that is NaN
  if (!in) return;
  *reinterpret_cast<uint2*>(codes) = code;
  if ((threadIdx.x & 3) == 0) *scale = static_cast<uint8_t>(sb);
}

// Threads and vectors per thread for a row of H columns: one vector per thread
// up to 1024 threads.  (Two vectors share a row's sum, but the backward at
// 8192 x 2880 then takes 66 us instead of 41.)
struct RowShape {
  int threads, vecs;
};
RowShape row_shape(int H) {
  const int n = (H + 7) / 8;
  int v = 1;
  while (n > 1024 * v) v *= 2;
  return {((n + v - 1) / v + 31) / 32 * 32, v};
}

// Resident blocks per SM of the kernels that walk rows: as many as hold
// kThreadsPerSm threads of up to 64 registers and kRingPerSm of shared memory.
// (1536 threads of 40 registers: 88 us instead of 80 for the forward at 16384 x
// 4096, 61 instead of 41 for the backward at 8192 x 2880.)
constexpr int kThreadsPerSm = 1024;
constexpr int kRingPerSm = 210 * 1024;
constexpr int kAhead = 3;   // the ring's rows

// A launch of K<..., D> with the ring where it fits, or without.  The ring needs a
// few rows per block to pay: with no more rows than blocks, loads go at their use.
struct NormLaunch {
  int blocks, threads, smem;
  bool ring;
};
NormLaunch norm_launch(int64_t T, int threads, int ring_bytes, int threads_per_sm, int sms) {
  const int fit = ring_bytes <= kRingPerSm ? kRingPerSm / ring_bytes : 0;
  const int by_threads = std::max(1, std::min(8, threads_per_sm / threads));
  const int64_t most = static_cast<int64_t>(sms) * (fit ? std::min(fit, by_threads) : by_threads);
  NormLaunch l;
  l.ring = fit > 0 && T > most;
  l.blocks = static_cast<int>(std::min<int64_t>(T, most));
  l.threads = threads;
  l.smem = l.ring ? ring_bytes : 0;
  return l;
}

// More than 48 KB of dynamic shared memory has to be asked for, once per device.
template <typename K>
cudaError_t allow_smem(K kernel, std::atomic<uint64_t>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (ready.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingPerSm);
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// An upper bound on the blocks of a backward that needs no device.
constexpr int kMaxSms = 256;
constexpr int kMaxBwdBlocks = 8 * kMaxSms;

}  // namespace
}  // namespace moe
