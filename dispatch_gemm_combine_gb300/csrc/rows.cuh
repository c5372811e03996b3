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
  __device__ __forceinline__ float get(int j) const {
    const uint32_t* w = &u[0].x;
    if (sizeof(E) == 4) return __uint_as_float(w[j]);
    return j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
  }
  __device__ __forceinline__ float2 pair(int j) const { return make_float2(get(2 * j), get(2 * j + 1)); }
};

// The rows that a block walks, N arrays of them, D - 1 rows ahead of their use: each
// warp copies its own columns asynchronously into its own part of shared memory and
// reads them back itself, so no barrier of the block is needed.  A copy instruction
// covers 512 contiguous bytes (in fp32 a lane copies other pieces than it reads: with
// its own, 32 bytes apart, the backward at 8192 x 2880 takes 100 us instead of 74).
// D = 0: loads at their use.
template <typename E, int N, int V, int D>
struct RowRing {
  static constexpr int W = Raw8<E>::W;
  static constexpr int bytes(int threads) { return D * N * V * W * 16 * threads; }
  uint4* ring;
  const E* src[N];   // null: absent
  int H;
  // Piece p of the warp's 32 W in vector i of array n.
  __device__ __forceinline__ uint4* slot(int stage, int n, int i, int p) const {
    if (W == 1) return ring + ((stage * N + n) * V + i) * blockDim.x + threadIdx.x;
    return ring + ((stage * N + n) * V + i) * W * blockDim.x + (threadIdx.x & ~31u) * W + p;
  }
  __device__ __forceinline__ void issue(int stage, int64_t row, int64_t T) {
    if (D == 0) return;
    if (row < T) {
      const int lane = threadIdx.x & 31;
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int c0 = ((threadIdx.x & ~31u) + i * blockDim.x) * 8;   // the warp's first column
#pragma unroll
          for (int w = 0; w < W; ++w) {
            const int p = w * 32 + lane, c = W == 1 ? (threadIdx.x + i * blockDim.x) * 8 : c0 + p * (8 / W);
            if (src[n] && c < H) cp_async16(smem_u32(slot(stage, n, i, p)), src[n] + row * H + c, 16);
          }
        }
    }
    cp_async_commit();
  }
  // The oldest row's copies are there, and may be read.
  __device__ __forceinline__ void wait() const {
    cp_async_wait<D >= 2 ? D - 2 : 0>();
    if (W > 1) __syncwarp();
  }
  __device__ __forceinline__ void take(int stage, int n, int i, int64_t row, int c, Raw8<E>& r) const {
    if (D == 0) {
      r.load(src[n] + row * H + c);
      return;
    }
#pragma unroll
    for (int w = 0; w < W; ++w) r.u[w] = *slot(stage, n, i, (threadIdx.x & 31) * W + w);
  }
};

// Sums of K values over the block, the same in every thread, in a fixed order.
// `part` may be reused after the next barrier.
template <int K>
__device__ __forceinline__ void block_sums(float (&v)[3], float (*part)[32]) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  const int lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) part[k][threadIdx.x >> 5] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(lane < warps ? part[k][lane] : 0.f);
}

// Eight of a row's values as e4m3 codes with their block's scale byte, which four
// neighbouring threads (32 columns, inside or outside the row together) find by two
// shuffles: all lanes of the warp call it, `in` where the columns exist.
__device__ __forceinline__ void store_e4m3(const float (&o)[8], bool in, uint8_t* codes, uint8_t* scale) {
  uint32_t amax = 0;
  if (in) {
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(o[j]) & 0x7fffffffu);
  }
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  if (!in) return;
  const uint32_t sb = mx_scale_byte(amax, 0x600000u, 8);
  const float inv = mx_inv_scale(sb);
  uint2 code;
  uint32_t h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float2 p = make_float2(o[2 * j] * inv, o[2 * j + 1] * inv);
    if (sb == 255u) p = make_float2(0.f, 0.f);
    h[j] = __nv_cvt_float2_to_fp8x2(p, __NV_SATFINITE, __NV_E4M3);
  }
  code.x = h[0] | (h[1] << 16);
  code.y = h[2] | (h[3] << 16);
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
