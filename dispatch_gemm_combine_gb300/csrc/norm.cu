// RMS norm with the residual's addition, the step that makes the expert
// layer's input, and its gradient.
//
//   r = x + residual,  rstd = (mean_h r^2 + eps)^-1/2,  y = r * rstd * weight
//
// Forward: a block walks rows (or has one), each thread holds 8 * V columns of r in
// registers, so x and the residual are read once and the outputs written once:
// HBM-bound.  Later rows' loads are in flight while a row is summed (RowRing).  r^2
// is summed in fp32 (eight values per thread, then a warp butterfly, then the warps).
// r itself is not rounded before the norm; `total` is r rounded once to the storage
// type.  The 8-bit output takes the block's scale from four neighbouring threads (32
// columns) by two shuffles.
//
// Backward, with xhat = r * rstd and n = dy * weight:
//   dx = rstd * (n - xhat * mean_h(n * xhat)) + d_total,
//   dweight[h] = sum_t dy * xhat.
// A block walks rows t = block, block + grid, ...; each thread owns the same
// columns in every row and keeps their dweight sums in registers, so dy and r
// are read once.  The blocks' sums go to the workspace and a second kernel adds
// them in block order: no atomics, the same bits every time.
//
// Measured: 16384 x 4096 bf16 with residual and 8-bit output 78 us, 6.1 TB/s;
// backward of 8192 x 2880 37 us, 5.1 TB/s, bound by instructions (60% of the issue
// slots), a barrier per row and the wait for its copies.
#include <algorithm>
#include <atomic>

#include "abi_internal.h"
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

template <typename E, bool OUT8, int V, int D>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(
    const E* __restrict__ x, const E* __restrict__ residual, const E* __restrict__ weight, int64_t T,
    int H, float eps, void* __restrict__ y, uint8_t* __restrict__ y_scale, E* __restrict__ total,
    float* __restrict__ rstd_out) {
  extern __shared__ uint4 ring_mem[];
  __shared__ float part[2][32];
  RowRing<E, 2, V, D> rows{ring_mem, {x, residual}, H};
#pragma unroll
  for (int d = 0; d < D - 1; ++d) rows.issue(d, blockIdx.x + static_cast<int64_t>(d) * gridDim.x, T);
  // the weight ahead, where registers allow
  constexpr bool KEEP = V < 4;
  Raw8<E> w[KEEP ? V : 1];
  if (KEEP)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c < H) w[i % (KEEP ? V : 1)].load(weight + c);
    }
  int stage = 0, flip = 0;   // a row's barrier also separates the reuse of the other sums
  for (int64_t row = blockIdx.x; row < T; row += gridDim.x, flip ^= 1) {
    const int64_t base = row * H;
    if (D > 0) {
      rows.wait();
      rows.issue(stage == 0 ? D - 1 : stage - 1, row + static_cast<int64_t>(D - 1) * gridDim.x, T);
    }
    float r[V][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c < H) {
        Raw8<E> a, b;
        rows.take(stage, 0, i, row, c, a);
        if (residual) rows.take(stage, 1, i, row, c, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          r[i][j] = residual ? a.get(j) + b.get(j) : a.get(j);
          ss = fmaf(r[i][j], r[i][j], ss);
        }
        if (total) store8(total + base + c, r[i]);
      }
    }
    if (D > 0) stage = stage + 1 == D ? 0 : stage + 1;
    ss = block_sum(ss, part[flip]);
    const float rstd = 1.f / sqrtf(ss / static_cast<float>(H) + eps);
    if (rstd_out && threadIdx.x == 0) rstd_out[row] = rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (!OUT8 && c >= H) continue;
      float o[8];
      if (c < H) {
        Raw8<E>& wi = w[i % (KEEP ? V : 1)];
        if (!KEEP) wi.load(weight + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = r[i][j] * rstd * wi.get(j);
      }
      if (!OUT8) {
        store8(static_cast<E*>(y) + base + c, o);
      } else {
        // the four threads of a block of 32 columns are inside or outside the row
        // together (H is a multiple of 32); all lanes take part in the shuffles
        uint32_t amax = 0;
        if (c < H) {
#pragma unroll
          for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(o[j]) & 0x7fffffffu);
        }
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        if (c < H) {
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
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(y) + base + c) = code;
          if ((threadIdx.x & 3) == 0) y_scale[row * (H / 32) + c / 32] = static_cast<uint8_t>(sb);
        }
      }
    }
  }
}

template <typename E, int V, int D>
__global__ void __launch_bounds__(1024) norm_bwd_kernel(
    const E* __restrict__ dy, const E* __restrict__ d_total, const E* __restrict__ total,
    const float* __restrict__ rstd_in, const E* __restrict__ weight, int64_t T, int H,
    E* __restrict__ dx, float* __restrict__ dw_part) {
  extern __shared__ uint4 ring_mem[];
  __shared__ float part[2][32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  RowRing<E, 3, V, D> rows{ring_mem, {dy, total, d_total}, H};
#pragma unroll
  for (int d = 0; d < D - 1; ++d) rows.issue(d, blockIdx.x + static_cast<int64_t>(d) * gridDim.x, T);
  constexpr bool KEEP = V < 4;   // the weight in registers
  // n and xhat stay in fp32 between the two passes over a row where registers allow
  constexpr bool HOLD = V == 1;
  float2 dw[V][4], n[4], xh[4];
  Raw8<E> w[KEEP ? V : 1], g[V], r[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8;
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[i][j] = make_float2(0.f, 0.f);
    if (KEEP && c < H) w[i % (KEEP ? V : 1)].load(weight + c);
  }
  int stage = 0, flip = 0;   // a row's barrier also separates the reuse of the other sums
  // rstd of 32 rows, one per lane: a load per row may share its scoreboard with the
  // rows' copies and then waits for them too (8192 x 2880: 47 us instead of 39)
  const int lane = threadIdx.x & 31;
  const float inv_H = 1.f / static_cast<float>(H);
  float rstds = 0.f;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < T; row += gridDim.x, flip ^= 1) {
    const int64_t base = row * H;
    if ((turn & 31) == 0) {
      const int64_t mine = row + static_cast<int64_t>(lane) * gridDim.x;
      rstds = mine < T ? __ldg(rstd_in + mine) : 0.f;
    }
    const float rstd = __shfl_sync(0xffffffffu, rstds, turn++ & 31);
    if (D > 0) {
      rows.wait();
      rows.issue(stage == 0 ? D - 1 : stage - 1, row + static_cast<int64_t>(D - 1) * gridDim.x, T);
    }
    float2 dot2 = make_float2(0.f, 0.f);
    const float2 rstd2 = make_float2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c < H) {
        rows.take(stage, 0, i, row, c, g[i]);
        rows.take(stage, 1, i, row, c, r[i]);
        Raw8<E>& wi = w[i % (KEEP ? V : 1)];
        if (!KEEP) wi.load(weight + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 gj = g[i].pair(j);
          n[j] = mul2(gj, wi.pair(j));
          xh[j] = mul2(r[i].pair(j), rstd2);
          dw[i][j] = fma2(gj, xh[j], dw[i][j]);
          dot2 = fma2(n[j], xh[j], dot2);
        }
      }
    }
    const float mean = block_sum(dot2.x + dot2.y, part[flip]) * inv_H;
    const float2 mean2 = make_float2(-mean, -mean);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c < H) {
        float o[8];
        Raw8<E>& wi = w[i % (KEEP ? V : 1)];
        if (!KEEP) wi.load(weight + c);
        Raw8<E> e;
        if (d_total) rows.take(stage, 2, i, row, c, e);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 nj = HOLD ? n[j] : mul2(g[i].pair(j), wi.pair(j));
          const float2 d = fma2(HOLD ? xh[j] : mul2(r[i].pair(j), rstd2), mean2, nj);
          const float2 v = d_total ? fma2(rstd2, d, e.pair(j)) : mul2(rstd2, d);
          o[2 * j] = v.x, o[2 * j + 1] = v.y;
        }
        store8(dx + base + c, o);
      }
    }
    if (D > 0) stage = stage + 1 == D ? 0 : stage + 1;
  }
  if (dw_part) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c < H) store8(dw_part + static_cast<int64_t>(blockIdx.x) * H + c, &dw[i][0].x);
    }
  }
}

// dweight[c] = sum of the blocks' partial sums: 32 columns by 32 groups of
// blocks per thread block, each group in block order, then the groups in order.
__global__ void __launch_bounds__(1024) norm_dweight_kernel(const float* __restrict__ part,
                                                            int blocks, int H,
                                                            float* __restrict__ dweight) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.f;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the sums are there
  if (c < H)
#pragma unroll 8
    for (int b = grp; b < blocks; b += 32) a += __ldcg(part + static_cast<int64_t>(b) * H + c);
  s[grp][lane] = a;
  __syncthreads();
  const float v = warp_sum(s[lane][grp]);
  if (lane == 0 && blockIdx.x * 32 + grp < H) dweight[blockIdx.x * 32 + grp] = v;
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

template <typename E, bool OUT8, int V>
cudaError_t launch_fwd_v(const E* x, const E* residual, const E* weight, int64_t T, int H, float eps,
                         void* y, uint8_t* y_scale, E* total, float* rstd, int threads, int sms,
                         cudaStream_t st) {
  const NormLaunch l = norm_launch(T, threads, RowRing<E, 2, V, kAhead>::bytes(threads), kThreadsPerSm, sms);
  // Without the 8-bit output there is little to compute, and where several rows fit an
  // SM a block for each is the faster form: 16384 x 4096 bf16 84 us instead of 94,
  // 32768 x 1024 43 and 50, 8192 x 4096 fp32 82 and 96.  (8192 x 7168 bf16: 83 and 81;
  // with 8-bit output 16384 x 4096 takes 123 and 80.)
  if (l.ring && (OUT8 || threads > 512)) {
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(norm_fwd_kernel<E, OUT8, V, kAhead>, ready);
    if (e != cudaSuccess) return e;
    norm_fwd_kernel<E, OUT8, V, kAhead><<<l.blocks, l.threads, l.smem, st>>>(x, residual, weight, T, H, eps, y, y_scale, total, rstd);
  } else {
    norm_fwd_kernel<E, OUT8, V, 0><<<static_cast<unsigned>(T), l.threads, 0, st>>>(x, residual, weight, T, H, eps, y, y_scale, total, rstd);
  }
  return cudaGetLastError();
}

template <typename E, bool OUT8>
cudaError_t launch_fwd(const E* x, const E* residual, const E* weight, int64_t T, int H, float eps,
                       void* y, uint8_t* y_scale, E* total, float* rstd, int sms, cudaStream_t st) {
  RowShape s = row_shape(H);
  // bf16 with 8-bit output: of 513 to 1023 threads one block fits an SM, so two
  // vectors per thread (8192 x 5120 53 us instead of 59, 8192 x 7168 70 and 72; the
  // other outputs lose: 8192 x 5120 65 and 56).
  if (OUT8 && sizeof(E) == 2 && s.threads > 512 && s.threads < 1024)
    s = {((H + 15) / 16 + 31) / 32 * 32, 2};
  if (s.vecs == 1) return launch_fwd_v<E, OUT8, 1>(x, residual, weight, T, H, eps, y, y_scale, total, rstd, s.threads, sms, st);
  if (s.vecs == 2) return launch_fwd_v<E, OUT8, 2>(x, residual, weight, T, H, eps, y, y_scale, total, rstd, s.threads, sms, st);
  return launch_fwd_v<E, OUT8, 4>(x, residual, weight, T, H, eps, y, y_scale, total, rstd, s.threads, sms, st);
}

template <typename E, int V>
cudaError_t launch_bwd_v(const E* dy, const E* d_total, const E* total, const float* rstd, const E* weight,
                         int64_t T, int H, E* dx, float* part, int threads, int sms, int* blocks,
                         cudaStream_t st) {
  const NormLaunch l = norm_launch(T, threads, RowRing<E, 3, V, kAhead>::bytes(threads), kThreadsPerSm, sms);
  *blocks = l.blocks;
  if (l.ring) {
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(norm_bwd_kernel<E, V, kAhead>, ready);
    if (e != cudaSuccess) return e;
    norm_bwd_kernel<E, V, kAhead><<<l.blocks, l.threads, l.smem, st>>>(dy, d_total, total, rstd, weight, T, H, dx, part);
  } else {
    norm_bwd_kernel<E, V, 0><<<l.blocks, l.threads, 0, st>>>(dy, d_total, total, rstd, weight, T, H, dx, part);
  }
  return cudaGetLastError();
}

// *blocks: of the launch, each of which leaves its sums in `part`.
template <typename E>
cudaError_t launch_bwd(const E* dy, const E* d_total, const E* total, const float* rstd,
                       const E* weight, int64_t T, int H, E* dx, float* part, int sms, int* blocks,
                       cudaStream_t st) {
  const RowShape s = row_shape(H);
  if (s.vecs == 1) return launch_bwd_v<E, 1>(dy, d_total, total, rstd, weight, T, H, dx, part, s.threads, sms, blocks, st);
  if (s.vecs == 2) return launch_bwd_v<E, 2>(dy, d_total, total, rstd, weight, T, H, dx, part, s.threads, sms, blocks, st);
  return launch_bwd_v<E, 4>(dy, d_total, total, rstd, weight, T, H, dx, part, s.threads, sms, blocks, st);
}

// An upper bound on the backward's blocks that needs no device.
constexpr int kMaxSms = 256;
constexpr int kMaxBwdBlocks = 8 * kMaxSms;

bool norm_dims_ok(int64_t T, int32_t H, int32_t dtype) {
  return T >= 0 && T < (1ll << 31) && H >= 8 && H % 8 == 0 && H <= kMaxH &&
         (dtype == MOE_BF16 || dtype == MOE_FP32);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_rms_norm_fwd(int64_t T, int32_t H, int32_t dtype, const void* x,
                            const void* residual, const void* weight, float eps, void* y,
                            uint8_t* y_scale, void* total, float* rstd, moe_stream_t stream) {
  if (!norm_dims_ok(T, H, dtype) || !(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if (y_scale && H % 32) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !weight || !y) return MOE_ERR_INVALID_ARG;
  for (const void* p : {x, residual, weight, static_cast<const void*>(y),
                        static_cast<const void*>(total)})
    if (!abi_aligned16(p)) return MOE_ERR_INVALID_ARG;
  int sms = 0;
  const moe_status ds = abi_device_sms(&sms);
  if (ds != MOE_OK) return ds;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = abi_tracked(kAbiNormFwd, 1, st, [&] {
    auto go = [&](auto* xt) {
      using E = std::remove_const_t<std::remove_pointer_t<decltype(xt)>>;
      auto* rt = static_cast<const E*>(residual);
      auto* wt = static_cast<const E*>(weight);
      auto* tt = static_cast<E*>(total);
      return y_scale ? launch_fwd<E, true>(xt, rt, wt, T, H, eps, y, y_scale, tt, rstd, sms, st)
                     : launch_fwd<E, false>(xt, rt, wt, T, H, eps, y, y_scale, tt, rstd, sms, st);
    };
    return dtype == MOE_FP32 ? go(static_cast<const float*>(x))
                             : go(static_cast<const __nv_bfloat16*>(x));
  });
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_rms_norm_workspace_size(int64_t T, int32_t H) {
  if (!norm_dims_ok(T, H, MOE_BF16)) return 0;
  return 256 + abi_align256(sizeof(float) * static_cast<size_t>(H) *
                            static_cast<size_t>(std::max<int64_t>(1, std::min<int64_t>(T, kMaxBwdBlocks))));
}

moe_status moe_rms_norm_bwd(int64_t T, int32_t H, int32_t dtype, const void* dy,
                            const void* d_total, const void* total, const float* rstd,
                            const void* weight, void* dx, float* dweight, void* ws,
                            size_t ws_bytes, moe_stream_t stream) {
  if (!norm_dims_ok(T, H, dtype)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!dy || !total || !rstd || !weight || !dx)) return MOE_ERR_INVALID_ARG;
  for (const void* p : {dy, d_total, total, weight, static_cast<const void*>(dx),
                        static_cast<const void*>(dweight)})
    if (!abi_aligned16(p)) return MOE_ERR_INVALID_ARG;
  if (dweight && T > 0) {
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < moe_rms_norm_workspace_size(T, H)) return MOE_ERR_WORKSPACE;
  }
  int sms = 0;
  const moe_status ds = abi_device_sms(&sms);
  if (ds != MOE_OK) return ds;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (dweight && abi_tracked_memset(dweight, 0, sizeof(float) * H, st) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  int blocks = 0;
  float* part = dweight ? reinterpret_cast<float*>(static_cast<char*>(ws) + 256) : nullptr;
  const cudaError_t e = abi_tracked(kAbiNormBwd, dweight ? 2 : 1, st, [&] {
    auto go = [&](auto* gt) {
      using E = std::remove_const_t<std::remove_pointer_t<decltype(gt)>>;
      return launch_bwd<E>(gt, static_cast<const E*>(d_total), static_cast<const E*>(total), rstd,
                           static_cast<const E*>(weight), T, H, static_cast<E*>(dx), part,
                           std::min(sms, kMaxSms), &blocks, st);
    };
    cudaError_t r = dtype == MOE_FP32 ? go(static_cast<const float*>(dy))
                                      : go(static_cast<const __nv_bfloat16*>(dy));
    if (r == cudaSuccess && dweight) {
      // (may start while the last rows are done)
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((H + 31) / 32);
      cfg.blockDim = dim3(1024);
      cfg.stream = st;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      r = cudaLaunchKernelEx(&cfg, norm_dweight_kernel, static_cast<const float*>(part), blocks, H, dweight);
    }
    return r;
  });
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
