// RMS norm with the residual's addition, the step that makes the expert
// layer's input, and its gradient.
//
//   r = x + residual,  rstd = (mean_h r^2 + eps)^-1/2,  y = r * rstd * weight
//
// Forward: one block per row, each thread holds 8 * V consecutive columns of r
// in registers, so x and the residual are read once and the outputs written
// once: HBM-bound.  r^2 is summed in fp32 (eight values per thread, then a
// warp butterfly, then the warps).  r itself is not rounded before the norm;
// `total` is r rounded once to the storage type.  The 8-bit output takes the
// block's scale from four neighbouring threads (32 columns) by two shuffles.
//
// Backward, with xhat = r * rstd and n = dy * weight:
//   dx = rstd * (n - xhat * mean_h(n * xhat)) + d_total,
//   dweight[h] = sum_t dy * xhat.
// A block walks rows t = block, block + grid, ...; each thread owns the same
// columns in every row and keeps their dweight sums in registers, so dy and r
// are read once.  The blocks' sums go to the workspace and a second kernel adds
// them in block order: no atomics, the same bits every time.
#include <algorithm>

#include "abi_internal.h"
#include "vec.cuh"

namespace moe {
namespace {

constexpr int kMaxVec = 4;                       // 8-column vectors per thread
constexpr int kMaxH = 1024 * 8 * kMaxVec;
constexpr int kBwdThreadsPerSm = 1024;

template <typename E, bool OUT8, int V>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(
    const E* __restrict__ x, const E* __restrict__ residual, const E* __restrict__ weight, int H,
    float eps, void* __restrict__ y, uint8_t* __restrict__ y_scale, E* __restrict__ total,
    float* __restrict__ rstd_out) {
  __shared__ float part[32];
  const int64_t row = blockIdx.x;
  const int64_t base = row * H;
  float r[V][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8;
    if (c < H) load8(x + base + c, r[i]);
  }
  if (residual) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c < H) {
        float b[8];
        load8(residual + base + c, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] += b[j];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8;
    if (c < H) {
      if (total) store8(total + base + c, r[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(r[i][j], r[i][j], ss);
    }
  }
  // the weight before the barrier, where registers allow: one latency less
  constexpr bool EARLY = V < 4;
  float w[EARLY ? V : 1][8];
  if (EARLY)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c < H) load8(weight + c, w[i % (EARLY ? V : 1)]);
    }
  ss = block_sum(ss, part);
  const float rstd = 1.f / sqrtf(ss / static_cast<float>(H) + eps);
  if (rstd_out && threadIdx.x == 0) rstd_out[row] = rstd;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8;
    if (!OUT8 && c >= H) continue;
    float o[8];
    if (c < H) {
      float* wi = w[i % (EARLY ? V : 1)];
      if (!EARLY) load8(weight + c, wi);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = r[i][j] * rstd * wi[j];
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

// Eight elements as they lie in memory.
template <typename E>
struct Raw8 {
  uint4 u[sizeof(E) / 2];
  __device__ __forceinline__ void load(const E* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(E) / 2); ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ float get(int j) const {
    const uint32_t* w = &u[0].x;
    if (sizeof(E) == 4) return __uint_as_float(w[j]);
    return j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
  }
};

// The next row's loads are issued before the current row's sum (AHEAD; not where a
// thread has so many columns that the registers would not hold them).
template <typename E, int V, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_bwd_kernel(
    const E* __restrict__ dy, const E* __restrict__ d_total, const E* __restrict__ total,
    const float* __restrict__ rstd_in, const E* __restrict__ weight, int64_t T, int H,
    E* __restrict__ dx, float* __restrict__ dw_part) {
  constexpr bool AHEAD = V * sizeof(E) <= (THREADS <= 512 ? 4 : 2);
  __shared__ float part[2][32];
  float dw[V][8];
  constexpr bool KEEP = V < 4;   // the weight in registers
  Raw8<E> w[KEEP ? V : 1], g[V], r[V], e[V], g1[AHEAD ? V : 1], r1[AHEAD ? V : 1], e1[AHEAD ? V : 1];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    if (KEEP && c < H) w[i % (KEEP ? V : 1)].load(weight + c);
  }
  auto load = [&](int64_t row, Raw8<E>* gd, Raw8<E>* rd, Raw8<E>* ed) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c < H) {
        gd[i].load(dy + row * H + c);
        rd[i].load(total + row * H + c);
        if (d_total) ed[i].load(d_total + row * H + c);
      }
    }
  };
  int flip = 0;   // a row's barrier also separates the reuse of the other buffer
  float rstd1 = 0.f;
  if (AHEAD) {
    load(blockIdx.x, g1, r1, e1);
    rstd1 = __ldg(rstd_in + blockIdx.x);
  }
  for (int64_t row = blockIdx.x; row < T; row += gridDim.x, flip ^= 1) {
    const int64_t base = row * H;
    float rstd;
    if (AHEAD) {
#pragma unroll
      for (int i = 0; i < V; ++i) g[i] = g1[i % (AHEAD ? V : 1)], r[i] = r1[i % (AHEAD ? V : 1)], e[i] = e1[i % (AHEAD ? V : 1)];
      rstd = rstd1;
      const int64_t next = row + gridDim.x;
      if (next < T) {
        load(next, g1, r1, e1);
        rstd1 = __ldg(rstd_in + next);
      }
    } else {
      load(row, g, r, e);
      rstd = __ldg(rstd_in + row);
    }
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c < H) {
        Raw8<E>& wi = w[i % (KEEP ? V : 1)];
        if (!KEEP) wi.load(weight + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float gj = g[i].get(j), xh = r[i].get(j) * rstd;
          dw[i][j] = fmaf(gj, xh, dw[i][j]);
          dot = fmaf(gj * wi.get(j), xh, dot);
        }
      }
    }
    const float mean = block_sum(dot, part[flip]) / static_cast<float>(H);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c < H) {
        float o[8];
        Raw8<E>& wi = w[i % (KEEP ? V : 1)];
        if (!KEEP) wi.load(weight + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[j] = rstd * (g[i].get(j) * wi.get(j) - r[i].get(j) * rstd * mean);
          if (d_total) o[j] += e[i].get(j);
        }
        store8(dx + base + c, o);
      }
    }
  }
  if (dw_part) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c < H) store8(dw_part + static_cast<int64_t>(blockIdx.x) * H + c, dw[i]);
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
  if (c < H)
    for (int b = grp; b < blocks; b += 32) a += part[static_cast<int64_t>(b) * H + c];
  s[grp][lane] = a;
  __syncthreads();
  const float v = warp_sum(s[lane][grp]);
  if (lane == 0 && blockIdx.x * 32 + grp < H) dweight[blockIdx.x * 32 + grp] = v;
}

// Threads and vectors per thread for a row of H columns: one vector per thread
// up to 1024 threads.
struct RowShape {
  int threads, vecs;
};
RowShape row_shape(int H) {
  const int n = (H + 7) / 8;
  int v = 1;
  while (n > 1024 * v) v *= 2;
  return {((n + v - 1) / v + 31) / 32 * 32, v};
}

// As many blocks as stay resident: a block's sums are written and read once more.
int bwd_blocks(int64_t T, int H, int sms) {
  const int per_sm = std::max(1, std::min(8, kBwdThreadsPerSm / row_shape(H).threads));
  return static_cast<int>(std::min<int64_t>(T, static_cast<int64_t>(sms) * per_sm));
}

template <typename E, bool OUT8>
cudaError_t launch_fwd(const E* x, const E* residual, const E* weight, int64_t T, int H, float eps,
                       void* y, uint8_t* y_scale, E* total, float* rstd, cudaStream_t st) {
  const RowShape s = row_shape(H);
  const unsigned grid = static_cast<unsigned>(T);
  if (s.vecs == 1)
    norm_fwd_kernel<E, OUT8, 1><<<grid, s.threads, 0, st>>>(x, residual, weight, H, eps, y, y_scale, total, rstd);
  else if (s.vecs == 2)
    norm_fwd_kernel<E, OUT8, 2><<<grid, s.threads, 0, st>>>(x, residual, weight, H, eps, y, y_scale, total, rstd);
  else
    norm_fwd_kernel<E, OUT8, 4><<<grid, s.threads, 0, st>>>(x, residual, weight, H, eps, y, y_scale, total, rstd);
  return cudaGetLastError();
}

template <typename E>
cudaError_t launch_bwd(const E* dy, const E* d_total, const E* total, const float* rstd,
                       const E* weight, int64_t T, int H, E* dx, float* part, int blocks,
                       cudaStream_t st) {
  const RowShape s = row_shape(H);
  if (s.threads <= 512)   // then one vector each
    norm_bwd_kernel<E, 1, 512><<<blocks, s.threads, 0, st>>>(dy, d_total, total, rstd, weight, T, H, dx, part);
  else if (s.vecs == 1)
    norm_bwd_kernel<E, 1, 1024><<<blocks, s.threads, 0, st>>>(dy, d_total, total, rstd, weight, T, H, dx, part);
  else if (s.vecs == 2)
    norm_bwd_kernel<E, 2, 1024><<<blocks, s.threads, 0, st>>>(dy, d_total, total, rstd, weight, T, H, dx, part);
  else
    norm_bwd_kernel<E, 4, 1024><<<blocks, s.threads, 0, st>>>(dy, d_total, total, rstd, weight, T, H, dx, part);
  return cudaGetLastError();
}

// More blocks than a device has SMs for: an upper bound that needs no device.
constexpr int kMaxBwdBlocks = 8 * 256;

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
      return y_scale ? launch_fwd<E, true>(xt, rt, wt, T, H, eps, y, y_scale, tt, rstd, st)
                     : launch_fwd<E, false>(xt, rt, wt, T, H, eps, y, y_scale, tt, rstd, st);
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
  const int blocks = std::min(kMaxBwdBlocks, bwd_blocks(T, H, sms));
  float* part = dweight ? reinterpret_cast<float*>(static_cast<char*>(ws) + 256) : nullptr;
  const cudaError_t e = abi_tracked(kAbiNormBwd, dweight ? 2 : 1, st, [&] {
    auto go = [&](auto* gt) {
      using E = std::remove_const_t<std::remove_pointer_t<decltype(gt)>>;
      return launch_bwd<E>(gt, static_cast<const E*>(d_total), static_cast<const E*>(total), rstd,
                           static_cast<const E*>(weight), T, H, static_cast<E*>(dx), part, blocks,
                           st);
    };
    cudaError_t r = dtype == MOE_FP32 ? go(static_cast<const float*>(dy))
                                      : go(static_cast<const __nv_bfloat16*>(dy));
    if (r == cudaSuccess && dweight) {
      norm_dweight_kernel<<<(H + 31) / 32, 1024, 0, st>>>(part, blocks, H, dweight);
      r = cudaGetLastError();
    }
    return r;
  });
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
