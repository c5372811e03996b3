// Gradient of the router: through the softmax of the chosen logits, with the
// load-balancing loss and the z-loss.
//
// Per row t, with p = softmax(logits[t]), l = log sum exp logits[t],
// f_e = counts[e] E / (T k), F = sum_e f_e p_e and the weights' dot product
// D = sum_j w_j dw_j:
//   d[e] = balance / T * p_e (f_e - F) + 2 z / T * l p_e
//        + sum over the choices j of e: w_j (dw_j - D).
// The balance loss is the mean of F over the rows, the z-loss that of l^2.
//
// One warp per row: the row's logits stay in registers (E <= 1024, so at most 32
// per lane), so they are read once and d is written once: bound by memory.  The
// next row's logits are loaded before this one's arithmetic.  The choices'
// terms go through a row of shared memory per warp (a lane writes its choice's
// term where the lane that owns the column picks it up); a row that names an expert
// twice adds its terms one after the other.  Sums over the rows: per warp and block
// in a fixed order, then one block over all blocks: no atomics.
#include <algorithm>

#include "abi_internal.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxRouteE = 1024;
constexpr int kMaxRouteK = 32;
constexpr int kMaxRouteBlocks = 8 * 256;   // of any device

struct RouteBwd {
  const float* logits;
  const int* idx;
  const float* w;
  const int* counts;
  const float* dw;
  float* d;
  float* part;      // [blocks][2]: sums of F and of l^2, or null
  int* err;
  int64_t T;
  int E, k;
  float balance_T, z2_T;   // balance / T, 2 z / T
  float f_scale;           // E / (T k)
  int softmax;             // the losses or their gradients are wanted
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}
__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// A running sum with what its roundings took (many rows per warp); beyond fp32's
// range it stays infinite.
struct Sum {
  float s = 0.f, c = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float y = v - c, n = s + y;
    c = isfinite(n) ? (n - s) - y : 0.f;
    s = n;
  }
};

// PER columns per lane.  VEC: groups of four, 4 (lane + 32 i) ..; otherwise
// lane + 32 i.
template <int PER, bool VEC>
struct RouteRow {
  static __device__ __forceinline__ int col(int i, int lane) {
    return VEC ? 4 * (lane + 32 * (i / 4)) + i % 4 : lane + 32 * i;
  }
  static __device__ __forceinline__ void load(const float* row, int E, int lane, float fill, float (&v)[PER]) {
    if (VEC) {
#pragma unroll
      for (int i = 0; i < PER; i += 4) {
        const int c = col(i, lane);
        float4 q = make_float4(fill, fill, fill, fill);
        if (c < E) q = __ldg(reinterpret_cast<const float4*>(row + c));
        v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = col(i, lane);
        v[i] = c < E ? __ldg(row + c) : fill;
      }
    }
  }
  static __device__ __forceinline__ void store(float* row, int E, int lane, const float (&v)[PER]) {
    if (VEC) {
#pragma unroll
      for (int i = 0; i < PER; i += 4) {
        const int c = col(i, lane);
        if (c < E) *reinterpret_cast<float4*>(row + c) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = col(i, lane);
        if (c < E) row[c] = v[i];
      }
    }
  }
};

template <int PER, bool VEC>
__global__ void __launch_bounds__(32 * kWarps) route_bwd_kernel(const RouteBwd a) {
  using Row = RouteRow<PER, VEC>;
  __shared__ __align__(16) float terms[kWarps][32 * PER];
  __shared__ float sums[kWarps][2];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* term = terms[warp];
  const bool chosen = a.dw != nullptr;
  const bool softmax = a.softmax != 0;
  if (chosen)
    for (int i = lane; i < 32 * PER; i += 32) term[i] = 0.f;
  __syncwarp();
  float f[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = Row::col(i, lane);
    f[i] = a.counts && c < a.E ? static_cast<float>(__ldg(a.counts + c)) * a.f_scale : 0.f;
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  float next[PER];
  int n_id = -1;
  float n_w = 0.f, n_dw = 0.f;
  auto fetch = [&](int64_t row) {
    if (softmax) Row::load(a.logits + row * a.E, a.E, lane, -INFINITY, next);
    if (chosen && lane < a.k) {
      n_id = __ldg(a.idx + row * a.k + lane);
      n_w = __ldg(a.w + row * a.k + lane);
      n_dw = __ldg(a.dw + row * a.k + lane);
    }
  };
  Sum sum_F, sum_l;
  if (t < a.T) fetch(t);
  for (; t < a.T; t += step) {
    float v[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = next[i];
    int id = n_id;
    const float w = n_w, dw = n_dw;
    if (t + step < a.T) fetch(t + step);
    float d[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) d[i] = 0.f;
    if (softmax) {
      float top = v[0];
#pragma unroll
      for (int i = 1; i < PER; ++i) top = fmaxf(top, v[i]);
      top = warp_max(top);
      if (top == -INFINITY) top = 0.f;      // every expert masked: p = 0
      float s = 0.f, F = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        v[i] = expf(v[i] - top);
        s += v[i];
        F = fmaf(v[i], f[i], F);
      }
      s = warp_add(s);
      F = warp_add(F);
      // (a row that is NaN has s = NaN, which is not 0: it stays NaN)
      const float inv = s == 0.f ? 0.f : 1.f / s;
      const float l = s == 0.f ? 0.f : top + logf(s);
      F *= inv;
      sum_F.add(F);
      sum_l.add(l * l);
      const float b = a.balance_T * inv, zl = a.z2_T * l * inv;
#pragma unroll
      for (int i = 0; i < PER; ++i) d[i] = v[i] * fmaf(b, f[i] - F, zl);
    }
    if (chosen) {
      const bool mine = lane < a.k;
      if (mine && static_cast<unsigned>(id) >= static_cast<unsigned>(a.E)) {
        record_error(a.err, kErrBadIndex);
        id = -1;
      }
      const float D = warp_add(mine ? w * dw : 0.f);
      const float c = w * (dw - D);
      const bool live = mine && id >= 0;
      // lanes with the same expert (the others have their own number, past all ids)
      const uint32_t same = __match_any_sync(0xffffffffu, live ? id : kMaxRouteE + lane);
      if (__any_sync(0xffffffffu, (same & (same - 1)) != 0)) {
        for (int j = 0; j < a.k; ++j) {
          if (lane == j && live) term[id] += c;
          __syncwarp();
        }
      } else if (live) {
        term[id] = c;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < PER; i += VEC ? 4 : 1) {
        const int col = Row::col(i, lane);
        if (VEC) {
          const float4 q = *reinterpret_cast<const float4*>(term + col);
          d[i] += q.x, d[i + 1] += q.y, d[i + 2] += q.z, d[i + 3] += q.w;
        } else {
          d[i] += term[col];
        }
      }
      __syncwarp();
      if (live) term[id] = 0.f;
      __syncwarp();
    }
    Row::store(a.d + t * a.E, a.E, lane, d);
  }
  if (!a.part) return;
  if (lane == 0) sums[warp][0] = sum_F.s - sum_F.c, sums[warp][1] = sum_l.s - sum_l.c;
  __syncthreads();
  if (threadIdx.x < 2) {
    float s = 0.f;
    for (int i = 0; i < kWarps; ++i) s += sums[i][threadIdx.x];
    a.part[2 * blockIdx.x + threadIdx.x] = s;
  }
}

// losses[i] = sum of the blocks' sums / T: thread q adds blocks q, q + 128, ...,
// the threads' sums are added in a tree; in 64 bits.
__global__ void __launch_bounds__(256) route_losses_kernel(const float* __restrict__ part, int blocks,
                                                           double inv_T, float* __restrict__ losses) {
  __shared__ double s[2][128];
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the sums are there
  const int i = threadIdx.x & 1, q = threadIdx.x >> 1;
  double v = 0.0;
  for (int b = q; b < blocks; b += 128) v += static_cast<double>(__ldcg(part + 2 * b + i));
  s[i][q] = v;
  __syncthreads();
  for (int n = 64; n > 0; n >>= 1) {
    if (q < n) s[i][q] += s[i][q + n];
    __syncthreads();
  }
  if (q == 0) losses[i] = static_cast<float>(s[i][0] * inv_T);
}

template <int PER, bool VEC>
cudaError_t launch_route_bwd(const RouteBwd& a, int blocks, cudaStream_t st) {
  route_bwd_kernel<PER, VEC><<<blocks, 32 * kWarps, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_route_bwd_workspace_size(const moe_shape* s) {
  if (!abi_shape_ok(s)) return 0;
  return 256 + abi_align256(sizeof(float) * 2 * kMaxRouteBlocks);
}

moe_status moe_route_bwd(const moe_shape* s, const float* logits, const int32_t* topk_idx,
                         const float* topk_w, const int32_t* counts, const float* d_topk_w,
                         float balance, float z, float* d_logits, float* losses, void* ws,
                         size_t ws_bytes, moe_stream_t stream) {
  if (!abi_shape_ok(s) || s->E > kMaxRouteE || s->k > kMaxRouteK) return MOE_ERR_INVALID_ARG;
  if (!(balance - balance == 0.f) || !(z - z == 0.f)) return MOE_ERR_INVALID_ARG;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_route_bwd_workspace_size(s)) return MOE_ERR_WORKSPACE;
  const bool softmax = losses || balance != 0.f || z != 0.f;
  if (s->T > 0) {
    if (!d_logits || (d_topk_w && (!topk_idx || !topk_w)) || (softmax && (!logits || !counts)))
      return MOE_ERR_INVALID_ARG;
    if (!abi_aligned16(logits) || !abi_aligned16(d_logits)) return MOE_ERR_INVALID_ARG;
  }
  int sms = 0;
  const moe_status ds = abi_device_sms(&sms);
  if (ds != MOE_OK) return ds;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (s->T == 0) {
    if (losses && abi_tracked_memset(losses, 0, 2 * sizeof(float), st) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  const double T = static_cast<double>(s->T);
  RouteBwd a;
  a.logits = softmax ? logits : nullptr, a.idx = topk_idx, a.w = topk_w, a.dw = d_topk_w;
  a.counts = softmax ? counts : nullptr, a.d = d_logits;
  a.part = losses ? reinterpret_cast<float*>(static_cast<char*>(ws) + 256) : nullptr;
  a.err = static_cast<int*>(ws);
  a.T = s->T, a.E = s->E, a.k = s->k;
  a.balance_T = static_cast<float>(balance / T), a.z2_T = static_cast<float>(2.0 * z / T);
  a.f_scale = static_cast<float>(s->E / (T * s->k));
  a.softmax = softmax ? 1 : 0;
  const int E = s->E;
  const int per_sm = E <= 256 ? 8 : (E <= 512 ? 4 : 2);
  const int blocks = static_cast<int>(std::min<int64_t>(
      (s->T + kWarps - 1) / kWarps, std::min(kMaxRouteBlocks, sms * per_sm)));
  const cudaError_t e = abi_tracked(kAbiRouteBwd, losses ? 2 : 1, st, [&] {
    cudaError_t r;
    if (E % 4 == 0)
      r = E <= 128 ? launch_route_bwd<4, true>(a, blocks, st)
          : E <= 256 ? launch_route_bwd<8, true>(a, blocks, st)
          : E <= 512 ? launch_route_bwd<16, true>(a, blocks, st)
                     : launch_route_bwd<32, true>(a, blocks, st);
    else
      r = E <= 128 ? launch_route_bwd<4, false>(a, blocks, st)
          : E <= 256 ? launch_route_bwd<8, false>(a, blocks, st)
          : E <= 512 ? launch_route_bwd<16, false>(a, blocks, st)
                     : launch_route_bwd<32, false>(a, blocks, st);
    if (r != cudaSuccess || !losses) return r;
    // (may start while the last rows are done)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, route_losses_kernel, static_cast<const float*>(a.part), blocks, 1.0 / T, losses);
  });
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
