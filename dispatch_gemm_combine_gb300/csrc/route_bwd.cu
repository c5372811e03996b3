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
// A row's logits stay in the registers of G lanes, PER in each (a warp for more than 128
// experts, half of one or a quarter for fewer: what a row costs beside its columns is
// then shared by two or four rows), so they are read once and d is written once.  The
// next rows' logits are loaded before this one's arithmetic.  The choices' terms go
// through a row of shared memory (a lane writes its choice's term where the lane that
// owns the column picks it up); a row that names an expert twice adds its terms one
// after the other.  Sums over the rows: per warp and block in a fixed order, then one
// block over all blocks: no atomics.
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

// Over the G lanes of a row.
template <int G>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int d = G / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}
// Four sums at once (two exchanges leave each lane one of the four), in every lane.
template <int G>
__device__ __forceinline__ float4 row_sum4(const float4& v) {
  const int lane = threadIdx.x & 31;
  const bool odd = lane & 1, high = lane & 2;
  float a = odd ? v.z : v.x, b = odd ? v.w : v.y;
  a += __shfl_xor_sync(0xffffffffu, odd ? v.x : v.z, 1);
  b += __shfl_xor_sync(0xffffffffu, odd ? v.y : v.w, 1);
  float s = high ? b : a;
  s += __shfl_xor_sync(0xffffffffu, high ? a : b, 2);
#pragma unroll
  for (int d = 4; d < G; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  return make_float4(__shfl_sync(0xffffffffu, s, 0, G), __shfl_sync(0xffffffffu, s, 2, G),
                     __shfl_sync(0xffffffffu, s, 1, G), __shfl_sync(0xffffffffu, s, 3, G));
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

// PER columns in each of a row's G lanes.  VEC: groups of four, 4 (g + G i) ..; otherwise
// g + G i.
template <int G, int PER, bool VEC>
struct RouteRow {
  static __device__ __forceinline__ int col(int i, int g) {
    return VEC ? 4 * (g + G * (i / 4)) + i % 4 : g + G * i;
  }
  static __device__ __forceinline__ void load(const float* row, int E, int g, bool on, float (&v)[PER]) {
    constexpr int S = VEC ? 4 : 1;
#pragma unroll
    for (int i = 0; i < PER; i += S) {
      const int c = col(i, g);
      const bool in = on && c < E;
      if (VEC) {
        const float4 q = in ? __ldg(reinterpret_cast<const float4*>(row + c))
                            : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
      } else {
        v[i] = in ? __ldg(row + c) : -INFINITY;
      }
    }
  }
  static __device__ __forceinline__ void store(float* row, int E, int g, bool on, const float (&v)[PER]) {
    constexpr int S = VEC ? 4 : 1;
#pragma unroll
    for (int i = 0; i < PER; i += S) {
      const int c = col(i, g);
      if (on && c < E) {
        if (VEC)
          *reinterpret_cast<float4*>(row + c) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        else
          row[c] = v[i];
      }
    }
  }
};

template <int G, int PER, bool VEC>
__global__ void __launch_bounds__(32 * kWarps) route_bwd_kernel(const RouteBwd a) {
  using Row = RouteRow<G, PER, VEC>;
  constexpr int R = 32 / G;      // rows of a warp
  __shared__ __align__(16) float terms[kWarps][32 * PER];
  __shared__ float sums[kWarps][2];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane % G, sub = lane / G;
  float* term = terms[warp] + sub * G * PER;
  const bool chosen = a.dw != nullptr;
  const bool softmax = a.softmax != 0;
  if (chosen)
    for (int i = lane; i < 32 * PER; i += 32) terms[warp][i] = 0.f;
  __syncwarp();
  float f[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = Row::col(i, g);
    f[i] = a.counts && c < a.E ? static_cast<float>(__ldg(a.counts + c)) * a.f_scale : 0.f;
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * R;
  struct Ahead {
    float v[PER];
    int id;
    float w, dw;
  };
  auto fetch = [&](int64_t row, Ahead& n) {
    const bool on = row < a.T;
    if (softmax) Row::load(a.logits + row * a.E, a.E, g, on, n.v);
    n.id = -1, n.w = n.dw = 0.f;
    if (chosen && on && g < a.k) {
      n.id = __ldg(a.idx + row * a.k + g);
      n.w = __ldg(a.w + row * a.k + g);
      n.dw = __ldg(a.dw + row * a.k + g);
    }
  };
  Sum sum_F, sum_l;
  // t: this lane's row; `now` holds it, `next` receives the one after
  auto work = [&](int64_t t, Ahead& now, Ahead& next) {
    fetch(t + step, next);
    const bool on = t < a.T;
    float d[PER];
    float4 s = make_float4(0.f, 0.f, now.w * now.dw, 0.f);
    float top = 0.f;
    if (softmax) {
      top = now.v[0];
#pragma unroll
      for (int i = 1; i < PER; ++i) top = fmaxf(top, now.v[i]);
      top = row_max<G>(top);
      if (top == -INFINITY) top = 0.f;      // every expert masked: p = 0
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        now.v[i] = exp2f((now.v[i] - top) * 1.44269504f);
        s.x += now.v[i];
        s.y = fmaf(now.v[i], f[i], s.y);
      }
    }
    s = row_sum4<G>(s);
#pragma unroll
    for (int i = 0; i < PER; ++i) d[i] = 0.f;
    if (chosen) {
      const float D = s.z, c = now.w * (now.dw - D);
      bool live = on && g < a.k;
      if (live && static_cast<unsigned>(now.id) >= static_cast<unsigned>(a.E)) {
        record_error(a.err, kErrBadIndex);
        live = false;
      }
      // lanes with the same expert of the same row (the others have numbers of their own)
      const uint32_t same = __match_any_sync(0xffffffffu, live ? now.id + sub * kMaxRouteE : 32 * kMaxRouteE + lane);
      if (__any_sync(0xffffffffu, (same & (same - 1)) != 0)) {
        for (int j = 0; j < a.k; ++j) {
          if (g == j && live) term[now.id] += c;
          __syncwarp();
        }
      } else if (live) {
        term[now.id] = c;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < PER; i += VEC ? 4 : 1) {
        const int col = Row::col(i, g);
        if (VEC) {
          const float4 q = *reinterpret_cast<const float4*>(term + col);
          d[i] = q.x, d[i + 1] = q.y, d[i + 2] = q.z, d[i + 3] = q.w;
        } else {
          d[i] = term[col];
        }
      }
      __syncwarp();
      if (live) term[now.id] = 0.f;
      __syncwarp();
    }
    if (softmax) {
      // (a row that is NaN has s = NaN, which is not 0: it stays NaN)
      const float inv = s.x == 0.f ? 0.f : __fdividef(1.f, s.x);
      const float l = s.x == 0.f ? 0.f : top + logf(s.x);
      const float F = s.y * inv;
      if (on) {
        sum_F.add(F);
        sum_l.add(l * l);
      }
      const float b = a.balance_T * inv, rest = fmaf(a.z2_T * l, inv, -b * F);
#pragma unroll
      for (int i = 0; i < PER; ++i) d[i] = fmaf(now.v[i], fmaf(b, f[i], rest), d[i]);
    }
    Row::store(a.d + t * a.E, a.E, g, on, d);
  };
  int64_t t = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * R + sub;
  Ahead x, y;
  fetch(t, x);
  // (the warp's rows begin together: t - sub is the same in all lanes)
  for (; t - sub < a.T; t += 2 * step) {
    work(t, x, y);
    if (t - sub + step < a.T) work(t + step, y, x);
  }
  if (!a.part) return;
  float2 v = make_float2(sum_F.s - sum_F.c, sum_l.s - sum_l.c);
#pragma unroll
  for (int n = G; n < 32; n <<= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, n);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, n);
  }
  if (lane == 0) sums[warp][0] = v.x, sums[warp][1] = v.y;
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

template <int G, int PER>
cudaError_t launch_route_bwd(const RouteBwd& a, int sms, int* blocks, cudaStream_t st) {
  constexpr int R = 32 / G * kWarps;
  constexpr int per_sm = PER <= 8 ? 4 : (PER <= 16 ? 2 : 1);      // by registers
  *blocks = static_cast<int>(std::min<int64_t>((a.T + R - 1) / R, std::min(kMaxRouteBlocks, sms * per_sm)));
  if (a.E % 4 == 0)
    route_bwd_kernel<G, PER, true><<<*blocks, 32 * kWarps, 0, st>>>(a);
  else
    route_bwd_kernel<G, PER, false><<<*blocks, 32 * kWarps, 0, st>>>(a);
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
  int blocks = 0;
  const cudaError_t e = abi_tracked(kAbiRouteBwd, losses ? 2 : 1, st, [&] {
    // a choice per lane: k lanes at least
    const cudaError_t r = E <= 64 && s->k <= 8 ? launch_route_bwd<8, 8>(a, sms, &blocks, st)
                          : E <= 128 && s->k <= 16 ? launch_route_bwd<16, 8>(a, sms, &blocks, st)
                          : E <= 256 ? launch_route_bwd<32, 8>(a, sms, &blocks, st)
                          : E <= 512 ? launch_route_bwd<32, 16>(a, sms, &blocks, st)
                                     : launch_route_bwd<32, 32>(a, sms, &blocks, st);
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
