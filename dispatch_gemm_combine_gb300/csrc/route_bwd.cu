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
// following rows' logits are copied ahead into shared memory, each warp's into its own
// part.  The choices' terms go through a row of shared memory (a lane writes its
// choice's term where the lane that owns the column picks it up); a row that names an
// expert twice adds its terms one after the other.  Sums over the rows: a lane keeps
// every G-th row's, then over warp and block in a fixed order, then a second kernel
// over all blocks, in their order too.
//
// Measured: 65536 x 256, top-8, 31 us (29 in the kernel): 300 instructions a row and the
// latency of its shuffles, at 29 warps per SM, hold it at two thirds of the memory's
// rate; 65536 x 128 on half warps 19 us (33 on whole ones).
#include <algorithm>
#include <atomic>

#include "abi_internal.h"
#include "common.cuh"
#include "rows.cuh"
#include "vec.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
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
  float2* part;     // [blocks]: sums of F and of l^2, or null
  float* losses;
  int* err;
  int64_t T;
  int E, k;
  float balance_T, z2_T;   // balance / T, 2 z / T
  float f_scale, inv_T;    // E / (T k), 1 / T
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

// 4 or 16 bytes to shared memory, without a branch.
template <int BYTES>
__device__ __forceinline__ void copy_if(uint32_t dst, const float* src, bool on) {
  if (BYTES == 16)
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(dst), "l"(src), "r"(static_cast<int>(on)) : "memory");
  else
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p cp.async.ca.shared.global [%0], [%1], 4;\n\t}" ::"r"(dst), "l"(src), "r"(static_cast<int>(on)) : "memory");
}

// losses[i] = sum of the blocks' sums / T: a thread adds blocks q, q + 256, ..., then the
// threads' sums by warps: sixteen fp32 additions deep.  (In 64 bits, of which this GPU
// adds few a clock, the call takes 2 us more.)  A kernel of its own, which starts while
// the last rows are done.  (The block that comes last could add them too, 8192 x 128 8.3 us
// a call among others instead of 10.2, 12.9 alone instead of 11.9, but would be found by a
// count that the workspace keeps from call to call.)
__global__ void __launch_bounds__(kThreads) route_losses_kernel(const float2* part, int blocks, float inv_T, float* losses) {
  __shared__ float sums[kWarps][2];
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the sums are there
  float2 v[kMaxRouteBlocks / kThreads];
#pragma unroll
  for (int i = 0; i < kMaxRouteBlocks / kThreads; ++i) {
    const int b = threadIdx.x + kThreads * i;
    v[i] = b < blocks ? __ldcg(part + b) : make_float2(0.f, 0.f);
  }
  float x = 0.f, y = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxRouteBlocks / kThreads; ++i) x += v[i].x, y += v[i].y;
  x = warp_sum(x), y = warp_sum(y);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5][0] = x, sums[threadIdx.x >> 5][1] = y;
  __syncthreads();
  if (threadIdx.x < 2) {
    float t = 0.f;
    for (int i = 0; i < kWarps; ++i) t += sums[i][threadIdx.x];
    losses[threadIdx.x] = t * inv_T;
  }
}

// PER columns in each of a row's G lanes.  VEC: groups of four, 4 (g + G i) ..; otherwise
// g + G i.
constexpr int kRowsAhead = 3;

template <int G, int PER, bool VEC>
__global__ void __launch_bounds__(kThreads) route_bwd_kernel(const RouteBwd a) {
  constexpr int R = 32 / G;             // rows of a warp
  constexpr int S = VEC ? 4 : 1;        // columns side by side
  constexpr int W = G * PER;            // floats of a row in shared memory
  extern __shared__ __align__(16) float row_mem[];      // [kWarps][kRowsAhead + 1][R][W]: the last one for the terms
  __shared__ float sums[kWarps][2];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane % G, sub = lane / G;
  const bool chosen = a.dw != nullptr;
  const bool softmax = a.softmax != 0;
  float* mine = row_mem + (warp * (kRowsAhead + 1) * R + sub) * W + g * S;   // this lane's first columns
  float* terms = row_mem + ((warp * (kRowsAhead + 1) + kRowsAhead) * R + sub) * W;
  constexpr int stage_floats = R * W;
  auto col = [&](int i) { return S * (g + G * (i / S)) + i % S; };
  // columns that do not exist: -inf for the logits
#pragma unroll
  for (int q = 0; q <= kRowsAhead; ++q)
#pragma unroll
    for (int i = 0; i < PER; ++i) mine[q * stage_floats + (i / S) * G * S + i % S] = q < kRowsAhead ? -INFINITY : 0.f;
  float f[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) f[i] = a.counts && col(i) < a.E ? static_cast<float>(__ldg(a.counts + col(i))) * a.f_scale : 0.f;
  __syncwarp();

  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * R;
  int64_t t = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * R + sub;
  int64_t ahead = t;                          // the next row to be copied
  const uint32_t mine_s = smem_u32(mine);
  auto copy = [&](int stage) {
    if (softmax && ahead < a.T) {
      const float* src = a.logits + ahead * a.E + g * S;
#pragma unroll
      for (int i = 0; i < PER; i += S)
        copy_if<4 * S>(mine_s + (stage * stage_floats + (i / S) * G * S) * 4, src + (i / S) * G * S, col(i) < a.E);
    }
    cp_async_commit();
    ahead += step;
  };
#pragma unroll
  for (int q = 0; q < kRowsAhead - 1; ++q) copy(q);
  int id = -1, n_id = -1;
  float w = 0.f, dw = 0.f, n_w = 0.f, n_dw = 0.f;
  auto choice = [&](int64_t row) {
    // (kept and advanced, the addresses cost a quarter of the warps: 65536 x 256 41 us
    // instead of 31)
    if (chosen && g < a.k && row < a.T) {
      n_id = __ldg(a.idx + row * a.k + g);
      n_w = __ldg(a.w + row * a.k + g);
      n_dw = __ldg(a.dw + row * a.k + g);
    }
  };
  choice(t);
  float sum_F = 0.f, sum_l = 0.f;
  int stage = 0, turn = 0;
  // (the warp's rows begin together: t - sub is the same in all lanes)
  for (; t - sub < a.T; t += step) {
    const bool on = R == 1 || t < a.T;
    id = n_id, w = n_w, dw = n_dw;
    choice(t + step);
    cp_async_wait<kRowsAhead - 2>();
    copy(stage == 0 ? kRowsAhead - 1 : stage - 1);
    float4 s = make_float4(0.f, 0.f, w * dw, 0.f);
    float v[PER];
    float top = 0.f;
    if (softmax) {
#pragma unroll
      for (int i = 0; i < PER; i += S) {
        const float* p = mine + stage * stage_floats + (i / S) * G * S;
        if (VEC) {
          const float4 q = *reinterpret_cast<const float4*>(p);
          v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
        } else {
          v[i] = *p;
        }
      }
      top = v[0];
#pragma unroll
      for (int i = 1; i < PER; ++i) top = fmaxf(top, v[i]);
      top = row_max<G>(top);
      if (top == -INFINITY) top = 0.f;      // every expert masked: p = 0
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        v[i] = __expf(v[i] - top);
        s.x += v[i];
        s.y = fmaf(v[i], f[i], s.y);
      }
    }
    stage = stage + 1 == kRowsAhead ? 0 : stage + 1;
    s = row_sum4<G>(s);
    const float c = w * (dw - s.z);
    bool live = false;
    if (chosen) {
      live = on && g < a.k;
      if (live && static_cast<unsigned>(id) >= static_cast<unsigned>(a.E)) {
        record_error(a.err, kErrBadIndex);
        live = false;
      }
      // lanes with the same expert of the same row (the others have numbers of their own)
      const uint32_t same = __match_any_sync(0xffffffffu, live ? id + sub * kMaxRouteE : 32 * kMaxRouteE + lane);
      if (__any_sync(0xffffffffu, (same & (same - 1)) != 0)) {
        for (int j = 0; j < a.k; ++j) {
          if (g == j && live) terms[id] += c;
          __syncwarp();
        }
      } else if (live) {
        terms[id] = c;
      }
      __syncwarp();
    }
    float b = 0.f, rest = 0.f;
    if (softmax) {
      // (a row that is NaN has s = NaN, which is not 0: it stays NaN)
      const float inv = s.x == 0.f ? 0.f : __fdividef(1.f, s.x);
      const float l = s.x == 0.f ? 0.f : top + logf(s.x);
      const float F = s.y * inv;
      if (on && g == (turn & (G - 1))) {
        sum_F += F;
        sum_l = fmaf(l, l, sum_l);
      }
      ++turn;
      b = a.balance_T * inv, rest = fmaf(a.z2_T * l, inv, -b * F);
    }
    float* out = a.d + t * a.E + g * S;
#pragma unroll
    for (int i = 0; i < PER; i += S) {
      float d[S];
      const float* p = terms + g * S + (i / S) * G * S;
      if (VEC) {
        const float4 q = *reinterpret_cast<const float4*>(p);
        d[0] = q.x, d[1 % S] = q.y, d[2 % S] = q.z, d[3 % S] = q.w;
      } else {
        d[0] = *p;
      }
      if (softmax)
#pragma unroll
        for (int j = 0; j < S; ++j) d[j] = fmaf(v[i + j], fmaf(b, f[i + j], rest), d[j]);
      if (on && col(i) < a.E) {
        if (VEC)
          *reinterpret_cast<float4*>(out + (i / S) * G * S) = make_float4(d[0], d[1 % S], d[2 % S], d[3 % S]);
        else
          out[(i / S) * G * S] = d[0];
      }
    }
    __syncwarp();
    if (live) terms[id] = 0.f;
    __syncwarp();
  }
  if (!a.part) return;
  sum_F = warp_sum(sum_F), sum_l = warp_sum(sum_l);
  if (lane == 0) sums[warp][0] = sum_F, sums[warp][1] = sum_l;
  __syncthreads();
  if (threadIdx.x == 0) {
    float2 v = make_float2(0.f, 0.f);
    for (int i = 0; i < kWarps; ++i) v.x += sums[i][0], v.y += sums[i][1];
    if (gridDim.x == 1)        // no other block's to be added
      a.losses[0] = v.x * a.inv_T, a.losses[1] = v.y * a.inv_T;
    else
      __stcg(a.part + blockIdx.x, v);
  }
}

template <int G, int PER, bool VEC>
cudaError_t launch_route_bwd_v(RouteBwd& a, int sms, int* blocks, cudaStream_t st) {
  constexpr int R = 32 / G * kWarps;
  constexpr int smem = kWarps * (kRowsAhead + 1) * 32 * PER * static_cast<int>(sizeof(float));
  // by registers (five blocks of 48 registers spill: 65536 x 256 38 us instead of 33), but
  // for 16 columns one by one: 107 registers leave room for two, and the third one waits
  constexpr int per_sm = std::min(PER <= 8 ? 4 : (PER <= 16 ? 3 : 1), kRingPerSm / smem);
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(route_bwd_kernel<G, PER, VEC>, ready);
  if (e != cudaSuccess) return e;
  const int most = std::min(kMaxRouteBlocks, sms * per_sm);
  *blocks = static_cast<int>(std::min<int64_t>((a.T + R - 1) / R, most));
  // two rounds of one block take less than the sum of two blocks' sums
  if (*blocks == 2 && a.losses) *blocks = 1;
  route_bwd_kernel<G, PER, VEC><<<*blocks, kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

template <int G, int PER>
cudaError_t launch_route_bwd(RouteBwd& a, int sms, int* blocks, cudaStream_t st) {
  return a.E % 4 == 0 ? launch_route_bwd_v<G, PER, true>(a, sms, blocks, st)
                      : launch_route_bwd_v<G, PER, false>(a, sms, blocks, st);
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
  a.part = losses ? reinterpret_cast<float2*>(static_cast<char*>(ws) + 256) : nullptr;
  a.err = static_cast<int*>(ws);
  a.T = s->T, a.E = s->E, a.k = s->k;
  a.balance_T = static_cast<float>(balance / T), a.z2_T = static_cast<float>(2.0 * z / T);
  a.losses = losses;
  a.f_scale = static_cast<float>(s->E / (T * s->k)), a.inv_T = static_cast<float>(1.0 / T);
  a.softmax = softmax ? 1 : 0;
  const int E = s->E;
  int blocks = 0;
  cudaError_t e = abi_tracked(kAbiRouteBwd, 1, st, [&] {
    // a choice per lane: k lanes at least
    return E <= 64 && s->k <= 8     ? launch_route_bwd<8, 8>(a, sms, &blocks, st)
           : E <= 128 && s->k <= 16 ? launch_route_bwd<16, 8>(a, sms, &blocks, st)
           : E <= 256               ? launch_route_bwd<32, 8>(a, sms, &blocks, st)
           : E <= 512               ? launch_route_bwd<32, 16>(a, sms, &blocks, st)
                                    : launch_route_bwd<32, 32>(a, sms, &blocks, st);
  });
  if (e == cudaSuccess && losses && blocks > 1)
    e = abi_tracked(kAbiRouteBwd, 1, st, [&] {
      // (may start while the last rows are done)
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(1);
      cfg.blockDim = dim3(kThreads);
      cfg.stream = st;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      return cudaLaunchKernelEx(&cfg, route_losses_kernel, static_cast<const float2*>(a.part), blocks, a.inv_T, losses);
    });
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
