// A block's output joins the residual stream, with the norms on either side:
//
//   p = y * rs_y * post_weight  (post_norm)  or  y * post_weight,
//   r = residual_scale * residual + gate * p,
//   n = r * rs * weight,       rs = (mean_h r^2 + eps)^-1/2, rs_y likewise of y,
//
// and the gradient.  Forward: as the RMS norm's (norm.cu): a block walks rows, each
// thread holds 8 * V columns in registers, y and the residual are read once and the
// outputs written once.  Two sums over a row: of y^2, then of r^2.
//
// Backward, with rhat = r * rs, q = y * rs_y * post_weight, v = dn * weight,
// u = d_total + rs * v:
//   m  = mean_h(v rhat),   dr = u - rs m rhat,
//   D  = sum_h dr q = sum u q - rs m sum rhat q           (the gate's gradient),
//   dy = rs_y (gate dr post_weight - y rs_y gate D / H),   d_residual = scale dr,
//   d_post_weight[h] = sum_t gate dr y rs_y,   d_weight[h] = sum_t dn rhat.
// The three sums over a row (v rhat, u q, rhat q) do not wait for one another, so a
// row costs one reduction.  The weights' sums stay in registers over a block's rows
// and are joined by a second kernel in block order: no atomics.
#include <algorithm>
#include <atomic>

#include "abi_internal.h"
#include "common.cuh"
#include "rows.cuh"
#include "vec.cuh"

namespace moe {
namespace {

struct JoinFwd {
  const void *y, *residual, *post_weight, *weight;
  const float* gate;
  void *total, *n;
  uint8_t* n_scale;
  float *rstd_post, *rstd;
  int64_t T;
  int H;
  float scale, eps;
  int post_norm;
};

enum JoinOut : int { kNoNorm = 0, kSameType = 1, kE4m3 = 2 };

template <typename E, int OUT, int V, int D>
__global__ void __launch_bounds__(1024) join_fwd_kernel(const JoinFwd a) {
  extern __shared__ uint4 ring_mem[];
  __shared__ float part[4][32];
  const int H = a.H;
  const int64_t T = a.T;
  const E* post_weight = static_cast<const E*>(a.post_weight);
  const E* weight = static_cast<const E*>(a.weight);
  E* total = static_cast<E*>(a.total);
  RowRing<E, 2, V, D> rows{ring_mem, {static_cast<const E*>(a.y), static_cast<const E*>(a.residual)}, H};
#pragma unroll
  for (int d = 0; d < D - 1; ++d) rows.issue(d, blockIdx.x + static_cast<int64_t>(d) * gridDim.x, T);
  int stage = 0, flip = 0;   // a row's barriers also separate the reuse of the other sums
  for (int64_t row = blockIdx.x; row < T; row += gridDim.x, flip ^= 2) {
    const int64_t base = row * H;
    if (D > 0) {
      rows.wait();
      rows.issue(stage == 0 ? D - 1 : stage - 1, row + static_cast<int64_t>(D - 1) * gridDim.x, T);
    }
    Raw8<E> ry[V], rr[V];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c < H) {
        rows.take(stage, 0, i, row, c, ry[i]);
        rows.take(stage, 1, i, row, c, rr[i]);
        if (a.post_norm) {
#pragma unroll
          for (int j = 0; j < 8; ++j) ss = fmaf(ry[i].get(j), ry[i].get(j), ss);
        }
      }
    }
    if (D > 0) stage = stage + 1 == D ? 0 : stage + 1;
    float rs_y = 1.f;
    if (a.post_norm) {
      ss = block_sum(ss, part[flip]);
      rs_y = 1.f / sqrtf(ss / static_cast<float>(H) + a.eps);
      if (a.rstd_post && threadIdx.x == 0) a.rstd_post[row] = rs_y;
    }
    const float gate = a.gate ? __ldg(a.gate + row) : 1.f;
    float r[V][8];
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c < H) {
        Raw8<E> w;
        if (post_weight) w.load(post_weight + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float p = ry[i].get(j) * rs_y;
          if (post_weight) p *= w.get(j);
          r[i][j] = fmaf(a.scale, rr[i].get(j), gate * p);
          if (OUT != kNoNorm) ss = fmaf(r[i][j], r[i][j], ss);
        }
        store8(total + base + c, r[i]);
      }
    }
    if (OUT == kNoNorm) continue;
    ss = block_sum(ss, part[flip + 1]);
    const float rs = 1.f / sqrtf(ss / static_cast<float>(H) + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rs;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (OUT == kSameType && c >= H) continue;
      float o[8];
      if (c < H) {
        Raw8<E> w;
        w.load(weight + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = r[i][j] * rs * w.get(j);
      }
      if (OUT == kSameType) {
        store8(static_cast<E*>(a.n) + base + c, o);
      } else {
        store_e4m3(o, c < H, static_cast<uint8_t*>(a.n) + base + c, a.n_scale + row * (H / 32) + c / 32);
      }
    }
  }
}

struct JoinBwd {
  const void *dn, *total, *d_total, *y, *weight, *post_weight;
  const float *rstd, *rstd_post, *gate;
  void *dy, *d_residual;
  float *d_gate, *part;      // part: [2][blocks][H] of the sums of d_weight, d_post_weight, or null
  int64_t T;
  int H;
  float scale;
};

// NEXT: a norm follows (dn, total, weight and rstd are there).
template <typename E, bool NEXT, int V, int D>
__global__ void __launch_bounds__(1024) join_bwd_kernel(const JoinBwd a) {
  extern __shared__ uint4 ring_mem[];
  __shared__ float part[2][3][32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int N = NEXT ? 4 : 2;
  const int H = a.H;
  const int64_t T = a.T;
  RowRing<E, N, V, D> rows{ring_mem, {}, H};
  rows.src[0] = static_cast<const E*>(a.y);
  rows.src[1] = static_cast<const E*>(a.d_total);
  if (NEXT) {
    rows.src[N - 2] = static_cast<const E*>(a.dn);
    rows.src[N - 1] = static_cast<const E*>(a.total);
  }
#pragma unroll
  for (int d = 0; d < D - 1; ++d) rows.issue(d, blockIdx.x + static_cast<int64_t>(d) * gridDim.x, T);
  const E* weight = static_cast<const E*>(a.weight);
  const E* post_weight = static_cast<const E*>(a.post_weight);
  float2 dw[NEXT ? V : 1][4], dwp[V][4];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) dwp[i][j] = dw[NEXT ? i : 0][j] = make_float2(0.f, 0.f);
  const float inv_H = 1.f / static_cast<float>(H);
  const int lane = threadIdx.x & 31;
  // 1 / rms and gate of 32 rows, one per lane (a load per row would wait for the
  // rows' copies)
  float rstds = 0.f, posts = 1.f, gates = 1.f;
  int stage = 0, flip = 0, turn = 0;
  for (int64_t row = blockIdx.x; row < T; row += gridDim.x, flip ^= 1) {
    const int64_t base = row * H;
    if ((turn & 31) == 0) {
      const int64_t mine = row + static_cast<int64_t>(lane) * gridDim.x;
      if (mine < T) {
        if (NEXT) rstds = __ldg(a.rstd + mine);
        if (a.rstd_post) posts = __ldg(a.rstd_post + mine);
        if (a.gate) gates = __ldg(a.gate + mine);
      }
    }
    const float rs = NEXT ? __shfl_sync(0xffffffffu, rstds, turn & 31) : 0.f;
    const float rs_y = __shfl_sync(0xffffffffu, posts, turn & 31);
    const float gate = __shfl_sync(0xffffffffu, gates, turn & 31);
    ++turn;
    if (D > 0) {
      rows.wait();
      rows.issue(stage == 0 ? D - 1 : stage - 1, row + static_cast<int64_t>(D - 1) * gridDim.x, T);
    }
    const float2 rs2 = make_float2(rs, rs), rs_y2 = make_float2(rs_y, rs_y);
    float2 u[V][4], rhat[NEXT ? V : 1][4], yhat[V][4];
    float2 s1 = make_float2(0.f, 0.f), s2 = s1, s3 = s1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c < H) {
        Raw8<E> ry, rt, rn, rr, w, wp;
        rows.take(stage, 0, i, row, c, ry);
        if (a.d_total) rows.take(stage, 1, i, row, c, rt);
        if (NEXT) {
          rows.take(stage, N - 2, i, row, c, rn);
          rows.take(stage, N - 1, i, row, c, rr);
          w.load(weight + c);
        }
        if (post_weight) wp.load(post_weight + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          yhat[i][j] = mul2(ry.pair(j), rs_y2);
          const float2 q = post_weight ? mul2(yhat[i][j], wp.pair(j)) : yhat[i][j];
          float2 uj = a.d_total ? rt.pair(j) : make_float2(0.f, 0.f);
          if (NEXT) {
            const float2 dn = rn.pair(j);
            const float2 v = mul2(dn, w.pair(j));
            const float2 rh = mul2(rr.pair(j), rs2);
            rhat[NEXT ? i : 0][j] = rh;
            uj = fma2(rs2, v, uj);
            s1 = fma2(v, rh, s1);
            s3 = fma2(rh, q, s3);
            dw[NEXT ? i : 0][j] = fma2(dn, rh, dw[NEXT ? i : 0][j]);
          }
          s2 = fma2(uj, q, s2);
          u[i][j] = uj;
        }
      }
    }
    if (D > 0) stage = stage + 1 == D ? 0 : stage + 1;
    float sums[3] = {s2.x + s2.y, s1.x + s1.y, s3.x + s3.y};
    block_sums<NEXT ? 3 : 1>(sums, part[flip]);
    const float rsm = NEXT ? rs * sums[1] * inv_H : 0.f;
    const float dot = NEXT ? fmaf(-rsm, sums[2], sums[0]) : sums[0];
    if (a.d_gate && threadIdx.x == 0) a.d_gate[row] = dot;
    const float back = a.rstd_post ? -gate * dot * inv_H : 0.f;
    const float2 rsm2 = make_float2(-rsm, -rsm), gate2 = make_float2(gate, gate), back2 = make_float2(back, back);
    const float2 scale2 = make_float2(a.scale, a.scale);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c < H) {
        Raw8<E> wp;
        if (post_weight) wp.load(post_weight + c);
        float oy[8], orr[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 dr = NEXT ? fma2(rsm2, rhat[NEXT ? i : 0][j], u[i][j]) : u[i][j];
          const float2 dres = mul2(scale2, dr);
          const float2 dp = mul2(gate2, dr);
          dwp[i][j] = fma2(dp, yhat[i][j], dwp[i][j]);
          const float2 dpw = post_weight ? mul2(dp, wp.pair(j)) : dp;
          const float2 dy = mul2(rs_y2, fma2(back2, yhat[i][j], dpw));
          oy[2 * j] = dy.x, oy[2 * j + 1] = dy.y;
          orr[2 * j] = dres.x, orr[2 * j + 1] = dres.y;
        }
        store8(static_cast<E*>(a.dy) + base + c, oy);
        store8(static_cast<E*>(a.d_residual) + base + c, orr);
      }
    }
  }
  if (a.part) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * 8;
      if (c < H) {
        const int64_t at = static_cast<int64_t>(blockIdx.x) * H + c;
        if (NEXT) store8(a.part + at, &dw[NEXT ? i : 0][0].x);
        store8(a.part + static_cast<int64_t>(gridDim.x) * H + at, &dwp[i][0].x);
      }
    }
  }
}

// out[which][c] = sum of the blocks' partial sums, as norm.cu's: 32 columns by 32
// groups of blocks per thread block, each group in block order, then the groups.
__global__ void __launch_bounds__(1024) join_dweight_kernel(const float* __restrict__ part, int blocks, int H,
                                                            float* __restrict__ d_weight,
                                                            float* __restrict__ d_post_weight) {
  __shared__ float s[32][33];
  float* out = blockIdx.y ? d_post_weight : d_weight;
  if (!out) return;
  const float* p = part + static_cast<int64_t>(blockIdx.y) * blocks * H;
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the sums are there
  if (c < H)
#pragma unroll 8
    for (int b = grp; b < blocks; b += 32) v += __ldcg(p + static_cast<int64_t>(b) * H + c);
  s[grp][lane] = v;
  __syncthreads();
  const float t = warp_sum(s[lane][grp]);
  if (lane == 0 && blockIdx.x * 32 + grp < H) out[blockIdx.x * 32 + grp] = t;
}

template <typename E, int OUT, int V>
cudaError_t launch_join_fwd_v(const JoinFwd& a, int threads, int sms, cudaStream_t st) {
  const NormLaunch l = norm_launch(a.T, threads, RowRing<E, 2, V, kAhead>::bytes(threads), kThreadsPerSm, sms);
  if (l.ring) {
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(join_fwd_kernel<E, OUT, V, kAhead>, ready);
    if (e != cudaSuccess) return e;
    join_fwd_kernel<E, OUT, V, kAhead><<<l.blocks, l.threads, l.smem, st>>>(a);
  } else {
    join_fwd_kernel<E, OUT, V, 0><<<l.blocks, l.threads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

template <typename E, int OUT>
cudaError_t launch_join_fwd(const JoinFwd& a, int sms, cudaStream_t st) {
  const RowShape s = row_shape(a.H);
  if (s.vecs == 1) return launch_join_fwd_v<E, OUT, 1>(a, s.threads, sms, st);
  if (s.vecs == 2) return launch_join_fwd_v<E, OUT, 2>(a, s.threads, sms, st);
  return launch_join_fwd_v<E, OUT, 4>(a, s.threads, sms, st);
}

template <typename E, bool NEXT, int V>
cudaError_t launch_join_bwd_v(const JoinBwd& a, int threads, int sms, int* blocks, cudaStream_t st) {
  const NormLaunch l = norm_launch(a.T, threads, RowRing<E, NEXT ? 4 : 2, V, kAhead>::bytes(threads), kThreadsPerSm, sms);
  *blocks = l.blocks;
  if (l.ring) {
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(join_bwd_kernel<E, NEXT, V, kAhead>, ready);
    if (e != cudaSuccess) return e;
    join_bwd_kernel<E, NEXT, V, kAhead><<<l.blocks, l.threads, l.smem, st>>>(a);
  } else {
    join_bwd_kernel<E, NEXT, V, 0><<<l.blocks, l.threads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

// *blocks: of the launch, each of which leaves its sums in a.part.
template <typename E, bool NEXT>
cudaError_t launch_join_bwd(const JoinBwd& a, int sms, int* blocks, cudaStream_t st) {
  const RowShape s = row_shape(a.H);
  if (s.vecs == 1) return launch_join_bwd_v<E, NEXT, 1>(a, s.threads, sms, blocks, st);
  if (s.vecs == 2) return launch_join_bwd_v<E, NEXT, 2>(a, s.threads, sms, blocks, st);
  return launch_join_bwd_v<E, NEXT, 4>(a, s.threads, sms, blocks, st);
}

bool join_dims_ok(int64_t T, int32_t H, int32_t dtype) {
  return T >= 0 && T < (1ll << 31) && H >= 8 && H % 8 == 0 && H <= kMaxH &&
         (dtype == MOE_BF16 || dtype == MOE_FP32);
}

bool finite(float v) { return v - v == 0.f; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_join_norm_fwd(int64_t T, int32_t H, int32_t dtype, const void* y, const void* residual,
                             int32_t post_norm, const void* post_weight, const float* gate,
                             float residual_scale, const void* weight, float eps, void* total, void* n,
                             uint8_t* n_scale, float* rstd_post, float* rstd, moe_stream_t stream) {
  if (!join_dims_ok(T, H, dtype) || !(eps >= 0.f) || !finite(residual_scale)) return MOE_ERR_INVALID_ARG;
  if ((post_norm != 0 && post_norm != 1) || (n_scale && (!n || H % 32)) || (!n != !weight))
    return MOE_ERR_INVALID_ARG;
  if ((rstd_post && !post_norm) || (rstd && !n)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!y || !residual || !total || n == total) return MOE_ERR_INVALID_ARG;
  for (const void* p : {y, residual, post_weight, weight, static_cast<const void*>(total),
                        static_cast<const void*>(n)})
    if (!abi_aligned16(p)) return MOE_ERR_INVALID_ARG;
  int sms = 0;
  const moe_status ds = abi_device_sms(&sms);
  if (ds != MOE_OK) return ds;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const JoinFwd a{y, residual, post_weight, weight, gate, total, n, n_scale, rstd_post, rstd, T, H,
                  residual_scale, eps, post_norm};
  const cudaError_t e = abi_tracked(kAbiJoinFwd, 1, st, [&] {
    if (dtype == MOE_FP32)
      return !n ? launch_join_fwd<float, kNoNorm>(a, sms, st)
             : n_scale ? launch_join_fwd<float, kE4m3>(a, sms, st)
                       : launch_join_fwd<float, kSameType>(a, sms, st);
    return !n ? launch_join_fwd<__nv_bfloat16, kNoNorm>(a, sms, st)
           : n_scale ? launch_join_fwd<__nv_bfloat16, kE4m3>(a, sms, st)
                     : launch_join_fwd<__nv_bfloat16, kSameType>(a, sms, st);
  });
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_join_norm_workspace_size(int64_t T, int32_t H) {
  if (!join_dims_ok(T, H, MOE_BF16)) return 0;
  return 256 + abi_align256(2 * sizeof(float) * static_cast<size_t>(H) *
                            static_cast<size_t>(std::max<int64_t>(1, std::min<int64_t>(T, kMaxBwdBlocks))));
}

moe_status moe_join_norm_bwd(int64_t T, int32_t H, int32_t dtype, const void* dn, const void* d_total,
                             const void* total, const float* rstd, const void* weight, const void* y,
                             const float* rstd_post, const void* post_weight, const float* gate,
                             float residual_scale, void* dy, void* d_residual, float* d_gate,
                             float* d_post_weight, float* d_weight, void* ws, size_t ws_bytes,
                             moe_stream_t stream) {
  if (!join_dims_ok(T, H, dtype) || !finite(residual_scale)) return MOE_ERR_INVALID_ARG;
  if (T > 0) {
    if (!dn && d_weight) return MOE_ERR_INVALID_ARG;
    if (!y || !dy || !d_residual || dy == d_residual || (!dn && !d_total)) return MOE_ERR_INVALID_ARG;
    if (dn && (!total || !rstd || !weight)) return MOE_ERR_INVALID_ARG;
  }
  for (const void* p : {dn, d_total, total, weight, y, post_weight, static_cast<const void*>(dy),
                        static_cast<const void*>(d_residual), static_cast<const void*>(d_post_weight),
                        static_cast<const void*>(d_weight)})
    if (!abi_aligned16(p)) return MOE_ERR_INVALID_ARG;
  const bool sums = d_weight || d_post_weight;
  if (sums && T > 0) {
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < moe_join_norm_workspace_size(T, H)) return MOE_ERR_WORKSPACE;
  }
  int sms = 0;
  const moe_status ds = abi_device_sms(&sms);
  if (ds != MOE_OK) return ds;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {
    for (float* p : {d_weight, d_post_weight})
      if (p && abi_tracked_memset(p, 0, sizeof(float) * H, st) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  float* part = sums ? reinterpret_cast<float*>(static_cast<char*>(ws) + 256) : nullptr;
  const JoinBwd a{dn, total, d_total, y, weight, post_weight, rstd, rstd_post, gate, dy, d_residual, d_gate,
                  part, T, H, residual_scale};
  int blocks = 0;
  const cudaError_t e = abi_tracked(kAbiJoinBwd, sums ? 2 : 1, st, [&] {
    const int most = std::min(sms, kMaxSms);
    cudaError_t r;
    if (dtype == MOE_FP32)
      r = dn ? launch_join_bwd<float, true>(a, most, &blocks, st) : launch_join_bwd<float, false>(a, most, &blocks, st);
    else
      r = dn ? launch_join_bwd<__nv_bfloat16, true>(a, most, &blocks, st)
             : launch_join_bwd<__nv_bfloat16, false>(a, most, &blocks, st);
    if (r != cudaSuccess || !sums) return r;
    // (may start while the last rows are done)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((H + 31) / 32, 2);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_dweight_kernel, static_cast<const float*>(part), blocks, H, d_weight, d_post_weight);
  });
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
