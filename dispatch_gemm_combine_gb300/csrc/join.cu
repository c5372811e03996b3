// A block's output joins the residual stream, with the norms on either side:
//
//   p = y * rs_y * post_weight  (post_norm)  or  y * post_weight,
//   r = residual_scale * residual + gate * p,
//   n = r * rs * weight,       rs = (mean_h r^2 + eps)^-1/2, rs_y likewise of y,
//
// and the gradient.  Forward: a block walks rows (or has one), y and the residual are
// read once and the outputs written once.  The sum of r^2 follows from four sums that do
// not wait for rs_y: with t = residual_scale * residual, q = y * post_weight and
// f = gate * rs_y, sum r^2 = sum t^2 + f (2 sum t q + f sum q^2), so a row costs one
// reduction (two, one after the other: 132 us instead of 76 at the size below, with the
// steps told at RowStream).  Where the terms cancel to less than a quarter of theirs, or
// leave fp32's range, r^2 is summed once more from r.
//
// Backward, with rhat = r * rs, q = y * rs_y * post_weight, v = dn * weight,
// u = d_total + rs * v:
//   m  = mean_h(v rhat),   dr = u - rs m rhat,
//   D  = sum_h dr q = sum u q - rs m sum rhat q           (the gate's gradient),
//   dy = rs_y (gate dr post_weight - y rs_y gate D / H),   d_residual = scale dr,
//   d_post_weight[h] = sum_t gate dr y rs_y,   d_weight[h] = sum_t dn rhat.
// The three sums over a row (v rhat, u q, rhat q) do not wait for one another either.
// The weights' sums stay in registers over a block's rows and are joined by a second
// kernel in block order: no atomics.
//
// Sums are fp32: 8 values a thread and vector, then butterflies over the warp and the
// warps.  Measured: forward of 16384 x 4096 bf16 with 8-bit output 75 us, 6.3 TB/s (70
// us in the kernel, memory-bound); backward of 8192 x 2880 51 us, of which 45 in the
// first kernel (6.3 TB/s) and the rest in the weights' sums and the step to them.
#include <algorithm>
#include <atomic>

#include "abi_internal.h"
#include "common.cuh"
#include "rows.cuh"
#include "vec.cuh"

namespace moe {
namespace {

__device__ __forceinline__ void cp_async16_if(uint32_t dst, const void* src, uint32_t on) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(dst),
               "l"(src), "r"(on)
               : "memory");
}

// The rows that a block walks (blockIdx.x, + gridDim.x, ..), N arrays of them, D - 1 rows
// ahead of their use.  A warp owns 256 V neighbouring columns, vector i of a lane is
// columns 256 i + 8 lane of them: each warp copies its columns asynchronously into its
// own part of shared memory and reads them back itself, so no barrier of the block is
// needed, and all addresses within a row are one register and constants.  Places whose
// columns or array do not exist hold zeros, which add nothing to a sum: the arithmetic
// has no branches (with a branch a vector and 64-bit addresses the forward of 16384 x 4096
// with e4m3 took 87 us instead of 76, of 253 instructions a warp and vector 175 are left).  In fp32 a copy instruction covers 512 contiguous bytes, so a lane
// copies other pieces than it reads.  D = 0: loads at their use.
template <typename E, int N, int V, int D>
struct RowStream {
  static constexpr int W = Raw8<E>::W;
  static constexpr int WARP_BYTES = N * V * W * 512;       // of a row
  static constexpr int bytes(int threads) { return D * WARP_BYTES * (threads / 32); }
  const char* src[N];   // this warp's columns of the next row to be copied; null: absent
  int64_t step;         // from one of the block's rows to the next
  uint32_t ring;        // this warp's part
  int put, get;         // stages
  uint32_t copies;      // a bit for each piece of the arrays' rows that exists
  bool in[V];           // the lane's vectors exist
  uint32_t present;     // a bit for each array that exists

  // The rows at, at + each, ..; this warp's columns from `first` on.
  __device__ __forceinline__ void init(uint4* smem, const E* const (&p)[N], int H, int at, int each, int first) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t row = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      in[i] = first + i * 256 + lane * 8 < H;
#pragma unroll
      for (int w = 0; w < W; ++w)
        if (first + i * 256 + (w * 32 + lane) * (8 / W) < H) row |= 1u << (i * W + w);
    }
    copies = present = 0;
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (p[n]) present |= 1u << n, copies |= row << (n * V * W);
    const int own = D > 0 ? lane * 16 : lane * 16 * W;
#pragma unroll
    for (int n = 0; n < N; ++n)
      src[n] = p[n] ? reinterpret_cast<const char*>(p[n] + static_cast<int64_t>(at) * H + first) + own : nullptr;
    step = static_cast<int64_t>(each) * H * sizeof(E);
    put = get = 0;
    if (D > 0) {
      ring = smem_u32(smem) + warp * (D * WARP_BYTES);
      for (int i = lane * 16; i < D * WARP_BYTES; i += 512) st_shared_v4(ring + i, 0.f, 0.f, 0.f, 0.f);
      __syncwarp();
    }
  }
  // Copies of the block's next row, where there is one.
  __device__ __forceinline__ void issue(bool more) {
    if (D == 0) return;
    if (more) {
      const uint32_t dst = ring + put * WARP_BYTES + (threadIdx.x & 31) * 16;
#pragma unroll
      for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int i = 0; i < V * W; ++i)
          cp_async16_if(dst + (n * V * W + i) * 512, src[n] + i * 512, copies & (1u << (n * V * W + i)));
        src[n] += step;
      }
      put = put + 1 == D ? 0 : put + 1;
    }
    cp_async_commit();
  }
  // The oldest row's copies are there, and may be read.
  __device__ __forceinline__ void wait() const {
    if (D == 0) return;
    cp_async_wait<D >= 2 ? D - 2 : 0>();
    if (W > 1) __syncwarp();
  }
  __device__ __forceinline__ void take(int n, int i, Raw8<E>& r) const { take(n, i, r, get); }
  __device__ __forceinline__ void take(int n, int i, Raw8<E>& r, int stage) const {
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (D > 0) {
        const uint32_t at = ring + stage * WARP_BYTES + (n * V + i) * W * 512 + (threadIdx.x & 31) * (16 * W) + w * 16;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.u[w].x), "=r"(r.u[w].y), "=r"(r.u[w].z), "=r"(r.u[w].w) : "r"(at) : "memory");
      } else {
        r.u[w] = make_uint4(0u, 0u, 0u, 0u);
        if ((present >> n & 1) && in[i]) r.u[w] = *reinterpret_cast<const uint4*>(src[n] + i * 512 * W + w * 16);
      }
    }
  }
  // The row's arrays have been taken.
  __device__ __forceinline__ void next() {
    if (D > 0) {
      get = get + 1 == D ? 0 : get + 1;
    } else {
#pragma unroll
      for (int n = 0; n < N; ++n) src[n] += step;
    }
  }
};

// Rows of a block: k-th is blockIdx.x + k gridDim.x.
__device__ __forceinline__ int block_rows(int64_t T) {
  return static_cast<int>((T - blockIdx.x + gridDim.x - 1) / gridDim.x);
}

// A column's weights as fp32 pairs, ones where there are none.
template <typename E>
__device__ __forceinline__ void load_weights(const E* p, bool in, float2 (&w)[4]) {
  Raw8<E> r;
  r.ones();
  if (p && in) r.load(p);
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = r.pair(j);
}

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

template <typename E, int OUT, int V, int D, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 2 : 1) join_fwd_kernel(const JoinFwd a) {
  extern __shared__ uint4 ring_mem[];
  __shared__ float part[2][128];
  const int H = a.H, count = block_rows(a.T);
  RowStream<E, 2, V, D> rows;
  rows.init(ring_mem, {static_cast<const E*>(a.y), static_cast<const E*>(a.residual)}, H, blockIdx.x, gridDim.x,
            (threadIdx.x >> 5) * 256 * V);
#pragma unroll
  for (int d = 0; d < D - 1; ++d) rows.issue(d < count);
  const int lane = threadIdx.x & 31;
  const int c0 = (threadIdx.x >> 5) * 256 * V + lane * 8;     // of vector 0
  // the weights, and a row's terms between its two passes, in registers where these
  // allow (twice unpacked, a vector takes a third more instructions)
  constexpr bool KEEP = V == 1 || MAXT <= 512;
  constexpr int K = KEEP ? V : 1;
  float2 wp[K][4], w[K][4];
  auto weights = [&](int i) {
    const E* pw = static_cast<const E*>(a.post_weight);
    load_weights(pw ? pw + c0 + i * 256 : pw, rows.in[i], wp[KEEP ? i : 0]);
    if (OUT != kNoNorm) load_weights(static_cast<const E*>(a.weight) + c0 + i * 256, rows.in[i], w[KEEP ? i : 0]);
  };
  if (KEEP)
#pragma unroll
    for (int i = 0; i < V; ++i) weights(i);
  const float inv_H = 1.f / static_cast<float>(H);
  const float2 scale2 = make_float2(a.scale, a.scale);
  const int64_t at0 = static_cast<int64_t>(blockIdx.x) * H + c0;
  E* total = static_cast<E*>(a.total) + at0;
  char* n_out = OUT == kNoNorm ? nullptr : static_cast<char*>(a.n) + at0 * (OUT == kE4m3 ? 1 : sizeof(E));
  uint8_t* s_out = OUT == kE4m3 ? a.n_scale + at0 / 32 : nullptr;
  float gates = 1.f;      // of 32 rows, one per lane (a load per row would wait for the rows' copies)
  for (int row = 0; row < count; ++row) {
    const int flip = row & 1;      // a row's barrier also separates the reuse of the other sums
    if (a.gate && (row & 31) == 0 && row + lane < count)
      gates = __ldg(a.gate + blockIdx.x + static_cast<int64_t>(row + lane) * gridDim.x);
    const float gate = __shfl_sync(0xffffffffu, gates, row & 31);
    rows.wait();
    rows.issue(row + D - 1 < count);
    // total = t + f q with t = scale * residual, q = y * post_weight, f = gate * rs_y
    Raw8<E> ry[V], rr[V];
    float2 t[K][4], q[K][4];
    auto terms = [&](int i) {
      const int k = KEEP ? i : 0;
      if (!KEEP) weights(i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        t[k][j] = __fmul2_rn(scale2, rr[i].pair(j));
        q[k][j] = __fmul2_rn(ry[i].pair(j), wp[k][j]);
      }
    };
    float2 yy = make_float2(0.f, 0.f), tt = yy, tq = yy, qq = yy;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = KEEP ? i : 0;
      rows.take(0, i, ry[i]);
      rows.take(1, i, rr[i]);
      terms(i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 y = ry[i].pair(j);
        yy = __ffma2_rn(y, y, yy);
        if (OUT != kNoNorm) {
          tt = __ffma2_rn(t[k][j], t[k][j], tt);
          tq = __ffma2_rn(t[k][j], q[k][j], tq);
          qq = __ffma2_rn(q[k][j], q[k][j], qq);
        }
      }
    }
    rows.next();
    float4 s = make_float4(yy.x + yy.y, tt.x + tt.y, tq.x + tq.y, qq.x + qq.y);
    if (OUT != kNoNorm)
      s = block_sum4<MAXT>(s, part[flip]);
    else if (a.post_norm)
      s.x = block_sum(s.x, part[flip]);
    const float rs_y = a.post_norm ? rsqrtf(s.x * inv_H + a.eps) : 1.f;
    const float f = gate * rs_y;
    const float2 f2 = make_float2(f, f);
    // the sum of total^2 from those of its terms, unless they cancel (or leave fp32's
    // range): then once more from total
    float ss = 0.f;
    if (OUT != kNoNorm) {
      const float terms2 = s.y + f * f * s.w;
      ss = terms2 + 2.f * f * s.z;
      if (!(ss >= 0.25f * terms2 && ss < INFINITY)) {
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (!KEEP) terms(i);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 r = __ffma2_rn(f2, q[KEEP ? i : 0][j], t[KEEP ? i : 0][j]);
            if (rows.in[i]) ss = fmaf(r.x, r.x, fmaf(r.y, r.y, ss));     // (an infinite f makes NaN of zeros)
          }
        }
        __syncthreads();      // all have read `part`
        ss = block_sum(ss, part[flip]);
      }
    }
    const float rs = rsqrtf(ss * inv_H + a.eps);
    if (threadIdx.x == 0) {
      const int64_t r = blockIdx.x + static_cast<int64_t>(row) * gridDim.x;
      if (a.rstd_post) a.rstd_post[r] = rs_y;
      if (OUT != kNoNorm && a.rstd) a.rstd[r] = rs;
    }
    const float2 rs2 = make_float2(rs, rs);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = KEEP ? i : 0;
      if (!KEEP) terms(i);
      float2 r[4], n[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[j] = __ffma2_rn(f2, q[k][j], t[k][j]);
        if (OUT != kNoNorm) n[j] = __fmul2_rn(__fmul2_rn(r[j], rs2), w[k][j]);
      }
      store8_if(total + i * 256, r, rows.in[i]);
      if (OUT == kSameType) store8_if(reinterpret_cast<E*>(n_out) + i * 256, n, rows.in[i]);
      if (OUT == kE4m3) store_e4m3(n, rows.in[i], reinterpret_cast<uint8_t*>(n_out) + i * 256, s_out + i * 8);
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * H;
    total += step;
    if (OUT != kNoNorm) n_out += step * (OUT == kE4m3 ? 1 : sizeof(E));
    if (OUT == kE4m3) s_out += step / 32;
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
template <typename E, bool NEXT, int V, int D, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 384 ? 2 : 1) join_bwd_kernel(const JoinBwd a) {
  extern __shared__ uint4 ring_mem[];
  __shared__ float part[2][128];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int N = NEXT ? 4 : 2;
  const int H = a.H, count = block_rows(a.T);
  RowStream<E, N, V, D> rows;
  {
    const E* p[N] = {static_cast<const E*>(a.y), static_cast<const E*>(a.d_total)};
    if (NEXT) p[N - 2] = static_cast<const E*>(a.dn), p[N - 1] = static_cast<const E*>(a.total);
    rows.init(ring_mem, p, H, blockIdx.x, gridDim.x, (threadIdx.x >> 5) * 256 * V);
  }
#pragma unroll
  for (int d = 0; d < D - 1; ++d) rows.issue(d < count);
  const int lane = threadIdx.x & 31;
  const int c0 = (threadIdx.x >> 5) * 256 * V + lane * 8;     // of vector 0
  // the weights, and a row's terms between its two passes, in registers where these allow
  // (with two vectors the weights are packed and the row is read from the ring again: with
  // all of it in registers or the weights loaded in each pass, 8192 x 5152 112 us, not 91)
  constexpr bool KEEP = V == 1, AGAIN = !KEEP && D > 0;
  float2 wp[1][4], w[1][4];
  Raw8<E> wp_raw[V], w_raw[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    wp_raw[i].ones(), w_raw[i].ones();
    if (a.post_weight && rows.in[i]) wp_raw[i].load(static_cast<const E*>(a.post_weight) + c0 + i * 256);
    if (NEXT && rows.in[i]) w_raw[i].load(static_cast<const E*>(a.weight) + c0 + i * 256);
  }
  auto weights = [&](int i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) wp[0][j] = wp_raw[i].pair(j), w[0][j] = w_raw[i].pair(j);
  };
  if (KEEP) weights(0);
  float2 dw[NEXT ? V : 1][4], dwp[V][4];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) dwp[i][j] = dw[NEXT ? i : 0][j] = make_float2(0.f, 0.f);
  const float inv_H = 1.f / static_cast<float>(H);
  const int64_t at0 = static_cast<int64_t>(blockIdx.x) * H + c0;
  E *dy = static_cast<E*>(a.dy) + at0, *d_residual = static_cast<E*>(a.d_residual) + at0;
  const float2 scale2 = make_float2(a.scale, a.scale);
  // 1 / rms and gate of 32 rows, one per lane (a load per row would wait for the
  // rows' copies)
  float rstds = 0.f, posts = 1.f, gates = 1.f;
  for (int row = 0; row < count; ++row) {
    const int flip = row & 1;
    if ((row & 31) == 0 && row + lane < count) {
      const int64_t mine = blockIdx.x + static_cast<int64_t>(row + lane) * gridDim.x;
      if (NEXT) rstds = __ldg(a.rstd + mine);
      if (a.rstd_post) posts = __ldg(a.rstd_post + mine);
      if (a.gate) gates = __ldg(a.gate + mine);
    }
    const float rs = NEXT ? __shfl_sync(0xffffffffu, rstds, row & 31) : 0.f;
    const float rs_y = __shfl_sync(0xffffffffu, posts, row & 31);
    const float gate = __shfl_sync(0xffffffffu, gates, row & 31);
    rows.wait();
    rows.issue(row + D - 1 < count);
    const float2 rs2 = make_float2(rs, rs), rs_y2 = make_float2(rs_y, rs_y);
    constexpr int R = AGAIN ? 1 : V;
    Raw8<E> ry[R], rt[R], rn[NEXT ? R : 1], rr[NEXT ? R : 1];
    auto take = [&](int i) {
      const int r = AGAIN ? 0 : i, k = NEXT ? r : 0;
      rows.take(0, i, ry[r]);
      rows.take(1, i, rt[r]);
      if (NEXT) {
        rows.take(N - 2, i, rn[k]);
        rows.take(N - 1, i, rr[k]);
      }
    };
    float2 u[4], rhat[4], yhat[4];
    // u = d_total + rs dn weight, rhat, yhat of vector i
    auto terms = [&](int i) {
      const int r = AGAIN ? 0 : i, k = NEXT ? r : 0;
      if (!KEEP) weights(i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        yhat[j] = __fmul2_rn(ry[r].pair(j), rs_y2);
        u[j] = rt[r].pair(j);
        if (NEXT) {
          rhat[j] = __fmul2_rn(rr[k].pair(j), rs2);
          u[j] = __ffma2_rn(rs2, __fmul2_rn(rn[k].pair(j), w[0][j]), u[j]);
        }
      }
    };
    float2 s1 = make_float2(0.f, 0.f), s2 = s1, s3 = s1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = NEXT && !AGAIN ? i : 0;
      take(i);
      terms(i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 q = __fmul2_rn(yhat[j], wp[0][j]);
        if (NEXT) {
          const float2 g = __fmul2_rn(rn[k].pair(j), rhat[j]);
          s1 = __ffma2_rn(g, w[0][j], s1);
          s3 = __ffma2_rn(rhat[j], q, s3);
          dw[i][j] = __ffma2_rn(rn[k].pair(j), rhat[j], dw[i][j]);
        }
        s2 = __ffma2_rn(u[j], q, s2);
      }
    }
    if (!AGAIN) rows.next();
    float m = 0.f, dot;
    if (NEXT) {
      const float4 s = block_sum4<MAXT>(make_float4(s1.x + s1.y, s2.x + s2.y, s3.x + s3.y, 0.f), part[flip]);
      m = rs * s.x * inv_H;
      dot = fmaf(-m, s.z, s.y);
    } else {
      dot = block_sum(s2.x + s2.y, part[flip]);
    }
    if (a.d_gate && threadIdx.x == 0) a.d_gate[blockIdx.x + static_cast<int64_t>(row) * gridDim.x] = dot;
    const float back = a.rstd_post ? -gate * dot * inv_H : 0.f;
    const float2 m2 = make_float2(-m, -m), gate2 = make_float2(gate, gate), back2 = make_float2(back, back);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (AGAIN) take(i);
      if (!KEEP) terms(i);
      float2 oy[4], od[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 dr = NEXT ? __ffma2_rn(m2, rhat[j], u[j]) : u[j];
        od[j] = __fmul2_rn(scale2, dr);
        const float2 dp = __fmul2_rn(gate2, dr);
        dwp[i][j] = __ffma2_rn(dp, yhat[j], dwp[i][j]);
        oy[j] = __fmul2_rn(rs_y2, __ffma2_rn(back2, yhat[j], __fmul2_rn(dp, wp[0][j])));
      }
      store8_if(dy + i * 256, oy, rows.in[i]);
      store8_if(d_residual + i * 256, od, rows.in[i]);
    }
    if (AGAIN) rows.next();
    const int64_t step = static_cast<int64_t>(gridDim.x) * H;
    dy += step, d_residual += step;
  }
  if (a.part) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (rows.in[i]) {
        const int64_t at = static_cast<int64_t>(blockIdx.x) * H + c0 + i * 256;
        if (NEXT) store8(a.part + at, &dw[NEXT ? i : 0][0].x);
        store8(a.part + static_cast<int64_t>(gridDim.x) * H + at, &dwp[i][0].x);
      }
  }
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The same for wide rows: a cluster of `ranks` CTAs takes a row, 512 columns a warp, and a
// row's second pass comes after the next one's first: what the warps' sums take through
// the cluster is then hidden, and a row stays in the ring until its second pass, so only
// the weights and their sums are kept in registers.  (One CTA with four vectors a thread
// spills and has no room for a ring: 4096 x 16384 bf16 275 us instead of 165, 1024 x 32768
// fp32 592 instead of 192.)  Each warp sends its sums to all CTAs; one that is a row ahead
// of another has passed the barrier before, so four rows' sums have to have room.
template <typename E, bool NEXT>
__global__ void __launch_bounds__(512, 1) join_bwd_wide_kernel(const JoinBwd a, int ranks) {
  constexpr int V = 2, N = NEXT ? 4 : 2;
  extern __shared__ uint4 ring_mem[];
  __shared__ float part[4][256];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, rank = cluster_ctarank();
  const int H = a.H, first_row = blockIdx.x / ranks, clusters = gridDim.x / ranks;
  const int count = static_cast<int>((a.T - first_row + clusters - 1) / clusters);
  const int first = (rank * warps + warp) * 256 * V, c0 = first + lane * 8;     // of vector 0
  RowStream<E, N, V, kAhead> rows;
  {
    const E* p[N] = {static_cast<const E*>(a.y), static_cast<const E*>(a.d_total)};
    if (NEXT) p[N - 2] = static_cast<const E*>(a.dn), p[N - 1] = static_cast<const E*>(a.total);
    rows.init(ring_mem, p, H, first_row, clusters, first);
  }
  rows.issue(true);
  rows.issue(count > 1);
  // lane l sends sum l & 3 to rank l >> 2
  const uint32_t send = mapa_shared(smem_u32(part) + ((rank * warps + warp) * 4 + (lane & 3)) * 4, (lane >> 2) % ranks);
  cluster_sync();      // the others' shared memory is there
  Raw8<E> wp[V], w[V];      // (packed; loaded again in each pass, a row waits for them: 4096 x 16384 179 us)
#pragma unroll
  for (int i = 0; i < V; ++i) {
    wp[i].ones(), w[i].ones();
    if (a.post_weight && rows.in[i]) wp[i].load(static_cast<const E*>(a.post_weight) + c0 + i * 256);
    if (NEXT && rows.in[i]) w[i].load(static_cast<const E*>(a.weight) + c0 + i * 256);
  }
  float2 dw[NEXT ? V : 1][4], dwp[V][4];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) dwp[i][j] = dw[NEXT ? i : 0][j] = make_float2(0.f, 0.f);
  const float inv_H = 1.f / static_cast<float>(H);
  const int64_t at0 = static_cast<int64_t>(first_row) * H + c0;
  E *dy = static_cast<E*>(a.dy) + at0, *d_residual = static_cast<E*>(a.d_residual) + at0;
  const float2 scale2 = make_float2(a.scale, a.scale);
  float rstds = 0.f, posts = 1.f, gates = 1.f;      // of 32 rows, one per lane
  float rs = 0.f, rs_y = 1.f, gate = 1.f;           // of the row of the first pass
  float2 u[4], rhat[4], yhat[4];
  Raw8<E> rn;
  // u = d_total + rs dn weight, rhat, yhat of vector i
  auto terms = [&](int i, int stage, float r, float ry) {
    const float2 r2 = make_float2(r, r), ry2 = make_float2(ry, ry);
    Raw8<E> x, t, rr;
    rows.take(0, i, x, stage);
    rows.take(1, i, t, stage);
    if (NEXT) {
      rows.take(N - 2, i, rn, stage);
      rows.take(N - 1, i, rr, stage);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      yhat[j] = __fmul2_rn(x.pair(j), ry2);
      u[j] = t.pair(j);
      if (NEXT) {
        rhat[j] = __fmul2_rn(rr.pair(j), r2);
        u[j] = __ffma2_rn(r2, __fmul2_rn(rn.pair(j), w[i].pair(j)), u[j]);
      }
    }
  };
  // a row's sums, on their way to all CTAs
  auto first_pass = [&](int row, int stage) {
    if ((row & 31) == 0 && row + lane < count) {
      const int64_t mine = first_row + static_cast<int64_t>(row + lane) * clusters;
      if (NEXT) rstds = __ldg(a.rstd + mine);
      if (a.rstd_post) posts = __ldg(a.rstd_post + mine);
      if (a.gate) gates = __ldg(a.gate + mine);
    }
    rs = NEXT ? __shfl_sync(0xffffffffu, rstds, row & 31) : 0.f;
    rs_y = __shfl_sync(0xffffffffu, posts, row & 31);
    gate = __shfl_sync(0xffffffffu, gates, row & 31);
    rows.wait();
    float2 s1 = make_float2(0.f, 0.f), s2 = s1, s3 = s1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      terms(i, stage, rs, rs_y);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 q = __fmul2_rn(yhat[j], wp[i].pair(j));
        if (NEXT) {
          s1 = __ffma2_rn(__fmul2_rn(rn.pair(j), rhat[j]), w[i].pair(j), s1);
          s3 = __ffma2_rn(rhat[j], q, s3);
          dw[i][j] = __ffma2_rn(rn.pair(j), rhat[j], dw[i][j]);
        }
        s2 = __ffma2_rn(u[j], q, s2);
      }
    }
    const float s = warp_sum4(make_float4(s1.x + s1.y, s2.x + s2.y, s3.x + s3.y, 0.f));
    if (lane < 4 * ranks)
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(send + (row & 3) * 1024), "f"(s) : "memory");
    __syncwarp();
  };
  first_pass(0, 0);
  cluster_arrive();
  int stage = 0;
  for (int row = 0; row < count; ++row) {
    const bool more = row + 1 < count;
    const float rs_0 = rs, rs_y_0 = rs_y, gate_0 = gate;
    const int next = stage + 1 == kAhead ? 0 : stage + 1;
    __syncwarp();      // all lanes have done with the row that is overwritten
    rows.issue(row + 2 < count);
    if (more) first_pass(row + 1, next);
    cluster_wait();
    if (more) cluster_arrive();
    float s = 0.f;
    for (int i = lane; i < ranks * warps * 4; i += 32) s += part[row & 3][i];
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const float sum1 = __shfl_sync(0xffffffffu, s, 0), sum2 = __shfl_sync(0xffffffffu, s, 2), sum3 = __shfl_sync(0xffffffffu, s, 1);
    const float m = NEXT ? rs_0 * sum1 * inv_H : 0.f, dot = NEXT ? fmaf(-m, sum3, sum2) : sum2;
    if (a.d_gate && rank == 0 && threadIdx.x == 0) a.d_gate[first_row + static_cast<int64_t>(row) * clusters] = dot;
    const float back = a.rstd_post ? -gate_0 * dot * inv_H : 0.f;
    const float2 m2 = make_float2(-m, -m), gate2 = make_float2(gate_0, gate_0), back2 = make_float2(back, back);
    const float2 rs_y2 = make_float2(rs_y_0, rs_y_0);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      terms(i, stage, rs_0, rs_y_0);
      float2 oy[4], od[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 dr = NEXT ? __ffma2_rn(m2, rhat[j], u[j]) : u[j];
        od[j] = __fmul2_rn(scale2, dr);
        const float2 dp = __fmul2_rn(gate2, dr);
        dwp[i][j] = __ffma2_rn(dp, yhat[j], dwp[i][j]);
        oy[j] = __fmul2_rn(rs_y2, __ffma2_rn(back2, yhat[j], __fmul2_rn(dp, wp[i].pair(j))));
      }
      store8_if(dy + i * 256, oy, rows.in[i]);
      store8_if(d_residual + i * 256, od, rows.in[i]);
    }
    const int64_t step = static_cast<int64_t>(clusters) * H;
    dy += step, d_residual += step;
    stage = next;
  }
  if (a.part) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (rows.in[i]) {
        const int64_t at = static_cast<int64_t>(first_row) * H + c0 + i * 256;
        if (NEXT) store8(a.part + at, &dw[NEXT ? i : 0][0].x);
        store8(a.part + static_cast<int64_t>(clusters) * H + at, &dwp[i][0].x);
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

// Threads of a launch's resident blocks per SM, where one block does not have more: fewer
// threads with more registers beat more threads (forward of 16384 x 4096 with e4m3: 512
// threads 76 us, 768 of at most 85 registers 124; backward of 16384 x 4096: 768 threads
// 125 us, 1024 130, of 32768 x 1024 74 and 82).
constexpr int kFwdThreads = 512;
constexpr int kBwdThreads = 768;

// Threads of v vectors each, and blocks.  The ring needs a few rows per block to pay.
struct JoinLaunch {
  int threads, blocks, smem;
};
JoinLaunch join_launch(int64_t T, int H, int v, int ring_per_warp, int threads_per_sm, int most, int sms) {
  JoinLaunch l;
  const int warps = (H + 256 * v - 1) / (256 * v);
  l.threads = 32 * warps;
  l.smem = ring_per_warp * warps;
  const int per_sm = std::min({l.smem <= kRingPerSm ? kRingPerSm / l.smem : 0, std::max(1, threads_per_sm / l.threads), most});
  l.blocks = l.threads > 1024 ? 0 : static_cast<int>(std::min<int64_t>(T, static_cast<int64_t>(sms) * per_sm));
  return l;
}

template <typename E, int OUT, int V, int MAXT>
cudaError_t launch_join_ring(const JoinFwd& a, const JoinLaunch& l, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(join_fwd_kernel<E, OUT, V, kAhead, MAXT>, ready);
  if (e != cudaSuccess) return e;
  join_fwd_kernel<E, OUT, V, kAhead, MAXT><<<l.blocks, l.threads, l.smem, st>>>(a);
  return cudaGetLastError();
}

template <typename E, int OUT>
cudaError_t launch_join_fwd(const JoinFwd& a, int sms, cudaStream_t st) {
  // two vectors per thread halve what a row costs beside its columns (16384 x 4096 with
  // e4m3: 147 us with one), four run out of registers (109)
  const int v = a.H <= 512 ? 1 : 2;
  const bool small = a.H <= 256 * 8 * v, wide = a.H <= 256 * 16 * v;      // at most 256 threads, more registers for each
  const JoinLaunch l = join_launch(a.T, a.H, v, RowStream<E, 2, 1, kAhead>::bytes(32) * v, small ? kFwdThreads : 1024, 24, sms);
  if (l.blocks > 0 && a.T > l.blocks) {
    if (v == 1) return launch_join_ring<E, OUT, 1, 256>(a, l, st);
    if (small) return launch_join_ring<E, OUT, 2, 256>(a, l, st);
    if (wide) return launch_join_ring<E, OUT, 2, 512>(a, l, st);
    return launch_join_ring<E, OUT, 2, 1024>(a, l, st);
  }
  // few rows: a block for each, as many threads as there are
  const unsigned T = static_cast<unsigned>(a.T);
  const int warps = (a.H + 255) / 256;
  if (warps <= 32)
    join_fwd_kernel<E, OUT, 1, 0, 1024><<<T, 32 * warps, 0, st>>>(a);
  else if (warps <= 64)
    join_fwd_kernel<E, OUT, 2, 0, 1024><<<T, 32 * ((warps + 1) / 2), 0, st>>>(a);
  else
    join_fwd_kernel<E, OUT, 4, 0, 1024><<<T, 32 * ((warps + 3) / 4), 0, st>>>(a);
  return cudaGetLastError();
}

// *blocks: of the launch, each of which leaves its sums in a.part.  WARPS: the fewest of
// a block; where their ring does not fit, there is none.
template <typename E, bool NEXT, int V, int MAXT, int WARPS>
cudaError_t launch_join_bwd_v(const JoinBwd& a, int sms, int* blocks, cudaStream_t st) {
  using Rows = RowStream<E, NEXT ? 4 : 2, V, kAhead>;
  JoinLaunch l = join_launch(a.T, a.H, V, Rows::bytes(32), kBwdThreads, 8, sms);
  if constexpr (Rows::bytes(32 * WARPS) <= kRingPerSm) {
    if (l.blocks > 0 && a.T > l.blocks) {
      static std::atomic<uint64_t> ready{0};
      const cudaError_t e = allow_smem(join_bwd_kernel<E, NEXT, V, kAhead, MAXT>, ready);
      if (e != cudaSuccess) return e;
      join_bwd_kernel<E, NEXT, V, kAhead, MAXT><<<l.blocks, l.threads, l.smem, st>>>(a);
      *blocks = l.blocks;
      return cudaGetLastError();
    }
  }
  const int per_sm = std::max(1, std::min(8, 1024 / l.threads));
  *blocks = static_cast<int>(std::min<int64_t>(a.T, static_cast<int64_t>(sms) * per_sm));
  join_bwd_kernel<E, NEXT, V, 0, MAXT><<<*blocks, l.threads, 0, st>>>(a);
  return cudaGetLastError();
}

// The same for wide rows: as few CTAs a row as fit an SM by twos, or by ones where eight do
// not suffice.
template <typename E, bool NEXT>
cudaError_t launch_join_bwd_wide(const JoinBwd& a, int sms, int* blocks, cudaStream_t st) {
  constexpr int kWarpBytes = RowStream<E, NEXT ? 4 : 2, 2, kAhead>::bytes(32);
  constexpr int kTwo = std::min(8, kRingPerSm / 2 / kWarpBytes), kOne = std::min(16, kRingPerSm / kWarpBytes);
  auto kern = join_bwd_wide_kernel<E, NEXT>;
  int ranks = 1, log = 0;
  const int most = a.H <= 8 * kTwo * 512 ? kTwo : kOne;
  while ((a.H + 512 * ranks - 1) / (512 * ranks) > most) ranks *= 2, ++log;
  const int warps = (a.H + 512 * ranks - 1) / (512 * ranks);
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(kern, ready);
  if (e != cudaSuccess) return e;
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = st;
  // the clusters that fit the device at once, asked for once per device and shape
  cfg.blockDim = dim3(32 * warps);
  cfg.dynamicSmemBytes = warps * kWarpBytes;
  static std::atomic<int> known[64][4][17];
  int fit = known[dev & 63][log][warps].load(std::memory_order_relaxed);
  if (fit == 0) {
    cfg.gridDim = dim3(8 * sms >> log << log);
    e = cudaOccupancyMaxActiveClusters(&fit, kern, &cfg);
    if (e != cudaSuccess) return e;
    if (fit < 1) return cudaErrorLaunchOutOfResources;
    known[dev & 63][log][warps].store(fit, std::memory_order_relaxed);
  }
  *blocks = static_cast<int>(std::min<int64_t>(a.T, std::min(fit, kMaxBwdBlocks)));
  cfg.gridDim = dim3(*blocks * ranks);
  return cudaLaunchKernelEx(&cfg, kern, a, ranks);
}

template <typename E, bool NEXT>
cudaError_t launch_join_bwd(const JoinBwd& a, int sms, int* blocks, cudaStream_t st) {
  const int warps = (a.H + 255) / 256;
  // one vector per thread up to 4096 columns; more than 80 registers where one block
  // per SM is all that the ring or the threads leave room for (8192 x 2880 fp32: 93 us
  // with up to 128 registers, 109 with 80; bf16, two blocks: 57 and 52)
  if (warps <= (sizeof(E) == 4 ? 8 : 12)) return launch_join_bwd_v<E, NEXT, 1, 384, 1>(a, sms, blocks, st);
  if (warps <= 16) return launch_join_bwd_v<E, NEXT, 1, 512, 9>(a, sms, blocks, st);
  // two up to 8192 in bf16 (8192 x 8192: 145 us, on clusters 161; 4096 x 8192 fp32, whose
  // ring does not fit: 198 and 154)
  if constexpr (sizeof(E) == 2)
    if (warps <= 32) return launch_join_bwd_v<E, NEXT, 2, 512, 9>(a, sms, blocks, st);
  return launch_join_bwd_wide<E, NEXT>(a, sms, blocks, st);
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
  if ((post_norm != 0 && post_norm != 1) || (n_scale && H % 32)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if ((n_scale && !n) || (!n != !weight) || (rstd_post && !post_norm) || (rstd && !n))
    return MOE_ERR_INVALID_ARG;
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
