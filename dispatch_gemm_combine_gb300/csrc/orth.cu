// Orthogonal weight updates by Newton-Schulz products, for each matrix g [M,N] of a
// batch:
//
//   x_0 = g / (|g|_F + eps),   a = x x^T,   x <- (c0 + c1 a + c2 a^2) x,
//   out = scale * x.
//
// The iteration works on the narrower side (m = min(M, N) rows; a tall g is
// transposed as it is read, and the result as it is written).  A step is three
// products on the tensor cores, in fp16 with fp32 accumulation:
//   gram    A  = X X^T            (m x m, symmetric)
//   poly    B  = c0 I + c1 A + c2 A A   (symmetric)
//   update  X' = B X              (m x n)
// so the sum over the step's terms happens in fp32 before B is rounded, and x's own
// term needs no second read of x.  The symmetric products compute the tiles on and
// above the diagonal and store the others mirrored: m^2 n + m^3 + 2 m^2 n operations
// a step instead of 2 m^2 n + 2 m^3 + 2 m^2 n.
//
// fp16 (11 bits) and not bf16 (8 bits): singular values far below the largest grow by
// up to c0 per step, and with them what the roundings left there; with bf16 operands
// the result of a Gaussian g is 1e-2 off, with fp16 1.1e-3 (the bf16 output's own
// rounding: 1.7e-3).  fp16's range is kept by powers of two: X holds S x and A and B
// hold S^2 times theirs, S near sqrt(max(M, N)), so that typical values are far from
// both ends; the coefficients' bounds (checked on the host) keep the largest below
// 60000.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "abi_internal.h"
#include "common.cuh"
#include "vec.cuh"

namespace moe {
namespace {

// ------------------------------------------------------------ norm and load
constexpr int kNormThreads = 256;
constexpr int kNormElems = 32768;      // of a matrix per block of the norm
constexpr int kMaxParts = 1024;         // blocks per matrix

// Squares of fp32 values leave fp32's range beyond 2^64 and below 2^-63: sums of
// g^2, (2^-80 g)^2 and (2^80 g)^2 side by side, of which the one in range is taken.
struct Squares {
  float mid = 0.f, big = 0.f, small = 0.f;
  __device__ __forceinline__ void add(float v) {
    mid = fmaf(v, v, mid);
    const float b = v * 0x1p-80f, s = v * 0x1p80f;
    big = fmaf(b, b, big);
    small = fmaf(s, s, small);
  }
};

struct OrthIn {
  const void* g;
  int64_t ld, stride;   // of rows and matrices
  int M, N;
  int bf16;
  int vec;              // rows start on 16 bytes
};

template <typename E>
__device__ __forceinline__ float elem(const void* g, int64_t i) {
  return to_f32(static_cast<const E*>(g)[i]);
}

// Sums of squares of rows [r0, r1) of matrix blockIdx.y.
template <typename E>
__device__ __forceinline__ void add_rows(const OrthIn& in, int64_t base, int r0, int r1, Squares& s) {
  constexpr int W = 16 / sizeof(E);
  const int nv = in.vec ? in.N / W : 0;   // whole vectors of a row
  const int tail = in.N - nv * W;
  const E* g = static_cast<const E*>(in.g);
  const int64_t vecs = static_cast<int64_t>(r1 - r0) * nv;
  for (int64_t i = threadIdx.x; i < vecs; i += kNormThreads) {
    const int r = static_cast<int>(i / nv), c = static_cast<int>(i - static_cast<int64_t>(r) * nv);
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(g + base + (r0 + r) * in.ld) + c);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (sizeof(E) == 4) {
        s.add(__uint_as_float(w[k]));
      } else {
        s.add(bf16_lo(w[k]));
        s.add(bf16_hi(w[k]));
      }
    }
  }
  const int64_t rest = static_cast<int64_t>(r1 - r0) * tail;
  for (int64_t i = threadIdx.x; i < rest; i += kNormThreads) {
    const int r = static_cast<int>(i / tail), c = nv * W + static_cast<int>(i - static_cast<int64_t>(r) * tail);
    s.add(elem<E>(in.g, base + (r0 + r) * in.ld + c));
  }
}

__global__ void __launch_bounds__(kNormThreads) orth_norm_kernel(const OrthIn in, int rows, Squares* parts) {
  __shared__ float part[3][32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t base = static_cast<int64_t>(blockIdx.y) * in.stride;
  const int r0 = blockIdx.x * rows, r1 = min(in.M, r0 + rows);
  Squares s;
  if (in.bf16)
    add_rows<__nv_bfloat16>(in, base, r0, r1, s);
  else
    add_rows<float>(in, base, r0, r1, s);
  s.mid = block_sum(s.mid, part[0]);
  s.big = block_sum(s.big, part[1]);
  s.small = block_sum(s.small, part[2]);
  if (threadIdx.x == 0) parts[static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = s;
}

// The factors (pre, f) with x_0 S = (g pre) f, of the matrix's parts: the same in
// every thread.
__device__ __forceinline__ float2 orth_factor(const Squares* parts, int n, float eps, float S) {
  __shared__ float part[3][32];
  Squares v;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const float* p = &parts[i].mid;
    v.mid += __ldcg(p), v.big += __ldcg(p + 1), v.small += __ldcg(p + 2);
  }
  v.mid = block_sum(v.mid, part[0]);
  v.big = block_sum(v.big, part[1]);
  v.small = block_sum(v.small, part[2]);
  float pre = 1.f, ss = v.mid;
  if (!isfinite(v.mid))
    pre = 0x1p-80f, ss = v.big;
  else if (v.mid < 0x1p-40f)
    pre = 0x1p80f, ss = v.small;
  const float norm = sqrtf(ss) + eps * pre;
  // a matrix of zeros stays zero without eps too; one that holds an infinity or a NaN
  // is NaN throughout
  const float f = norm == 0.f ? 0.f : (isfinite(norm) ? S / norm : __int_as_float(0x7fc00000));
  return make_float2(pre, f);
}

// X [m, ldx] fp16 from g: a block takes a tile of 64 x 64 (64 rows of the result).
template <typename E, bool FLIP>
__global__ void __launch_bounds__(256) orth_load_kernel(const OrthIn in, const Squares* parts, int nparts, float eps,
                                                        float S, __half* X, int ldx, int64_t xstride) {
  __shared__ float tile[64][65];
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the sums are there
  const int e = blockIdx.z;
  const float2 f = orth_factor(parts + static_cast<int64_t>(e) * nparts, nparts, eps, S);
  const int64_t base = static_cast<int64_t>(e) * in.stride;
  const int c0 = blockIdx.x * 64, r0 = blockIdx.y * 64;   // of g
  const int lc = threadIdx.x & 63, lr = threadIdx.x >> 6;
  for (int i = lr; i < 64; i += 4) {
    const int r = r0 + i, c = c0 + lc;
    float v = 0.f;
    if (r < in.M && c < in.N) v = elem<E>(in.g, base + r * in.ld + c) * f.x * f.y;
    tile[i][lc] = v;
  }
  __syncthreads();
  __half* x = X + static_cast<int64_t>(e) * xstride;
  const int rows = FLIP ? in.N : in.M;
  const int xr0 = FLIP ? c0 : r0, xc0 = FLIP ? r0 : c0;
  const int xc = (threadIdx.x & 31) * 2;
  for (int i = threadIdx.x >> 5; i < 64; i += 8) {
    const float a = FLIP ? tile[xc][i] : tile[i][xc];
    const float b = FLIP ? tile[xc + 1][i] : tile[i][xc + 1];
    // columns up to ldx (a multiple of 8) are in the buffer; those past the matrix hold 0
    if (xr0 + i < rows && xc0 + xc < ldx)
      *reinterpret_cast<__half2*>(x + static_cast<int64_t>(xr0 + i) * ldx + xc0 + xc) = __floats2half2_rn(a, b);
  }
}

// ------------------------------------------------------------ products
// A persistent batched product D = A B^T on CTA pairs (2-SM MMA, M = 256, N = 256):
// each CTA loads 128 rows of A and 128 of B per 64 columns of K into a ring, one
// thread of the even CTA issues the MMAs, the accumulators are double-buffered in
// tensor memory and four warps per CTA store them.  Warp roles and unwinding as in
// the expert layer's grouped products.
enum OrthMode : int { kGram = 0, kPoly = 1, kUpdate = 2 };

constexpr int kOrthStages = 6;
constexpr int kStageBytes = 2 * 128 * 128;
constexpr int kEpiWarpBytes = 2 * 4096;
constexpr int kOrthBars = (2 * kOrthStages + 5) * 8 + 16;
constexpr int kOrthSmem = 1024 + kOrthStages * kStageBytes + 4 * kEpiWarpBytes + kOrthBars;
static_assert(kOrthSmem <= 232448, "shared memory budget");

struct OrthMaps {
  CUtensorMap a, b;        // operands
  CUtensorMap out, out_t;  // fp16 result: boxes {64 columns, 32 rows}, mirrored {32, 64}
};

struct OrthArgs {
  int m, n;              // of the result
  int num_kb;            // blocks of 64 of the contraction
  int batch;
  int mt, nt;            // tiles of 256
  float ds;              // factor on the accumulator
  float cA, cI;          // poly: factor on A, addend on the diagonal
  const __half* A;       // poly: A [batch][m][lda]
  int lda;
  int64_t astride;
  // the last update: bf16 out[e][r][c], transposed when `flip`
  __nv_bfloat16* out;
  int64_t out_ld, out_stride;
  int flip, vec;         // vec: rows of out start on 16 bytes
  int* err;
  uint64_t timeout_ns;
};

struct OrthTile {
  int e, i, j;
};

// Unit t: matrix, row tile, column tile; symmetric results have the column tiles
// from the diagonal on only.
template <int MODE>
__device__ __forceinline__ OrthTile orth_tile(const OrthArgs& a, int t) {
  OrthTile r;
  if (MODE == kUpdate) {
    const int per = a.mt * a.nt;
    r.e = t / per;
    const int u = t - r.e * per;
    r.j = u / a.mt;
    r.i = u - r.j * a.mt;
  } else {
    const int per = a.mt * (a.mt + 1) / 2;
    r.e = t / per;
    int u = t - r.e * per;
    // row i has mt - i tiles
    int i = 0;
    while (u >= a.mt - i) {
      u -= a.mt - i;
      ++i;
    }
    r.i = i;
    r.j = i + u;
  }
  return r;
}

// Instruction descriptor: fp16 operands, fp32 accumulator, M = 256, N = 256.
__host__ __device__ constexpr uint32_t orth_idesc(bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((256u >> 3) << 17) | ((256u >> 4) << 24);
}

__device__ __forceinline__ void st_shared_v4u(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int MODE, bool LAST>
__global__ void __launch_bounds__(192, 1)
    orth_gemm_kernel(const __grid_constant__ OrthMaps maps, const __grid_constant__ OrthArgs args) {
  constexpr bool B_MN = MODE == kUpdate;
  constexpr int STAGES = kOrthStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (sbase - raw);
  const uint32_t s_epi = sbase + STAGES * kStageBytes;
  const uint32_t bars = s_epi + 4 * kEpiWarpBytes;
  const uint32_t full_bar = bars;                    // [STAGES]
  const uint32_t empty_bar = bars + 8 * STAGES;      // [STAGES]
  const uint32_t tfull_bar = bars + 16 * STAGES;     // [2]
  const uint32_t tempty_bar = tfull_bar + 16;        // [2]
  const uint32_t drain_bar = tempty_bar + 16;        // end of the MMA stream
  const uint32_t tmem_slot = drain_bar + 8;
  volatile uint32_t* tmem_slot_g = reinterpret_cast<volatile uint32_t*>(gbase + (tmem_slot - sbase));

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int crank = static_cast<int>(cluster_ctarank());
  const bool leader = crank == 0;
  constexpr uint16_t kPairMask = 0x3;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar + 8 * s, 1);
      mbar_init(empty_bar + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(tfull_bar + 8 * s, 1);
      mbar_init(tempty_bar + 8 * s, 8);   // one lane of every epilogue warp of the pair
    }
    mbar_init(drain_bar, 1);
    fence_barrier_init();
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.b);
  }
  if (warp == 1) {
    tmem_alloc2(tmem_slot, 512);
    tmem_relinquish2();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist before any remote use
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot_g;
  const int per = MODE == kUpdate ? args.mt * args.nt : args.mt * (args.mt + 1) / 2;
  const int total = args.batch * per;
  const int unit0 = blockIdx.x / 2, ustride = gridDim.x / 2;
  const uint64_t tmo = args.timeout_ns;
  auto ring_next = [](int& s, uint32_t& p) {
    if (++s == STAGES) {
      s = 0;
      p ^= 1u;
    }
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint32_t full_l = mapa_shared(full_bar, 0);   // the leader's, for the bytes of both
      int stage = 0;
      uint32_t phase = 0;
      int64_t issued = 0;
      bool ok = true;
      for (int t = unit0; t < total && ok; t += ustride) {
        const OrthTile ti = orth_tile<MODE>(args, t);
        const int ra = ti.i * 256 + crank * 128, rb = ti.j * 256 + crank * 128;
        for (int kb = 0; kb < args.num_kb; ++kb) {
          if (!mbar_wait(empty_bar + 8 * stage, phase ^ 1u, tmo)) {
            record_error(args.err, kErrTimeout);
            ok = false;
            break;
          }
          const uint32_t sA = sbase + stage * kStageBytes, sB = sA + 128 * 128;
          const uint32_t fb = full_l + 8 * stage;
          if (leader) mbar_arrive_expect_tx(full_bar + 8 * stage, 2 * kStageBytes);
          tma_load_3d_g2(sA, &maps.a, fb, kb * 64, ra, ti.e);
          if constexpr (B_MN) {
            tma_load_3d_g2(sB, &maps.b, fb, rb, kb * 64, ti.e);
            tma_load_3d_g2(sB + 64 * 128, &maps.b, fb, rb + 64, kb * 64, ti.e);
          } else {
            tma_load_3d_g2(sB, &maps.b, fb, kb * 64, rb, ti.e);
          }
          ++issued;
          ring_next(stage, phase);
        }
      }
      // Before the CTAs may exit, every load issued must have landed: the leader's
      // full barriers count the bytes of both.
      if (leader) {
        for (int s = 0; s < STAGES; ++s) {
          const int64_t n_s = issued > s ? (issued - 1 - s) / STAGES + 1 : 0;
          if (n_s > 0 && !mbar_wait(full_bar + 8 * s, static_cast<uint32_t>((n_s - 1) & 1), 1000000000ull))
            record_error(args.err, kErrTimeout);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (leader && lane == 0) {
      constexpr uint32_t idesc = orth_idesc(B_MN);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int t = unit0; t < total && ok; t += ustride) {
        if (!mbar_wait(tempty_bar + 8 * acc, acc_phase ^ 1u, tmo)) {
          record_error(args.err, kErrTimeout);
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * 256;
        for (int kb = 0; kb < args.num_kb; ++kb) {
          if (!mbar_wait(full_bar + 8 * stage, phase, tmo)) {
            record_error(args.err, kErrTimeout);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sA = sbase + stage * kStageBytes, sB = sA + 128 * 128;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t ad = smem_desc_sw128(sA + kk * 32, 16, 1024);
            const uint64_t bd = B_MN ? smem_desc_sw128(sB + kk * 16 * 128, 64 * 128, 1024)
                                     : smem_desc_sw128(sB + kk * 32, 16, 1024);
            tc_mma2(d_tmem, ad, bd, idesc, (kb | kk) != 0 ? 1u : 0u);
          }
          // the slot is free in both CTAs once these MMAs have read it
          tc_commit2_mc(empty_bar + 8 * stage, kPairMask);
          ring_next(stage, phase);
        }
        if (!ok) break;
        tc_commit2_mc(tfull_bar + 8 * acc, kPairMask);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      // one more commit arrives in both CTAs once everything issued has completed
      tc_commit2_mc(drain_bar, kPairMask);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;             // tensor-memory lanes, and rows of the CTA's 128
    uint8_t* stage_g = gbase + (s_epi - sbase) + (warp - 2) * kEpiWarpBytes;
    const uint32_t stage_s = s_epi + (warp - 2) * kEpiWarpBytes;
    int buf = 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = unit0; t < total; t += ustride) {
      const OrthTile ti = orth_tile<MODE>(args, t);
      int good = 1;
      if (lane == 0) good = mbar_wait(tfull_bar + 8 * acc, acc_phase, tmo);
      good = __shfl_sync(0xffffffffu, good, 0);
      if (!good) {
        if (lane == 0) record_error(args.err, kErrTimeout);
        break;
      }
      tc_fence_after();
      const int r0 = ti.i * 256 + crank * 128 + q * 32, c0 = ti.j * 256;
      const uint32_t tacc = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * 256;
      if (r0 < args.m) {
        const bool mirror = MODE != kUpdate && ti.i != ti.j;
#pragma unroll 1
        for (int c = 0; c < 256 && c0 + c < args.n; c += 64) {
          float v[64];
          tmem_ld64(tacc + c, v);
          const int row = r0 + lane, col = c0 + c;
          if constexpr (MODE == kPoly) {
#pragma unroll
            for (int j = 0; j < 64; j += 8) {
              float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
              if (row < args.m && col + j < args.lda) {   // lda: a multiple of 8, as col is
                const uint4 u = __ldg(reinterpret_cast<const uint4*>(
                    args.A + ti.e * args.astride + static_cast<int64_t>(row) * args.lda + col + j));
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
                  x[2 * k] = f.x, x[2 * k + 1] = f.y;
                }
              }
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                v[j + k] = fmaf(args.cA, x[k], args.ds * v[j + k]);
                if (row == col + j + k) v[j + k] += args.cI;
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < 64; ++j) v[j] *= args.ds;
          }
          if constexpr (!LAST) {
            // 32 rows of 64 values, in the 128-byte swizzle, stored by one lane
            const uint32_t st = stage_s + buf * 4096;
            if (lane == 0) bulk_wait_read<1>();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              st_shared_v4u(st + lane * 128 + ((j ^ (lane & 7)) << 4), pack_half(v[8 * j], v[8 * j + 1]),
                            pack_half(v[8 * j + 2], v[8 * j + 3]), pack_half(v[8 * j + 4], v[8 * j + 5]),
                            pack_half(v[8 * j + 6], v[8 * j + 7]));
            fence_async_shared();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(&maps.out, st, col, r0, ti.e);
              bulk_commit();
            }
            buf ^= 1;
            if (mirror) {
              // 64 rows (the tile's columns) of 32 values
              const uint32_t tt = stage_s + buf * 4096;
              if (lane == 0) bulk_wait_read<1>();
              __syncwarp();
              __half* h = reinterpret_cast<__half*>(stage_g + buf * 4096);
#pragma unroll
              for (int j = 0; j < 64; ++j) h[j * 32 + lane] = __float2half_rn(v[j]);
              fence_async_shared();
              __syncwarp();
              if (lane == 0) {
                tma_store_3d(&maps.out_t, tt, r0, col, ti.e);
                bulk_commit();
              }
              buf ^= 1;
            }
          } else {
            // bf16, through the warp's stage, in rows of the result
            __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(stage_g);
            __nv_bfloat16* out = args.out + ti.e * args.out_stride;
            const int rows = min(32, args.m - r0), cols = min(64, args.n - col);
            if (!args.flip) {
              // 32 rows of 64 (16-byte pieces at piece ^ (row & 7))
#pragma unroll
              for (int j = 0; j < 8; ++j)
                st_shared_v4u(stage_s + lane * 128 + ((j ^ (lane & 7)) << 4), pack_bf16(v[8 * j], v[8 * j + 1]),
                              pack_bf16(v[8 * j + 2], v[8 * j + 3]), pack_bf16(v[8 * j + 4], v[8 * j + 5]),
                              pack_bf16(v[8 * j + 6], v[8 * j + 7]));
              __syncwarp();
              if (args.vec) {
                for (int r = lane >> 3; r < rows; r += 4) {
                  const int p = lane & 7;
                  const uint4 u = *reinterpret_cast<const uint4*>(stage_g + r * 128 + ((p ^ (r & 7)) << 4));
                  __nv_bfloat16* d = out + static_cast<int64_t>(r0 + r) * args.out_ld + col + 8 * p;
                  if (8 * p + 8 <= cols) {
                    *reinterpret_cast<uint4*>(d) = u;
                  } else {
                    const __nv_bfloat16* s = reinterpret_cast<const __nv_bfloat16*>(&u);
                    for (int k = 0; 8 * p + k < cols; ++k) d[k] = s[k];
                  }
                }
              } else {
                for (int r = 0; r < rows; ++r)
                  for (int k = lane; k < cols; k += 32)
                    out[static_cast<int64_t>(r0 + r) * args.out_ld + col + k] =
                        h[r * 64 + (((k >> 3) ^ (r & 7)) << 3) + (k & 7)];
              }
            } else {
              // the tile's columns are rows of out: 64 rows of 32
#pragma unroll
              for (int j = 0; j < 64; ++j) h[j * 32 + lane] = __float2bfloat16_rn(v[j]);
              __syncwarp();
              if (args.vec) {
                for (int r = lane >> 2; r < cols; r += 8) {
                  const int p = lane & 3;
                  const uint4 u = *reinterpret_cast<const uint4*>(stage_g + r * 64 + p * 16);
                  __nv_bfloat16* d = out + static_cast<int64_t>(col + r) * args.out_ld + r0 + 8 * p;
                  if (8 * p + 8 <= rows) {
                    *reinterpret_cast<uint4*>(d) = u;
                  } else {
                    const __nv_bfloat16* s = reinterpret_cast<const __nv_bfloat16*>(&u);
                    for (int k = 0; 8 * p + k < rows; ++k) d[k] = s[k];
                  }
                }
              } else {
                for (int r = 0; r < cols; ++r)
                  if (lane < rows) out[static_cast<int64_t>(col + r) * args.out_ld + r0 + lane] = h[r * 32 + lane];
              }
            }
            __syncwarp();
          }
        }
      }
      // release the accumulator to the MMA issuer
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader)
          mbar_arrive(tempty_bar + 8 * acc);
        else
          mbar_arrive_cluster_relaxed(mapa_shared(tempty_bar + 8 * acc, 0));
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (!LAST) {
      if (lane == 0) bulk_wait_all();
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  // Every MMA of the pair has completed once the drain barrier has seen the leader's
  // final commit; only then may tensor memory be freed and the CTAs exit.
  if (warp == 1 && lane == 0 && !mbar_wait(drain_bar, 0, 1000000000ull)) record_error(args.err, kErrTimeout);
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc2(tmem_base, 512);
}

template <int MODE, bool LAST>
cudaError_t launch_orth(const OrthMaps& maps, const OrthArgs& args, int sms, cudaStream_t st) {
  auto kern = orth_gemm_kernel<MODE, LAST>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kOrthSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  const int64_t units = static_cast<int64_t>(args.batch) *
                        (MODE == kUpdate ? args.mt * args.nt : args.mt * (args.mt + 1) / 2);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<int64_t>(units, sms / 2)));
  cfg.blockDim = dim3(192);
  cfg.dynamicSmemBytes = kOrthSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, maps, args);
}

// ------------------------------------------------------------ host
constexpr int kMaxOrthSide = 65536;
constexpr int kMaxOrthSteps = 32;
const float kDefaultCoefs[3] = {3.4445f, -4.7750f, 2.0315f};

struct OrthPlan {
  int m, n;            // m <= n
  int flip;
  int ldx, lda;
  int nparts, part_rows;
  int chunk;           // matrices per launch
  size_t parts, x[2], a, b, total;
};

int64_t round8(int64_t v) { return (v + 7) & ~static_cast<int64_t>(7); }

// Matrices go through in chunks of about kChunkUnits tiles, enough to fill the last
// wave of the 76 CTA pairs well, so the workspace does not grow with E.
constexpr int kChunkUnits = 1200;

bool orth_plan(int64_t E, int64_t M, int64_t N, OrthPlan* p) {
  if (E < 0 || M < 1 || N < 1 || M > kMaxOrthSide || N > kMaxOrthSide) return false;
  p->flip = M > N;
  p->m = static_cast<int>(std::min(M, N));
  p->n = static_cast<int>(std::max(M, N));
  p->ldx = static_cast<int>(round8(p->n));
  p->lda = static_cast<int>(round8(p->m));
  p->nparts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({(M * N + kNormElems - 1) / kNormElems, M, kMaxParts})));
  p->part_rows = static_cast<int>((M + p->nparts - 1) / p->nparts);
  p->nparts = static_cast<int>((M + p->part_rows - 1) / p->part_rows);
  const int64_t mt = (p->m + 255) / 256;
  const int64_t units = mt * (mt + 1) / 2;
  p->chunk = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({E, (kChunkUnits + units - 1) / units, 4096})));
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += abi_align256(bytes);
    return o;
  };
  const size_t C = p->chunk;
  p->parts = take(sizeof(Squares) * C * p->nparts);
  p->x[0] = take(2 * C * p->m * static_cast<size_t>(p->ldx));
  p->x[1] = take(2 * C * p->m * static_cast<size_t>(p->ldx));
  p->a = take(2 * C * p->m * static_cast<size_t>(p->lda));
  p->b = take(2 * C * p->m * static_cast<size_t>(p->lda));
  p->total = at;
  return true;
}

// Bounds of the iteration for singular values in [0, u]: of B's eigenvalues, and of
// the next singular values.
void orth_bounds(const float* c, double u, double* B, double* next) {
  const double c0 = c[0], c1 = c[1], c2 = c[2];
  auto b = [&](double t) { return c0 + t * (c1 + t * c2); };
  auto p = [&](double s) { return s * b(s * s); };
  *B = std::max(std::fabs(b(0)), std::fabs(b(u * u)));
  if (c2 != 0) {
    const double t = -c1 / (2 * c2);
    if (t > 0 && t < u * u) *B = std::max(*B, std::fabs(b(t)));
  }
  *next = std::fabs(p(u));
  // p' = c0 + 3 c1 t + 5 c2 t^2 with t = s^2
  const double disc = 9 * c1 * c1 - 20 * c0 * c2;
  double roots[2] = {-1, -1};
  if (c2 != 0 && disc >= 0) {
    roots[0] = (-3 * c1 + std::sqrt(disc)) / (10 * c2);
    roots[1] = (-3 * c1 - std::sqrt(disc)) / (10 * c2);
  } else if (c2 == 0 && c1 != 0) {
    roots[0] = -c0 / (3 * c1);
  }
  for (double t : roots)
    if (t > 0 && t < u * u) *next = std::max(*next, std::fabs(p(std::sqrt(t))));
}

// The factor S (a power of two) for these coefficients, or 0 where fp16 does not hold
// what they lead to.
float orth_scale(const float* coefs, int steps, int n) {
  double u = 1.0, top = 1.0;
  for (int i = 0; i < steps; ++i) {
    const float* c = coefs ? coefs + 3 * i : kDefaultCoefs;
    double B, next;
    if (!std::isfinite(c[0]) || !std::isfinite(c[1]) || !std::isfinite(c[2])) return 0.f;
    orth_bounds(c, u, &B, &next);
    if (!(B < 1e4) || !(next < 100.0)) return 0.f;
    top = std::max({top, B, u * u});
    u = std::max(next * 1.01, 1e-3);     // what the roundings may add
    if (i + 1 < steps) top = std::max(top, u * u);
  }
  int s = static_cast<int>(std::lround(std::log2(static_cast<double>(n)) / 2));
  while (s > 0 && std::ldexp(top, 2 * s) > 60000.0) --s;
  return std::ldexp(top, 2 * s) <= 60000.0 ? std::ldexp(1.f, s) : 0.f;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_orthogonalize_workspace_size(int64_t E, int64_t M, int64_t N) {
  OrthPlan p;
  return orth_plan(E, M, N, &p) ? p.total : 0;
}

moe_status moe_orthogonalize(int64_t E, int64_t M, int64_t N, int32_t dtype, const void* g, int64_t g_ld,
                             int64_t g_stride, int32_t steps, const float* coefs, float eps, float scale,
                             void* out, int64_t out_ld, int64_t out_stride, void* ws, size_t ws_bytes,
                             moe_stream_t stream) {
  OrthPlan p;
  if (!orth_plan(E, M, N, &p) || (dtype != MOE_BF16 && dtype != MOE_FP32)) return MOE_ERR_INVALID_ARG;
  if (steps < 1 || steps > kMaxOrthSteps || !(eps >= 0.f) || eps - eps != 0.f || scale - scale != 0.f)
    return MOE_ERR_INVALID_ARG;
  const float S = orth_scale(coefs, steps, p.n);
  if (S == 0.f) return MOE_ERR_INVALID_ARG;
  if (g_ld < N || out_ld < N || g_stride < 0 || out_stride < 0) return MOE_ERR_INVALID_ARG;
  if (E > 1 && out_stride < (M - 1) * out_ld + N) return MOE_ERR_INVALID_ARG;
  if (E == 0) return MOE_OK;
  const int es = dtype == MOE_FP32 ? 4 : 2;
  if (!g || !out || (reinterpret_cast<uintptr_t>(g) & (es - 1)) || (reinterpret_cast<uintptr_t>(out) & 1))
    return MOE_ERR_INVALID_ARG;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < p.total) return MOE_ERR_WORKSPACE;
  int sms = 0;
  const moe_status ds = abi_device_sms(&sms);
  if (ds != MOE_OK) return ds;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(ws);
  Squares* parts = reinterpret_cast<Squares*>(w + p.parts);
  __half* x[2] = {reinterpret_cast<__half*>(w + p.x[0]), reinterpret_cast<__half*>(w + p.x[1])};
  __half* a = reinterpret_cast<__half*>(w + p.a);
  __half* b = reinterpret_cast<__half*>(w + p.b);
  const uint64_t C = p.chunk;
  const auto SW = CU_TENSOR_MAP_SWIZZLE_128B, NOSW = CU_TENSOR_MAP_SWIZZLE_NONE;
  OrthMaps gram[2], poly, update[2];
  bool ok = true;
  for (int i = 0; i < 2; ++i) {
    ok = ok && abi_map_half(&gram[i].a, x[i], p.n, p.m, C, p.ldx, 64, 128, SW) &&
         abi_map_half(&gram[i].out, a, p.m, p.m, C, p.lda, 64, 32, SW) &&
         abi_map_half(&gram[i].out_t, a, p.m, p.m, C, p.lda, 32, 64, NOSW) &&
         abi_map_half(&update[i].a, b, p.m, p.m, C, p.lda, 64, 128, SW) &&
         abi_map_half(&update[i].b, x[i], p.n, p.m, C, p.ldx, 64, 64, SW) &&
         abi_map_half(&update[i].out, x[1 - i], p.n, p.m, C, p.ldx, 64, 32, SW);
    gram[i].b = gram[i].a;
    update[i].out_t = update[i].out;
  }
  ok = ok && abi_map_half(&poly.a, a, p.m, p.m, C, p.lda, 64, 128, SW) &&
       abi_map_half(&poly.out, b, p.m, p.m, C, p.lda, 64, 32, SW) &&
       abi_map_half(&poly.out_t, b, p.m, p.m, C, p.lda, 32, 64, NOSW);
  if (!ok) return MOE_ERR_CUDA;
  poly.b = poly.a;
  const float S2 = S * S;
  OrthArgs base = {};
  base.mt = (p.m + 255) / 256;
  base.err = static_cast<int*>(ws);
  base.timeout_ns = abi_wait_timeout_ns();
  base.m = p.m;
  base.A = a, base.lda = p.lda, base.astride = static_cast<int64_t>(p.m) * p.lda;
  for (int64_t e0 = 0; e0 < E; e0 += p.chunk) {
    const int batch = static_cast<int>(std::min<int64_t>(p.chunk, E - e0));
    const char* gp = static_cast<const char*>(g) + e0 * g_stride * es;
    const int W = 16 / es;
    OrthIn in{gp, g_ld, g_stride, static_cast<int>(M), static_cast<int>(N), dtype == MOE_BF16,
              (reinterpret_cast<uintptr_t>(gp) & 15) == 0 && g_ld % W == 0 && (batch == 1 || g_stride % W == 0)};
    cudaError_t e = abi_tracked(kAbiOrthLoad, 2, st, [&] {
      orth_norm_kernel<<<dim3(p.nparts, batch), kNormThreads, 0, st>>>(in, p.part_rows, parts);
      cudaError_t r = cudaGetLastError();
      if (r != cudaSuccess) return r;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>((N + 63) / 64), static_cast<unsigned>((M + 63) / 64), batch);
      cfg.blockDim = dim3(256);
      cfg.stream = st;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      auto go = [&](auto kern) {
        return cudaLaunchKernelEx(&cfg, kern, in, static_cast<const Squares*>(parts), p.nparts, eps, S, x[0], p.ldx,
                                  static_cast<int64_t>(p.m) * p.ldx);
      };
      if (dtype == MOE_FP32) return p.flip ? go(orth_load_kernel<float, true>) : go(orth_load_kernel<float, false>);
      return p.flip ? go(orth_load_kernel<__nv_bfloat16, true>) : go(orth_load_kernel<__nv_bfloat16, false>);
    });
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    base.batch = batch;
    for (int i = 0; i < steps; ++i) {
      const float* c = coefs ? coefs + 3 * i : kDefaultCoefs;
      OrthArgs args = base;
      args.n = p.m, args.nt = args.mt, args.num_kb = (p.n + 63) / 64, args.ds = 1.f;
      e = abi_tracked(kAbiOrthGram, 1, st, [&] { return launch_orth<kGram, false>(gram[i & 1], args, sms, st); });
      if (e != cudaSuccess) return MOE_ERR_CUDA;
      args.num_kb = (p.m + 63) / 64, args.ds = c[2] / S2, args.cA = c[1], args.cI = c[0] * S2;
      e = abi_tracked(kAbiOrthPoly, 1, st, [&] { return launch_orth<kPoly, false>(poly, args, sms, st); });
      if (e != cudaSuccess) return MOE_ERR_CUDA;
      args.n = p.n, args.nt = (p.n + 255) / 256, args.ds = 1.f / S2;
      const bool last = i + 1 == steps;
      if (last) {
        args.ds = scale / (S2 * S);
        args.out = static_cast<__nv_bfloat16*>(out) + e0 * out_stride;
        args.out_ld = out_ld, args.out_stride = out_stride, args.flip = p.flip;
        args.vec = (reinterpret_cast<uintptr_t>(args.out) & 15) == 0 && out_ld % 8 == 0 &&
                   (batch == 1 || out_stride % 8 == 0);
      }
      e = abi_tracked(kAbiOrthUpdate, 1, st, [&] {
        return last ? launch_orth<kUpdate, true>(update[i & 1], args, sms, st)
                    : launch_orth<kUpdate, false>(update[i & 1], args, sms, st);
      });
      if (e != cudaSuccess) return MOE_ERR_CUDA;
    }
  }
  return MOE_OK;
}

}  // extern "C"
