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
// rounding: 1.7e-3).  A g of low rank shows it most, 2.5e-2 for rank 32 and 8e-2 for
// rank 4: what it does not contain is nothing but roundings, grown c0-fold a step.
// fp16's range is kept by powers of two: X holds S x and A and B hold S^2 times theirs,
// S near sqrt(max(M, N)), so that typical values are far from both ends; the
// coefficients' bounds (checked on the host) keep the largest below 60000.
//
// Measured, five steps: 4 of 2880 x 2880 fp32 1.27 ms, 1.48 in a row of them (by the clock
// that the power leaves), 8 of 2816 x 2816 at 1.66 PFLOP/s of what is needed, at the rate that a library
// product sustains; 6 of 333 x 1001 101 us and 8 of 128 x 128 23 us, both bound by the
// chain of dependent steps.
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
constexpr int kNormElems = 8192;       // of a matrix per block of the norm, at least
constexpr int kNormBlocks = 1216;      // about, of a launch
constexpr int kMaxParts = 1024;        // blocks per matrix

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
  int vec;              // rows start on 16 bytes
};

// Elements [c, c + 8) of a row, 0 past its end.
template <typename E>
__device__ __forceinline__ void load_row8(const OrthIn& in, const E* row, int c, float (&v)[8]) {
  if (in.vec && c + 8 <= in.N) {
    load8(row + c, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = c + k < in.N ? to_f32(row[c + k]) : 0.f;
  }
}

// Sum of squares of rows [blockIdx.x * rows, ...) of matrix blockIdx.y: the block's
// threads walk the rows' groups of eight columns, four at a time.
template <typename E>
__global__ void __launch_bounds__(kNormThreads) orth_norm_kernel(const OrthIn in, int rows, Squares* parts) {
  __shared__ float part[3][32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int r1 = min(in.M, static_cast<int>(blockIdx.x + 1) * rows);
  const E* g = static_cast<const E*>(in.g) + static_cast<int64_t>(blockIdx.y) * in.stride;
  const int nv = (in.N + 7) / 8;
  const int dr = kNormThreads / nv, dc = kNormThreads - dr * nv;   // a step of all threads
  int r = blockIdx.x * rows + static_cast<int>(threadIdx.x) / nv, c = static_cast<int>(threadIdx.x) % nv;
  Squares s;
  while (r < r1) {
    float v[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (r < r1) {
        load_row8(in, g + r * in.ld, 8 * c, v[u]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[u][k] = 0.f;
      }
      r += dr, c += dc;
      if (c >= nv) c -= nv, ++r;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int k = 0; k < 8; ++k) s.add(v[u][k]);
  }
  s.mid = block_sum(s.mid, part[0]);
  s.big = block_sum(s.big, part[1]);
  s.small = block_sum(s.small, part[2]);
  if (threadIdx.x == 0) parts[static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = s;
}

// The factors (pre, f) with x_0 S = (g pre) f, of the matrix's sums of squares.
__device__ __forceinline__ float2 orth_factor_of(const Squares& v, float eps, float S) {
  float pre = 1.f, ss = v.mid;
  if (!isfinite(v.mid))
    pre = 0x1p-80f, ss = v.big;
  else if (v.mid < 0x1p-40f)
    pre = 0x1p80f, ss = v.small;
  const float norm = sqrtf(ss) + eps * pre;
  // a matrix of zeros stays zero without eps too; one that holds an infinity or a NaN
  // is NaN throughout (eps * pre may be infinite beside a finite matrix: x_0 = 0)
  const float f = norm == 0.f ? 0.f : (isfinite(ss) ? S / norm : __int_as_float(0x7fc00000));
  return make_float2(pre, f);
}

// The same of its blocks' sums, in every thread.
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
  return orth_factor_of(v, eps, S);
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// X [m, ldx] fp16 from g, tiles of 64 x 64 of matrix blockIdx.y in turn; the columns
// from n to ldx hold 0.  Also clears the counters of the products.
template <typename E, bool FLIP>
__global__ void __launch_bounds__(256) orth_load_kernel(const OrthIn in, const Squares* parts, int nparts, float eps,
                                                        float S, __half* X, int ldx, int64_t xstride, int* counters,
                                                        int ncounters) {
  __shared__ float tile[FLIP ? 64 : 1][FLIP ? 65 : 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the sums are there
  const int e = blockIdx.y;
  if (blockIdx.x == 0 && e == 0)
    for (int i = threadIdx.x; i < ncounters; i += 256) counters[i] = 0;
  const float2 f = orth_factor(parts + static_cast<int64_t>(e) * nparts, nparts, eps, S);
  const E* g = static_cast<const E*>(in.g) + static_cast<int64_t>(e) * in.stride;
  __half* x = X + static_cast<int64_t>(e) * xstride;
  const int tc = (in.N + 63) / 64, tiles = tc * ((in.M + 63) / 64);
  const int c8 = (threadIdx.x & 7) * 8, i0 = threadIdx.x >> 3;   // 32 rows of eight groups of eight
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int r0 = t / tc * 64, c0 = t % tc * 64;   // of g
    float v[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + i0 + 32 * h;
      if (r < in.M && c0 + c8 < in.N) {
        load_row8(in, g + r * in.ld, c0 + c8, v[h]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[h][k] = 0.f;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = i0 + 32 * h;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[h][k] = v[h][k] * f.x * f.y;
      if (FLIP) {
#pragma unroll
        for (int k = 0; k < 8; ++k) tile[c8 + k][i] = v[h][k];
      }
    }
    if (FLIP) {
      __syncthreads();
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[h][k] = tile[i0 + 32 * h][c8 + k];
      __syncthreads();
    }
    const int rows = FLIP ? in.N : in.M, xr0 = FLIP ? c0 : r0, xc = (FLIP ? r0 : c0) + c8;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (xr0 + i0 + 32 * h < rows && xc < ldx)
        *reinterpret_cast<uint4*>(x + static_cast<int64_t>(xr0 + i0 + 32 * h) * ldx + xc) =
            make_uint4(pack_half(v[h][0], v[h][1]), pack_half(v[h][2], v[h][3]), pack_half(v[h][4], v[h][5]),
                       pack_half(v[h][6], v[h][7]));
  }
}

// ------------------------------------------------------------ products
// All steps of a batch in one persistent kernel on CTA pairs (2-SM MMA, M = 256,
// N <= 256): the phases gram, poly, update of every step, in each phase the tiles of
// every matrix, make one list of units that the pairs take in turn.  A unit waits for
// the phase before it of its own matrix only (a counter per matrix and phase), so
// with a few matrices no pair waits for the end of a phase, and a step costs no
// launches.  The launch is cooperative: pairs wait for one another, so all of them
// have to be resident (one CTA per SM).
//
// Within a unit each CTA loads 128 rows of A and half of B's columns per 64 columns
// of K into a ring, one lane of the even CTA issues the MMAs, the accumulators are
// double-buffered in tensor memory and eight warps per CTA store them.  The producer's
// and the issuer's warps stay whole and elect the lane that issues: with one lane in a
// branch of its own a block of K takes 300 ns whatever its width, so 64-column tiles
// took 3.5 ms where they now take 2.5 (4 x 2816 x 2816).  Unwinding as in the expert
// layer's grouped products.
enum OrthPhase : int { kGram = 0, kPoly = 1, kUpdate = 2 };

constexpr int kOrthStages = 6;
constexpr int kStageBytes = 2 * 128 * 128;
constexpr int kEpiWarps = 8;             // two for each quarter of the tensor memory's lanes
constexpr int kOrthThreads = 64 + 32 * kEpiWarps;
constexpr int kTileBytes = 32 * 32 * 2;  // what a warp stores at once
constexpr int kEpiWarpBytes = 2 * kTileBytes;
constexpr int kOrthBars = (2 * kOrthStages + 5) * 8 + 40;
constexpr int kOrthSmem = 1024 + kOrthStages * kStageBytes + kEpiWarps * kEpiWarpBytes + kOrthBars;
constexpr int kMaxOrthSteps = 32;
constexpr int kUnitArrivals = 2;               // one per CTA
static_assert(kOrthSmem <= 232448, "shared memory budget");

struct OrthMaps {
  CUtensorMap xk[2];   // X as a K-major operand, rows of A: box {64, 128}
  CUtensorMap xs[2];   //   rows of B: box {64, bn_sym / 2}
  CUtensorMap xn[2];   // X as the MN-major operand of the update: box {64, 64}
  CUtensorMap xo[2];   // X as a result: box {32, 32}
  CUtensorMap ak, as, ao, at;   // A likewise; at: mirrored
  CUtensorMap bk, bo, bt;       // B
};

struct OrthArgs {
  int m, n;              // of X
  int batch, steps;
  int mt;                // row tiles of 256
  int bn_sym, nt_sym;    // column tiles of the symmetric products: width and number
  int bn_upd, nt_upd;    // of the update
  int units_sym, units_upd;   // per matrix
  float S2, inv_S2;      // A and B hold S2 times theirs
  float out_scale;       // scale / S
  const __half* A;       // [batch][m][lda]
  int lda;
  int64_t astride;
  __nv_bfloat16* out;    // the last update: out[e][r][c], transposed when `flip`
  int64_t out_ld, out_stride;
  int flip, vec;         // vec: rows of out start on 16 bytes
  int* counters;         // [3 steps][batch], cleared before the launch
  int* err;
  uint64_t timeout_ns;
  float coefs[kMaxOrthSteps][3];
};

struct OrthUnit {
  int phase;       // 3 * step + OrthPhase
  int kind, step;
  int e, i, c0;    // matrix, row tile, first column
  int nn;          // columns: a multiple of 16
  bool mirror;     // the tile lies above the diagonal
};

// Unit t.  A symmetric result has the column tiles from the diagonal tile's first
// column on: those inside the diagonal 256 x 256 block are stored as they are, those
// beyond it mirrored too.
__device__ __forceinline__ OrthUnit orth_unit(const OrthArgs& a, int t) {
  OrthUnit u;
  const int us = a.units_sym * a.batch, per_step = 2 * us + a.units_upd * a.batch;
  u.step = t / per_step;
  int r = t - u.step * per_step;
  int cols, bn;
  if (r < 2 * us) {
    u.kind = r < us ? kGram : kPoly;
    if (u.kind == kPoly) r -= us;
    u.e = r / a.units_sym;
    r -= u.e * a.units_sym;
    const int f = 256 / a.bn_sym;   // column tiles in a diagonal block
    int i = 0;
    while (r >= a.nt_sym - i * f) {
      r -= a.nt_sym - i * f;
      ++i;
    }
    u.i = i;
    bn = a.bn_sym, cols = a.m;
    u.c0 = (i * f + r) * bn;
    u.mirror = r >= f;
  } else {
    r -= 2 * us;
    u.kind = kUpdate;
    u.e = r / a.units_upd;
    r -= u.e * a.units_upd;
    const int j = r / a.mt;
    u.i = r - j * a.mt;
    bn = a.bn_upd, cols = a.n;
    u.c0 = j * bn;
    u.mirror = false;
  }
  u.phase = 3 * u.step + u.kind;
  u.nn = (min(bn, cols - u.c0) + 15) & ~15;
  return u;
}

// Instruction descriptor: fp16 operands, fp32 accumulator, M = 256.
__device__ __forceinline__ uint32_t orth_idesc(bool b_mn, int n) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) | ((256u >> 4) << 24);
}

__device__ __forceinline__ void st_shared_v4u(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Halves of a shared-memory descriptor (128-byte swizzle, 1024 bytes between groups of
// eight rows): the low one with the address and the leading offset, the high one fixed.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo_bytes) {
  return ((saddr >> 4) & 0x3fffu) | ((lbo_bytes >> 4) << 16);
}
__device__ __forceinline__ void orth_mma(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  tc_mma2(d_tmem, static_cast<uint64_t>(kDescHi) << 32 | a_lo, static_cast<uint64_t>(kDescHi) << 32 | b_lo, idesc, accumulate);
}

// One lane of the (whole, converged) warp: unlike a comparison with the lane's number it
// leaves the compiler's knowledge of what is the same in all lanes alone.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r) : : "memory");
  return r != 0;
}

__device__ __forceinline__ int load_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ void add_release(int* p, int v) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// To a count in shared memory; what is done before it, in any of the warps that have
// counted, is before what the last one does.
__device__ __forceinline__ uint32_t add_cta(uint32_t addr, uint32_t v) {
  uint32_t old;
  asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(addr), "r"(v) : "memory");
  return old;
}

__device__ __forceinline__ void store_release_cta(uint32_t addr, int v) {
  asm volatile("st.release.cta.shared::cta.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Wait until the count has come to v: false when that takes longer than the limit.
__device__ __forceinline__ bool wait_count_cta(uint32_t addr, int v, uint64_t timeout_ns) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t i = 1;; ++i) {
    int now;
    asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];" : "=r"(now) : "r"(addr) : "memory");
    if (now >= v) return true;
    if ((i & 31u) == 0 && global_timer_ns() - t0 > timeout_ns) return false;
  }
}

// Wait until the unit's matrix has finished the phase before: false when that takes
// longer than the limit.
__device__ __forceinline__ bool orth_wait(const OrthArgs& a, const OrthUnit& u, uint64_t timeout_ns) {
  if (u.phase == 0) return true;      // X is the load kernel's
  const int* c = a.counters + (u.phase - 1) * a.batch + u.e;
  const int target = kUnitArrivals * (u.kind == kGram ? a.units_upd : a.units_sym);
  if (load_acquire(c) >= target) return true;
  const uint64_t t0 = global_timer_ns();
  while (load_acquire(c) < target) {
    if (global_timer_ns() - t0 > timeout_ns) return false;
  }
  return true;
}

// Byte of 16-byte piece j of row r in a 32 x 32 tile of 16-bit values in the 64-byte
// swizzle.
__device__ __forceinline__ uint32_t tile_piece(int r, int j) { return r * 64 + ((j ^ ((r >> 1) & 3)) << 4); }

// The bf16 values of a 32 x 32 tile (lane: row) to out[r0 + row][col + ...] or, with `flip`,
// to its transpose, through the warp's stage of 2 KB.
__device__ __forceinline__ void store_out(const OrthArgs& a, __nv_bfloat16* out, int r0, int col, int rows, int cols,
                                          const float (&v)[32], uint8_t* stage_g, uint32_t stage_s, int lane) {
  __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(stage_g);
  // rows of the stage are rows of out: the tile's own, or its columns
  if (!a.flip) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      st_shared_v4u(stage_s + tile_piece(lane, j), pack_bf16(v[8 * j], v[8 * j + 1]), pack_bf16(v[8 * j + 2], v[8 * j + 3]),
                    pack_bf16(v[8 * j + 4], v[8 * j + 5]), pack_bf16(v[8 * j + 6], v[8 * j + 7]));
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) h[tile_piece(j, lane >> 3) / 2 + (lane & 7)] = __float2bfloat16_rn(v[j]);
  }
  __syncwarp();
  const int or0 = a.flip ? col : r0, oc0 = a.flip ? r0 : col, n = a.flip ? cols : rows, len = a.flip ? rows : cols;
  if (a.vec) {
    for (int r = lane >> 2; r < n; r += 8) {
      const int p = lane & 3;
      const uint4 u = *reinterpret_cast<const uint4*>(stage_g + tile_piece(r, p));
      __nv_bfloat16* d = out + static_cast<int64_t>(or0 + r) * a.out_ld + oc0 + 8 * p;
      if (8 * p + 8 <= len) {
        *reinterpret_cast<uint4*>(d) = u;
      } else {
        const __nv_bfloat16* s = reinterpret_cast<const __nv_bfloat16*>(&u);
        for (int k = 0; 8 * p + k < len; ++k) d[k] = s[k];
      }
    }
  } else if (lane < len) {
    for (int r = 0; r < n; ++r)
      out[static_cast<int64_t>(or0 + r) * a.out_ld + oc0 + lane] = h[tile_piece(r, lane >> 3) / 2 + (lane & 7)];
  }
  __syncwarp();
}

__global__ void __launch_bounds__(kOrthThreads, 1)
    orth_steps_kernel(const __grid_constant__ OrthMaps maps, const __grid_constant__ OrthArgs args) {
  constexpr int STAGES = kOrthStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (sbase - raw);
  const uint32_t s_epi = sbase + STAGES * kStageBytes;
  const uint32_t bars = s_epi + kEpiWarps * kEpiWarpBytes;
  const uint32_t full_bar = bars;                    // [STAGES]
  const uint32_t empty_bar = bars + 8 * STAGES;      // [STAGES]
  const uint32_t tfull_bar = bars + 16 * STAGES;     // [2]
  const uint32_t tempty_bar = tfull_bar + 16;        // [2]
  const uint32_t drain_bar = tempty_bar + 16;        // end of the MMA stream
  const uint32_t tmem_slot = drain_bar + 8;
  const uint32_t stored = tmem_slot + 8;             // [4]: warps that have stored a unit
  const uint32_t begun = stored + 16;                // units whose matrix the producer has waited for
  const uint32_t issued_slot = begun + 4;            // the leader's [2]: stages that each CTA has loaded
  volatile uint32_t* tmem_slot_g = reinterpret_cast<volatile uint32_t*>(gbase + (tmem_slot - sbase));

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int crank = static_cast<int>(cluster_ctarank());
  const bool leader = crank == 0;
  constexpr uint16_t kPairMask = 0x3;
  constexpr uint64_t kDrain = 1000000000ull;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar + 8 * s, 2);      // of each CTA's producer
      mbar_init(empty_bar + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(tfull_bar + 8 * s, 1);
      mbar_init(tempty_bar + 8 * s, 2 * kEpiWarps);   // one lane of every epilogue warp of the pair
    }
    mbar_init(drain_bar, 1);
    fence_barrier_init();
    st_shared_v4u(stored, 0u, 0u, 0u, 0u);
    store_release_cta(begun, 0);
  }
  if (warp == 2 && lane < static_cast<int>(sizeof(OrthMaps) / sizeof(CUtensorMap)))
    prefetch_tmap(reinterpret_cast<const CUtensorMap*>(&maps) + lane);
  if (warp == 1) {
    tmem_alloc2(tmem_slot, 512);
    tmem_relinquish2();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist before any remote use
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot_g;
  const int total = args.steps * args.batch * (2 * args.units_sym + args.units_upd);
  const int unit0 = blockIdx.x / 2, ustride = gridDim.x / 2;
  const uint64_t tmo = args.timeout_ns;
  auto ring_next = [](int& s, uint32_t& p) {
    if (++s == STAGES) {
      s = 0;
      p ^= 1u;
    }
  };
  auto num_kb = [&](const OrthUnit& u) { return ((u.kind == kGram ? args.n : args.m) + 63) >> 6; };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint32_t full_l = mapa_shared(full_bar, 0);   // the leader's, for the bytes of both
    int stage = 0;
    uint32_t phase = 0;
    uint32_t issued = 0;
    int unit = 0;
    bool ok = true;
    for (int t = unit0; t < total && ok; t += ustride) {
      const OrthUnit u = orth_unit(args, t);
      if (!__all_sync(0xffffffffu, orth_wait(args, u, tmo))) {
        if (lane == 0) record_error(args.err, kErrTimeout);
        break;
      }
      if (lane == 0) store_release_cta(begun, ++unit);
      asm volatile("fence.proxy.async.global;" ::: "memory");   // the loads see what the wait saw (a fence for all memory: 6 of 333 x 1001 116 us)
      const int x = u.step & 1;
      const CUtensorMap* am = u.kind == kGram ? &maps.xk[x] : (u.kind == kPoly ? &maps.ak : &maps.bk);
      const CUtensorMap* bm = u.kind == kGram ? &maps.xs[x] : (u.kind == kPoly ? &maps.as : &maps.xn[x]);
      const bool upd = u.kind == kUpdate, two = upd && args.bn_upd == 256;
      const uint32_t bytes = 128 * 128 + (upd ? (two ? 2 : 1) * 64 * 128 : args.bn_sym / 2 * 128);
      const int ra = u.i * 256 + crank * 128, rb = u.c0 + crank * (u.nn >> 1);
      const int nkb = num_kb(u);
      for (int kb = 0; kb < nkb; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_wait(empty_bar + 8 * stage, phase ^ 1u, tmo))) {
          if (lane == 0) record_error(args.err, kErrTimeout);
          ok = false;
          break;
        }
        const uint32_t sA = sbase + stage * kStageBytes, sB = sA + 128 * 128;
        const uint32_t fb = full_l + 8 * stage;
        const int k0 = kb * 64;
        if (elect_one()) {
          if (leader)
            mbar_arrive_expect_tx(full_bar + 8 * stage, bytes);
          else
            mbar_arrive_expect_tx_cluster(fb, bytes);
          tma_load_3d_g2(sA, am, fb, k0, ra, u.e);
          tma_load_3d_g2(sB, bm, fb, upd ? rb : k0, upd ? k0 : rb, u.e);
          if (two) tma_load_3d_g2(sB + 64 * 128, bm, fb, rb + 64, k0, u.e);
        }
        __syncwarp();
        ++issued;
        ring_next(stage, phase);
      }
    }
    if (lane == 0) st_cluster_u32(mapa_shared(issued_slot + 4 * crank, 0), issued);
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (leader) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int t = unit0; t < total && ok; t += ustride) {
        const OrthUnit u = orth_unit(args, t);
        const bool b_mn = u.kind == kUpdate;
        const uint32_t idesc = orth_idesc(b_mn, u.nn);
        const int nkb = num_kb(u);
        // descriptors of stage 0, and what a step of 16 columns of K adds to B's: one
        // thread issues everything, so each instruction of this loop counts
        const uint32_t a0 = desc_lo(sbase, 16), b0 = desc_lo(sbase + 128 * 128, b_mn ? 64 * 128 : 16);
        const uint32_t b_step = b_mn ? 16 * 128 / 16 : 32 / 16;
        // (the producer has waited for this unit's matrix before; its wait and the
        // loads may take two limits)
        if (!__all_sync(0xffffffffu, mbar_wait(tempty_bar + 8 * acc, acc_phase ^ 1u, tmo))) {
          if (lane == 0) record_error(args.err, kErrTimeout);
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * 256;
        uint64_t limit = 2 * tmo;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!__all_sync(0xffffffffu, mbar_wait(full_bar + 8 * stage, phase, limit))) {
            if (lane == 0) record_error(args.err, kErrTimeout);
            ok = false;
            break;
          }
          limit = tmo;
          tc_fence_after();
          const uint32_t ad = a0 + stage * (kStageBytes / 16), bd = b0 + stage * (kStageBytes / 16);
          if (elect_one()) {
            orth_mma(d_tmem, ad, bd, idesc, kb != 0 ? 1u : 0u);
            orth_mma(d_tmem, ad + 2, bd + b_step, idesc, 1u);
            orth_mma(d_tmem, ad + 4, bd + 2 * b_step, idesc, 1u);
            orth_mma(d_tmem, ad + 6, bd + 3 * b_step, idesc, 1u);
            // the slot is free in both CTAs once these MMAs have read it
            tc_commit2_mc(empty_bar + 8 * stage, kPairMask);
          }
          __syncwarp();
          ring_next(stage, phase);
        }
        if (!ok) break;
        if (elect_one()) tc_commit2_mc(tfull_bar + 8 * acc, kPairMask);
        __syncwarp();
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      // one more commit arrives in both CTAs once everything issued has completed
      if (elect_one()) tc_commit2_mc(drain_bar, kPairMask);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;             // tensor-memory lanes, and rows of the CTA's 128
    const int first = warp < 6 ? 0 : 32;   // every other 32 columns
    uint8_t* stage_g = gbase + (s_epi - sbase) + (warp - 2) * kEpiWarpBytes;
    const uint32_t stage_s = s_epi + (warp - 2) * kEpiWarpBytes;
    int buf = 0;
    int unit = 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = unit0; t < total; t += ustride) {
      const OrthUnit u = orth_unit(args, t);
      const int r0 = u.i * 256 + crank * 128 + q * 32;
      const bool last = u.kind == kUpdate && u.step + 1 == args.steps;
      const int cols = u.kind == kUpdate ? args.n : args.m;
      const uint32_t tacc = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * 256;
      const float cI = args.coefs[u.step][0] * args.S2, cA = args.coefs[u.step][1];
      const float ds = u.kind == kGram ? 1.f
                       : u.kind == kPoly ? args.coefs[u.step][2] * args.inv_S2
                                         : (last ? args.out_scale : 1.f) * args.inv_S2;
      const CUtensorMap* om = u.kind == kGram ? &maps.ao : (u.kind == kPoly ? &maps.bo : &maps.xo[1 - (u.step & 1)]);
      const CUtensorMap* tm = u.kind == kGram ? &maps.at : &maps.bt;
      int good = 1;
      uint4 ax[4];      // poly: A's values of the columns, ahead of the products
      auto fetch_a = [&](int col) {
        const __half* p = args.A + u.e * args.astride + static_cast<int64_t>(r0 + lane) * args.lda + col;
#pragma unroll
        for (int j = 0; j < 4; ++j)      // lda: a multiple of 8, as col is
          ax[j] = r0 + lane < args.m && col + 8 * j < args.lda ? __ldcg(reinterpret_cast<const uint4*>(p) + j)
                                                               : make_uint4(0u, 0u, 0u, 0u);
      };
      if (u.kind == kPoly) {
        // (the producer's word for it: polls of the counters by all warps slow the others
        // down)
        if (lane == 0) good = wait_count_cta(begun, unit + 1, 2 * tmo);
        good = __shfl_sync(0xffffffffu, good, 0);
        if (good) fetch_a(u.c0 + first);
      }
      if (lane == 0 && good) good = mbar_wait(tfull_bar + 8 * acc, acc_phase, 3 * tmo);
      good = __shfl_sync(0xffffffffu, good, 0);
      if (!good) {
        if (lane == 0) record_error(args.err, kErrTimeout);
        break;
      }
      tc_fence_after();
      if (r0 < args.m) {
#pragma unroll 1
        for (int c = first; c < u.nn; c += 64) {
          float v[32];
          tmem_ld32(tacc + c, v);
          const int row = r0 + lane, col = u.c0 + c;
          if (u.kind == kPoly) {
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              float x[8];
              const uint32_t w[4] = {ax[j / 8].x, ax[j / 8].y, ax[j / 8].z, ax[j / 8].w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
                x[2 * k] = f.x, x[2 * k + 1] = f.y;
              }
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                v[j + k] = fmaf(cA, x[k], ds * v[j + k]);
                if (row == col + j + k) v[j + k] += cI;
              }
            }
            if (c + 64 < u.nn) fetch_a(col + 64);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] *= ds;
          }
          if (col >= cols) break;      // (nn is rounded up)
          if (last) {
            store_out(args, args.out + u.e * args.out_stride, r0, col, min(32, args.m - r0), min(32, cols - col), v,
                      stage_g, stage_s, lane);
            continue;
          }
          // 32 rows of 32 values, stored by one lane
          const uint32_t st = stage_s + buf * kTileBytes;
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j)
            st_shared_v4u(st + tile_piece(lane, j), pack_half(v[8 * j], v[8 * j + 1]), pack_half(v[8 * j + 2], v[8 * j + 3]),
                          pack_half(v[8 * j + 4], v[8 * j + 5]), pack_half(v[8 * j + 6], v[8 * j + 7]));
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(om, st, col, r0, u.e);
            bulk_commit();
          }
          buf ^= 1;
          if (u.mirror) {
            // the tile's columns as rows
            const uint32_t tt = stage_s + buf * kTileBytes;
            if (lane == 0) bulk_wait_read<1>();
            __syncwarp();
            __half* h = reinterpret_cast<__half*>(stage_g + buf * kTileBytes);
#pragma unroll
            for (int j = 0; j < 32; ++j) h[j * 32 + lane] = __float2half_rn(v[j]);
            fence_async_shared();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(tm, tt, r0, col, u.e);
              bulk_commit();
            }
            buf ^= 1;
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
        if (!last) {
          // (a completed bulk store is ordered before what follows without a proxy fence)
          bulk_wait_all();
          // the last of the CTA's warps tells the others: releases and additions to one
          // address are dear (each warp for itself, 6 x 333 x 1001 111 us instead of 101).  (A
          // warp is at most two units ahead of another, so four units' counts do not meet)
          if ((add_cta(stored + (unit & 3) * 4, 1) & (kEpiWarps - 1)) == kEpiWarps - 1)
            add_release(args.counters + u.phase * args.batch + u.e, 1);
        }
      }
      __syncwarp();
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
      ++unit;
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  cluster_sync();
  // Before the CTAs may exit, every load that either has issued must have landed.
  if (leader && warp == 0 && lane == 0 &&
      !drain_pair_loads<STAGES>(full_bar, ld_shared_u32(issued_slot), ld_shared_u32(issued_slot + 4), kDrain))
    record_error(args.err, kErrTimeout);
  // Every MMA of the pair has completed once the drain barrier has seen the leader's
  // final commit; only then may tensor memory be freed and the CTAs exit.
  if (warp == 1 && lane == 0 && !mbar_wait(drain_bar, 0, 4 * tmo + kDrain)) record_error(args.err, kErrTimeout);
  __syncwarp();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc2(tmem_base, 512);
}

// The pairs that fit the device at once, asked for once per device; also allows the
// kernel its shared memory.
cudaError_t orth_pairs(int sms, int* pairs) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((*pairs = known[dev & 63].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  e = cudaFuncSetAttribute(orth_steps_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kOrthSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2));
  cfg.blockDim = dim3(kOrthThreads);
  cfg.dynamicSmemBytes = kOrthSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  e = cudaOccupancyMaxActiveClusters(&n, orth_steps_kernel, &cfg);
  if (e != cudaSuccess) return e;
  if (n < 1) return cudaErrorLaunchOutOfResources;
  *pairs = std::min(n, sms / 2);
  known[dev & 63].store(*pairs, std::memory_order_relaxed);
  return cudaSuccess;
}

cudaError_t launch_orth_steps(const OrthMaps& maps, const OrthArgs& args, int sms, cudaStream_t st) {
  int pairs = 0;
  const cudaError_t e = orth_pairs(sms, &pairs);
  if (e != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(args.steps) * args.batch * (2 * args.units_sym + args.units_upd);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<int64_t>(units, pairs)));
  cfg.blockDim = dim3(kOrthThreads);
  cfg.dynamicSmemBytes = kOrthSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeCooperative;
  attr[1].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, orth_steps_kernel, maps, args);
}

// ------------------------------------------------------------ narrow matrices
// m <= 128: a matrix stays in shared memory from its first read to the result, in one
// kernel.  A cluster of `ranks` CTAs takes a matrix, each CTA `chunks` blocks of 64
// columns of X [128 rows, zeros past m], in the 128-byte swizzle: one layout serves as
// the K-major operand of the gram and as the MN-major one of the update.
//   norm and load   from g, the squares joined over the cluster
//   gram            each CTA's columns; the CTAs' sums on and above the diagonal are added
//                   in a fixed order, a share of the rows by each, which hands it to all
//   poly            128 x 128 in every CTA; B as an fp16 value and what it leaves, so its
//                   rounding, the largest one's share of the error, falls away (the products
//                   are not what takes the time)
//   update          in place: a group of 256 columns is overwritten when its product
//                   is done
// What bounds it is the chain of dependent steps, not the products.  At most one CTA
// fits an SM (kSmallSmemMin): tensor memory of two clusters on shared SMs could each
// wait for the other's.
constexpr int kSmallThreads = 512;
constexpr int kChunkBytes = 128 * 128;            // 128 rows of 64 columns
constexpr int kMaxSmallChunks = 8;                // per CTA
constexpr int kSmallTail = 2 * kChunkBytes + 4 * kChunkBytes + 1024 + 512;   // A, P (or both parts of B), alignment, rest
constexpr int kSmallSmemMin = 120 * 1024;
constexpr int kSmallM = 128;
constexpr int kSmallN = 8 * kMaxSmallChunks * 64;   // on 8 CTAs
static_assert(kMaxSmallChunks * kChunkBytes + kSmallTail <= 232448, "shared memory budget");

struct OrthSmall {
  OrthIn in;
  int m, n, chunks, ranks, steps;
  float eps, S, out_scale;
  __nv_bfloat16* out;
  int64_t out_ld, out_stride;
  int vec;               // rows of out start on 16 bytes
  int* err;
  uint64_t timeout_ns;
  float coefs[kMaxOrthSteps][3];
};

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster4u(uint32_t addr, const uint4& u) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w) : "memory");
}
__device__ __forceinline__ void st_cluster1(uint32_t addr, float a) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(a) : "memory");
}

__device__ __forceinline__ void small_mma(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  tc_mma<false>(d_tmem, static_cast<uint64_t>(kDescHi) << 32 | a_lo, static_cast<uint64_t>(kDescHi) << 32 | b_lo, idesc, accumulate);
}

// Byte of element (row, column) in blocks of 64 columns in the 128-byte swizzle.
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return (c >> 6) * kChunkBytes + r * 128 + ((((c >> 3) & 7) ^ (r & 7)) << 4) + (c & 7) * 2;
}

// Eight of g's elements as X sees them: row r, columns c .. c + 7 (not FLIP), or rows
// r .. r + 7, column c (FLIP); 0 outside.
template <typename E, bool FLIP>
__device__ __forceinline__ void small_load8(const OrthIn& in, const E* g, int r, int c, float (&v)[8]) {
  const int gr = FLIP ? c : r, gc = FLIP ? r : c;
  if (gr < in.M && gc < in.N) {
    load_row8(in, g + gr * in.ld, gc, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.f;
  }
}

template <typename E, bool FLIP>
__global__ void __launch_bounds__(kSmallThreads, 1) orth_small_kernel(const __grid_constant__ OrthSmall a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ float part[3][32];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (sbase - raw);
  const uint32_t sX = sbase, sA = sX + a.chunks * kChunkBytes, sP = sA + 2 * kChunkBytes, sB = sP;
  const uint32_t bars = sP + 4 * kChunkBytes, slots = bars + 32, tmem_slot = bars + 24;
  uint8_t *gX = gbase, *gA = gbase + (sA - sbase);
  const float* gslots = reinterpret_cast<const float*>(gbase + (slots - sbase));   // [ranks][3]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = a.ranks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int e = blockIdx.x / a.ranks;
  const int width = a.chunks * 64, first = rank * width;   // this CTA's columns of X
  const E* g = static_cast<const E*>(a.in.g) + static_cast<int64_t>(e) * a.in.stride;

  if (tid == 0) {
    mbar_init(bars, 1);
    mbar_init(bars + 8, 1);
    mbar_init(bars + 16, 1);
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }

  // ---- norm and load: eight elements a thread; without FLIP neighbours along a row
  // of X, with it along g's rows, which are X's columns
  const int groups = FLIP ? 16 * width : 128 * (width / 8);
  auto at = [&](int i, int& r, int& c) {
    if (FLIP) {
      r = i / width * 8;
      c = i % width;
    } else {
      r = i / (width / 8);
      c = i % (width / 8) * 8;
    }
  };
  // up to 3 blocks of columns stay in registers between the two (groups is a multiple
  // of 2 kSmallThreads: 128 rows of a multiple of 64 columns)
  constexpr int U = 6;
  float v[U][8];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kSmallThreads;
      if (i < groups) {
        int r, c;
        at(i, r, c);
        small_load8<E, FLIP>(a.in, g, r, first + c, v[u]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[u][k] = 0.f;
      }
    }
  };
  Squares s;
  for (int i = tid; i < groups; i += U * kSmallThreads) {
    fetch(i);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < 8; ++k) s.add(v[u][k]);
  }
  s.mid = block_sum(s.mid, part[0]);
  s.big = block_sum(s.big, part[1]);
  s.small = block_sum(s.small, part[2]);
  if (a.ranks > 1) {
    // (a CTA of the cluster may be written to once all have started)
    cluster_sync();
    if (tid < a.ranks) {
      const uint32_t p = mapa_shared(slots + rank * 12, tid);
      st_cluster1(p, s.mid), st_cluster1(p + 4, s.big), st_cluster1(p + 8, s.small);
    }
    __syncwarp();
    cluster_sync();
    s = Squares{0.f, 0.f, 0.f};
    for (int k = 0; k < a.ranks; ++k)
      s.mid += gslots[3 * k], s.big += gslots[3 * k + 1], s.small += gslots[3 * k + 2];
  }
  const float2 f = orth_factor_of(s, a.eps, a.S);
  for (int i0 = tid; i0 < groups; i0 += U * kSmallThreads) {
    if (groups > U * kSmallThreads) fetch(i0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kSmallThreads;
      if (i >= groups) break;
      int r, c;
      at(i, r, c);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[u][k] = v[u][k] * f.x * f.y;
      if (FLIP) {
#pragma unroll
        for (int k = 0; k < 8; ++k) *reinterpret_cast<__half*>(gX + swz(r + k, c)) = __float2half_rn(v[u][k]);
      } else {
        st_shared_v4u(sX + swz(r, c), pack_half(v[u][0], v[u][1]), pack_half(v[u][2], v[u][3]),
                      pack_half(v[u][4], v[u][5]), pack_half(v[u][6], v[u][7]));
      }
    }
  }
  fence_async_shared();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + (tmem_slot - sbase));

  const int q = warp & 3, part_c = (warp >> 2) * 32;      // rows of this warp, and its columns of 128
  const int row = q * 32 + lane;
  const uint32_t tq = tmem + (static_cast<uint32_t>(q * 32) << 16);
  const int mc = (a.m + 15) & ~15;               // columns of A and B
  const uint32_t idesc_sym = (1u << 4) | (static_cast<uint32_t>(mc >> 3) << 17) | ((128u >> 4) << 24);
  const float S2 = a.S * a.S;
  // descriptors: X as the K-major and as the MN-major operand, A, B
  const uint32_t dX = desc_lo(sX, 16), dXn = desc_lo(sX, kChunkBytes), dA = desc_lo(sA, 16), dB = desc_lo(sB, 16);
  uint32_t phase[2] = {0, 0};
  auto wait = [&](int b) {
    if (!mbar_wait(bars + 8 * b, phase[b], a.timeout_ns)) record_error(a.err, kErrTimeout);
    phase[b] ^= 1u;
    tc_fence_after();
  };

  for (int step = 0; step < a.steps; ++step) {
    // ---- gram
    if (warp == 0 && elect_one()) {
#pragma unroll 1
      for (int c = 0; c < a.chunks; ++c) {
        const uint32_t d = dX + c * (kChunkBytes / 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) small_mma(tmem, d + 2 * k, d + 2 * k, idesc_sym, c + k != 0 ? 1u : 0u);
      }
      tc_commit(bars);
    }
    wait(0);
    if (part_c < mc) {
      const int c = part_c;
      float v[32];
      tmem_ld32(tq + c, v);
      if (a.ranks == 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          st_shared_v4u(sA + swz(row, c + 8 * j), pack_half(v[8 * j], v[8 * j + 1]), pack_half(v[8 * j + 2], v[8 * j + 3]),
                        pack_half(v[8 * j + 4], v[8 * j + 5]), pack_half(v[8 * j + 6], v[8 * j + 7]));
      } else {
        // rows of 512 bytes, 16-byte pieces at piece ^ (row & 7)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          st_shared_v4(sP + row * 512 + (((c >> 2) + j) ^ (row & 7)) * 16, v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      }
    }
    if (a.ranks > 1) {
      __syncwarp();
      cluster_sync();
      // this CTA's share of the rows, some of each 32: the ranks' sums from its own on
      // (all from rank 0 on, they wait for one another there: 0.8 us more a step), then to
      // all of them.  A lane takes four columns, with more than eight ranks two lanes take
      // the same four, of eight ranks each; two neighbours' sums are 16 bytes, which the
      // lanes that hold them send to a part of the ranks each.  Columns of the 32 x 32
      // blocks below the diagonal are not sent but mirrored where they arrive (0.8 us less
      // a step): what the cluster's network carries, 14 bytes a clock and SM, is what this
      // takes, by asynchronous copies too.
      const int rows = 128 / a.ranks, each = rows / 4;      // of a block of 32
      const bool halves = a.ranks > 8;
      for (int i = tid; i < (rows << (halves ? 6 : 5)); i += kSmallThreads) {   // (whole warps)
        const int o = i >> (halves ? 6 : 5), block = o / each, r = block * 32 + rank * each + o % each;
        const int p = halves ? (i >> 1 & 16) + (lane & 15) : lane, k0 = halves ? lane >> 4 << 3 : 0;
        const bool in = 4 * p < mc && p >= 8 * block;      // (rows past m are zeros, and wanted as such)
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
        const uint32_t from = sP + r * 512 + (p ^ (r & 7)) * 16;
        float4 x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          x[j] = in && k0 + j < a.ranks ? ld_cluster4(mapa_shared(from, (rank + k0 + j) & (a.ranks - 1)))
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 8; ++j) t.x += x[j].x, t.y += x[j].y, t.z += x[j].z, t.w += x[j].w;
        if (halves) {
          t.x += __shfl_xor_sync(0xffffffffu, t.x, 16), t.y += __shfl_xor_sync(0xffffffffu, t.y, 16);
          t.z += __shfl_xor_sync(0xffffffffu, t.z, 16), t.w += __shfl_xor_sync(0xffffffffu, t.w, 16);
        }
        const uint32_t u0 = pack_half(t.x, t.y), u1 = pack_half(t.z, t.w);
        const uint32_t v0 = __shfl_xor_sync(0xffffffffu, u0, 1), v1 = __shfl_xor_sync(0xffffffffu, u1, 1);
        const uint4 u = lane & 1 ? make_uint4(v0, v1, u0, u1) : make_uint4(u0, u1, v0, v1);
        const uint32_t to = sA + swz(r, 4 * (p & ~1));
        for (int k = halves ? (lane & 1) + (lane >> 4 << 1) : lane & 1; in && k < a.ranks; k += halves ? 4 : 2)
          st_cluster4u(mapa_shared(to, (rank + k) & (a.ranks - 1)), u);
      }
      __syncwarp();
      cluster_sync();
      // (what the others stored is behind the barrier, and before the fence below)
      // rows of the blocks below the diagonal, eight columns at a time
      for (int i = warp; i < 24; i += kSmallThreads / 32) {
        const int t = i >> 2, block = t < 1 ? 1 : (t < 3 ? 2 : 3);      // (1,0) (2,0) (2,1) (3,0) ..
        const int r = block * 32 + lane, c = (t - block * (block - 1) / 2) * 32 + (i & 3) * 8;
        if (block * 32 >= mc) break;
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          u[k] = r < mc ? *reinterpret_cast<const uint16_t*>(gA + swz(c + 2 * k, r)) |
                              static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(gA + swz(c + 2 * k + 1, r))) << 16
                        : 0u;
        st_shared_v4u(sA + swz(r, c), u[0], u[1], u[2], u[3]);
      }
      fence_async_shared();
      tc_fence_before();
      __syncthreads();
    } else {
      fence_async_shared();
      tc_fence_before();
      __syncthreads();
    }
    // ---- poly
    if (warp == 0 && elect_one()) {
      tc_fence_after();
#pragma unroll 1
      for (int k = 0; k < mc / 16; ++k) {
        const uint32_t d = dA + (k >> 2) * (kChunkBytes / 16) + 2 * (k & 3);
        small_mma(tmem + 128, d, d, idesc_sym, k != 0 ? 1u : 0u);
      }
      tc_commit(bars);
    }
    wait(0);
    const float cI = a.coefs[step][0] * S2, cA = a.coefs[step][1], cP = a.coefs[step][2] / S2;
    if (part_c < mc) {
      const int c = part_c;
      float v[32];
      tmem_ld32(tq + 128 + c, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 u = *reinterpret_cast<const uint4*>(gA + swz(row, c + 8 * j));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        uint32_t o[4], rest[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
          float b0 = fmaf(cA, x.x, cP * v[8 * j + 2 * k]), b1 = fmaf(cA, x.y, cP * v[8 * j + 2 * k + 1]);
          if (c == q * 32) {      // (the warp's diagonal block)
            if (lane == 8 * j + 2 * k) b0 += cI;
            if (lane == 8 * j + 2 * k + 1) b1 += cI;
          }
          const __half2 h = __floats2half2_rn(b0, b1);
          const float2 f = __half22float2(h);
          o[k] = *reinterpret_cast<const uint32_t*>(&h);
          rest[k] = pack_half(b0 - f.x, b1 - f.y);
        }
        st_shared_v4u(sB + swz(row, c + 8 * j), o[0], o[1], o[2], o[3]);
        st_shared_v4u(sB + 2 * kChunkBytes + swz(row, c + 8 * j), rest[0], rest[1], rest[2], rest[3]);
      }
    }
    fence_async_shared();
    tc_fence_before();
    __syncthreads();
    // ---- update: groups of 256 columns, the first into columns 256.. of the tensor
    // memory, the second into 0..255, where gram and poly are done with
    const int ngroups = (a.chunks + 3) >> 2;
    if (warp == 0 && elect_one()) {
      tc_fence_after();
#pragma unroll 1
      for (int b = 0; b < ngroups; ++b) {
        const int cols = min(256, width - 256 * b);
        const uint32_t idesc = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(cols >> 3) << 17) | ((128u >> 4) << 24);
        const uint32_t x = dXn + 4 * b * (kChunkBytes / 16);
#pragma unroll 1
        for (int k = 0; k < mc / 16; ++k) {
          const uint32_t d = dB + (k >> 2) * (kChunkBytes / 16) + 2 * (k & 3);
          // B's fp16 values, and what they left
          small_mma(tmem + 256 * (1 - b), d, x + k * 128, idesc, k != 0 ? 1u : 0u);
          small_mma(tmem + 256 * (1 - b), d + 2 * (kChunkBytes / 16), x + k * 128, idesc, 1u);
        }
        tc_commit(bars + 8 * b);
      }
    }
    const bool last = step + 1 == a.steps;
    const float ds = (last ? a.out_scale : 1.f) / S2;
#pragma unroll 1
    for (int b = 0; b < ngroups; ++b) {
      wait(b);
      const int cols = min(256, width - 256 * b);
#pragma unroll 1
      for (int c = part_c; c < cols; c += 128) {
        float v[32];
        tmem_ld32(tq + 256 * (1 - b) + c, v);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] *= ds;
        const int xc = 256 * b + c;
        if (!last) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            st_shared_v4u(sX + swz(row, xc + 8 * j), pack_half(v[8 * j], v[8 * j + 1]), pack_half(v[8 * j + 2], v[8 * j + 3]),
                          pack_half(v[8 * j + 4], v[8 * j + 5]), pack_half(v[8 * j + 6], v[8 * j + 7]));
        } else if (FLIP && a.vec) {
          // a warp's rows lie side by side: two lanes' rows of every other column each
          const int col = first + xc, live = a.n - col, odd = lane & 1, r = row & ~1;
          __nv_bfloat16* o = a.out + e * a.out_stride + static_cast<int64_t>(col + odd) * a.out_ld + r;
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float other = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
            const uint32_t u = odd ? pack_bf16(other, v[j + 1]) : pack_bf16(v[j], other);
            if (j + odd < live) {
              if (r + 1 < a.m)
                *reinterpret_cast<uint32_t*>(o) = u;
              else if (r < a.m)
                *o = __ushort_as_bfloat16(static_cast<uint16_t>(u));
            }
            o += 2 * a.out_ld;
          }
        } else if (row < a.m) {
          const int col = first + xc, live = a.n - col;    // columns that exist, from here
          __nv_bfloat16* out = a.out + e * a.out_stride;
          if (FLIP) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j < live) out[static_cast<int64_t>(col + j) * a.out_ld + row] = __float2bfloat16_rn(v[j]);
          } else {
            __nv_bfloat16* o = out + static_cast<int64_t>(row) * a.out_ld + col;
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              if (a.vec && j + 8 <= live) {
                store8(o + j, v + j);
              } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  if (j + k < live) o[j + k] = __float2bfloat16_rn(v[j + k]);
              }
            }
          }
        }
      }
    }
    fence_async_shared();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  // every product has completed before the tensor memory is given back
  if (warp == 0) {
    if (elect_one()) tc_commit(bars + 16);
    if (!mbar_wait(bars + 16, 0, 1000000000ull)) record_error(a.err, kErrTimeout);
  }
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// CTAs per matrix: the number with the least time.  Measured, five steps at m = 128: 16
// us, 4.4 for each block of 64 columns of a CTA, and 17 + r / 5 for the exchanges in a
// cluster of r (512 columns: 51.4 us on one CTA, 41.3 on 4, 40.3 on 8; 2048: 53.5 on 8,
// 45.4 on 16).  Matrices that do not fit at once go in waves (8 of 128 x 2880: 98 us on 16
// CTAs each, of which this GPU holds 7, 62 on 8).
constexpr int kRankLogs = 5;      // 1, 2, 4, 8, 16
void orth_small_ranks(OrthSmall* a, int batch, const int (&clusters)[kRankLogs]) {
  double least = 1e300;
  for (int log = 0; log < kRankLogs; ++log) {
    const int r = 1 << log, chunks = (a->n + 64 * r - 1) / (64 * r);
    if (chunks > kMaxSmallChunks || clusters[log] == 0) continue;
    const double waves = std::ceil(static_cast<double>(batch) / clusters[log]);
    const double t = waves * (16 + 4.4 * chunks + (r > 1 ? 17 + 0.2 * r : 0));
    if (t < least) least = t, a->ranks = r, a->chunks = chunks;
  }
}

template <typename E, bool FLIP>
cudaError_t launch_orth_small(OrthSmall& a, int batch, int sms, cudaStream_t st) {
  auto kern = orth_small_kernel<E, FLIP>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  constexpr int kMost = kMaxSmallChunks * kChunkBytes + kSmallTail;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(kSmallThreads);
  // the clusters of each size that fit the device at once, asked for once per device
  static std::atomic<int> known[64][kRankLogs];
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    known[dev & 63][0].store(sms, std::memory_order_relaxed);
    for (int log = 1; log < kRankLogs; ++log) {
      cfg.gridDim = dim3(sms >> log << log);
      cfg.dynamicSmemBytes = kMost;
      attr[0].val.clusterDim.x = 1 << log;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) (void)cudaGetLastError(), n = 0;
      known[dev & 63][log].store(n, std::memory_order_relaxed);
    }
    ready.fetch_or(bit, std::memory_order_release);
  }
  int clusters[kRankLogs];
  for (int log = 0; log < kRankLogs; ++log) clusters[log] = known[dev & 63][log].load(std::memory_order_relaxed);
  a.ranks = 0;
  orth_small_ranks(&a, batch, clusters);
  if (a.ranks == 0) return cudaErrorLaunchOutOfResources;
  cfg.gridDim = dim3(static_cast<unsigned>(batch * a.ranks));
  cfg.dynamicSmemBytes = std::max(kSmallSmemMin, a.chunks * kChunkBytes + kSmallTail);
  cfg.stream = st;
  attr[0].val.clusterDim.x = a.ranks;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

// ------------------------------------------------------------ host
constexpr int kMaxOrthSide = 65536;
const float kDefaultCoefs[3] = {3.4445f, -4.7750f, 2.0315f};

struct OrthPlan {
  int m, n;            // m <= n
  int flip;
  int ldx, lda;
  int nparts, part_rows;
  int chunk;           // matrices per launch
  int small;           // narrow matrices: orth_small_kernel
  size_t counters, parts, x[2], a, b, total;
};

int64_t round8(int64_t v) { return (v + 7) & ~static_cast<int64_t>(7); }

// Tiles of a symmetric m x m result with column tiles of bn: those from the diagonal
// 256 x 256 block on.
int64_t sym_units(int64_t m, int bn) {
  const int64_t mt = (m + 255) / 256, nt = (m + bn - 1) / bn, f = 256 / bn;
  return mt * nt - f * mt * (mt - 1) / 2;
}

// Matrices go through in chunks of about kChunkUnits tiles of a product and at most
// kChunkBytesMax of workspace (or one matrix's), so the workspace does not grow with E.
constexpr int kChunkUnits = 1200;
constexpr int64_t kChunkBytesMax = 1ll << 30;

// The limit of a wait, of which the kernels take up to four at once.
uint64_t orth_limit() { return std::min<uint64_t>(abi_wait_timeout_ns(), 1ull << 60); }

bool orth_plan(int64_t E, int64_t M, int64_t N, OrthPlan* p) {
  if (E < 0 || M < 1 || N < 1 || M > kMaxOrthSide || N > kMaxOrthSide) return false;
  p->flip = M > N;
  p->m = static_cast<int>(std::min(M, N));
  p->n = static_cast<int>(std::max(M, N));
  p->ldx = static_cast<int>(round8(p->n));
  p->lda = static_cast<int>(round8(p->m));
  p->small = 0;
  if (p->m <= kSmallM && p->n <= kSmallN) {
    p->small = 1;
    p->chunk = 1 << 24;
    p->total = 256;
    return true;
  }
  const int64_t units = sym_units(p->m, 256);
  const int64_t bytes = 4ll * p->m * (p->ldx + p->lda);      // of a matrix: X twice, A and B
  p->chunk = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({E, (kChunkUnits + units - 1) / units, kChunkBytesMax / bytes})));
  const int64_t want = std::min<int64_t>((M * N + kNormElems - 1) / kNormElems, kNormBlocks / p->chunk);
  p->nparts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({want, M, kMaxParts})));
  p->part_rows = static_cast<int>((M + p->nparts - 1) / p->nparts);
  p->nparts = static_cast<int>((M + p->part_rows - 1) / p->part_rows);
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += abi_align256(bytes);
    return o;
  };
  const size_t C = p->chunk;
  p->counters = take(sizeof(int) * 3 * kMaxOrthSteps * C);
  // (N x M takes what M x N takes)
  p->parts = take(sizeof(Squares) * C * static_cast<size_t>(std::max<int64_t>(1, std::min<int64_t>({want, p->n, kMaxParts}))));
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

bool rows_on_16(const void* p, int es, int64_t ld, int64_t stride, int batch) {
  const int W = 16 / es;
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % W == 0 && (batch == 1 || stride % W == 0);
}

OrthIn orth_in(const void* g, int32_t dtype, int64_t e0, int batch, int64_t M, int64_t N, int64_t ld, int64_t stride) {
  const int es = dtype == MOE_FP32 ? 4 : 2;
  const char* p = static_cast<const char*>(g) + e0 * stride * es;
  return OrthIn{p, ld, stride, static_cast<int>(M), static_cast<int>(N), rows_on_16(p, es, ld, stride, batch)};
}

// Width of the column tiles of a product with kb blocks of K: the one with the least time,
// in cycles.  A block takes 512 (bound by the products), 328 or 296 (narrower tiles are
// bound by what the producer and the issuer do for a block); beside them, once,
// the start, the last tile's results (twice as many to store where they are mirrored) and the
// word to the next phase.  One matrix alone waits for each phase's last tiles, several fill
// one another's gaps, from the second round on.  (8 x 1000 x 1000: 256 columns for both
// kinds 278 us, 128 for the symmetric ones 248; 32 x 140 x 500: 128 and 256 99, 64 and 128 90.)
template <typename F>
int orth_width(const F& units, int batch, int pairs, double kb, bool sym) {
  int best = 256;
  double least = 1e300;
  for (int bn = 256; bn >= 64; bn /= 2) {
    double waves = static_cast<double>(units(bn)) * batch / pairs;
    if (batch == 1)
      waves = std::ceil(waves);
    else if (waves < 2)
      waves = waves <= 1 ? 1 : waves + 0.3 * (2 - waves);
    const double block = bn == 256 ? 512 : bn == 128 ? 328 : 296;
    const double once = bn == 64 ? 4500 : bn == 128 ? (sym ? 6000 : 5600) : (sym ? 10000 : 7000);
    const double t = waves * kb * block + once;
    if (t < least) least = t, best = bn;
  }
  return best;
}

void orth_tiles(OrthArgs* a, int pairs) {
  const auto upd = [&](int bn) { return static_cast<int64_t>(a->mt) * ((a->n + bn - 1) / bn); };
  const double kb_m = (a->m + 63) / 64, kb_n = (a->n + 63) / 64;
  int bn = orth_width([&](int w) { return sym_units(a->m, w); }, a->batch, pairs, (kb_n + kb_m) / 2, true);
  a->bn_sym = bn, a->nt_sym = (a->m + bn - 1) / bn;
  a->units_sym = static_cast<int>(sym_units(a->m, bn));
  bn = orth_width(upd, a->batch, pairs, kb_m, false);
  a->bn_upd = bn, a->nt_upd = (a->n + bn - 1) / bn;
  a->units_upd = static_cast<int>(upd(bn));
}

bool orth_maps(OrthMaps* t, const OrthPlan& p, const OrthArgs& a, __half* const* x, const __half* A, const __half* B) {
  const auto SW = CU_TENSOR_MAP_SWIZZLE_128B, SW64 = CU_TENSOR_MAP_SWIZZLE_64B, NOSW = CU_TENSOR_MAP_SWIZZLE_NONE;
  const uint64_t m = p.m, n = p.n, C = a.batch, lda = p.lda;
  const uint32_t bs = a.bn_sym / 2;
  bool ok = true;
  for (int i = 0; i < 2; ++i)
    ok = ok && abi_map_half(&t->xk[i], x[i], n, m, C, p.ldx, 64, 128, SW) &&
         abi_map_half(&t->xs[i], x[i], n, m, C, p.ldx, 64, bs, SW) &&
         abi_map_half(&t->xn[i], x[i], n, m, C, p.ldx, 64, 64, SW) &&
         abi_map_half(&t->xo[i], x[i], n, m, C, p.ldx, 32, 32, SW64);
  return ok && abi_map_half(&t->ak, A, m, m, C, lda, 64, 128, SW) && abi_map_half(&t->as, A, m, m, C, lda, 64, bs, SW) &&
         abi_map_half(&t->ao, A, m, m, C, lda, 32, 32, SW64) && abi_map_half(&t->at, A, m, m, C, lda, 32, 32, NOSW) &&
         abi_map_half(&t->bk, B, m, m, C, lda, 64, 128, SW) && abi_map_half(&t->bo, B, m, m, C, lda, 32, 32, SW64) &&
         abi_map_half(&t->bt, B, m, m, C, lda, 32, 32, NOSW);
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
  // (scale / S^3 is to be a normal number)
  if (scale != 0.f && std::fabs(scale) < 0x1p-100f) return MOE_ERR_INVALID_ARG;
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
  if (p.small) {
    OrthSmall a = {};
    a.m = p.m, a.n = p.n, a.steps = steps;
    a.eps = eps, a.S = S, a.out_scale = scale / S;
    a.out_ld = out_ld, a.out_stride = out_stride;
    a.err = static_cast<int*>(ws);
    a.timeout_ns = orth_limit();
    for (int i = 0; i < steps; ++i)
      for (int k = 0; k < 3; ++k) a.coefs[i][k] = coefs ? coefs[3 * i + k] : kDefaultCoefs[k];
    for (int64_t e0 = 0; e0 < E; e0 += p.chunk) {
      const int batch = static_cast<int>(std::min<int64_t>(p.chunk, E - e0));
      a.in = orth_in(g, dtype, e0, batch, M, N, g_ld, g_stride);
      a.out = static_cast<__nv_bfloat16*>(out) + e0 * out_stride;
      a.vec = rows_on_16(a.out, 2, out_ld, out_stride, batch);
      const cudaError_t e = abi_tracked(kAbiOrthSmall, 1, st, [&] {
        if (dtype == MOE_FP32)
          return p.flip ? launch_orth_small<float, true>(a, batch, sms, st) : launch_orth_small<float, false>(a, batch, sms, st);
        return p.flip ? launch_orth_small<__nv_bfloat16, true>(a, batch, sms, st)
                      : launch_orth_small<__nv_bfloat16, false>(a, batch, sms, st);
      });
      if (e != cudaSuccess) return MOE_ERR_CUDA;
    }
    return MOE_OK;
  }
  char* w = static_cast<char*>(ws);
  Squares* parts = reinterpret_cast<Squares*>(w + p.parts);
  int* counters = reinterpret_cast<int*>(w + p.counters);
  __half* x[2] = {reinterpret_cast<__half*>(w + p.x[0]), reinterpret_cast<__half*>(w + p.x[1])};
  __half* a = reinterpret_cast<__half*>(w + p.a);
  __half* b = reinterpret_cast<__half*>(w + p.b);
  OrthArgs args = {};
  args.m = p.m, args.n = p.n, args.steps = steps;
  args.mt = (p.m + 255) / 256;
  args.S2 = S * S, args.inv_S2 = 1.f / args.S2, args.out_scale = scale / S;
  args.A = a, args.lda = p.lda, args.astride = static_cast<int64_t>(p.m) * p.lda;
  args.out_ld = out_ld, args.out_stride = out_stride, args.flip = p.flip;
  args.counters = counters;
  args.err = static_cast<int*>(ws);
  args.timeout_ns = orth_limit();
  for (int i = 0; i < steps; ++i)
    for (int k = 0; k < 3; ++k) args.coefs[i][k] = coefs ? coefs[3 * i + k] : kDefaultCoefs[k];
  for (int64_t e0 = 0; e0 < E; e0 += p.chunk) {
    const int batch = static_cast<int>(std::min<int64_t>(p.chunk, E - e0));
    const OrthIn in = orth_in(g, dtype, e0, batch, M, N, g_ld, g_stride);
    cudaError_t e = abi_tracked(kAbiOrthLoad, 2, st, [&] {
      if (dtype == MOE_FP32)
        orth_norm_kernel<float><<<dim3(p.nparts, batch), kNormThreads, 0, st>>>(in, p.part_rows, parts);
      else
        orth_norm_kernel<__nv_bfloat16><<<dim3(p.nparts, batch), kNormThreads, 0, st>>>(in, p.part_rows, parts);
      cudaError_t r = cudaGetLastError();
      if (r != cudaSuccess) return r;
      const int64_t tiles = ((M + 63) / 64) * ((N + 63) / 64);
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(tiles, (sms * 8 + batch - 1) / batch)), batch);
      cfg.blockDim = dim3(256);
      cfg.stream = st;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      auto go = [&](auto kern) {
        return cudaLaunchKernelEx(&cfg, kern, in, static_cast<const Squares*>(parts), p.nparts, eps, S, x[0], p.ldx,
                                  static_cast<int64_t>(p.m) * p.ldx, counters, 3 * steps * batch);
      };
      if (dtype == MOE_FP32) return p.flip ? go(orth_load_kernel<float, true>) : go(orth_load_kernel<float, false>);
      return p.flip ? go(orth_load_kernel<__nv_bfloat16, true>) : go(orth_load_kernel<__nv_bfloat16, false>);
    });
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    args.batch = batch;
    orth_tiles(&args, sms / 2);
    args.out = static_cast<__nv_bfloat16*>(out) + e0 * out_stride;
    args.vec = rows_on_16(args.out, 2, out_ld, out_stride, batch);
    OrthMaps maps;
    if (!orth_maps(&maps, p, args, x, a, b)) return MOE_ERR_CUDA;
    e = abi_tracked(kAbiOrthSteps, 1, st, [&] { return launch_orth_steps(maps, args, sms, st); });
    if (e != cudaSuccess) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
