// The whole expert layer for a few tokens, in two kernels:
//
//   gate_up:  a[s]  = act(x[s / k] Wgu[e_s] (+ b_gate_up))      for every slot s
//   down:     y[t]  = sum_j w[t,j] (a[t k + j] Wd[e] (+ b_down))
//
// With a few rows per expert the layer reads each touched expert's weights once
// and does next to nothing with them: it is bound by HBM, not by the tensor
// cores.  So the weights go from global memory straight into registers, as
// operands of warp-level matrix instructions (weights on the 16-row side, up to
// 8 tokens per instruction on the other), with no shared-memory ring between,
// and everything else is arranged to keep loads in flight and every SM busy to
// the end:
//
// Work.  A unit is (expert and up to 8 NT of its rows, tile of weight columns)
// and takes KS steps along the contraction.  All units' steps, laid end to end,
// are cut into equal runs, one per block (two blocks per SM), so a single token
// on four experts spreads as evenly as a batch on all of them.  A unit cut by a
// run's end is summed from its blocks' parts, in block order, by the block that
// finishes last: the same bits every time.  The down kernel joins the parts, the
// k experts and the routing weights of a column tile in one such step.
//
// Dispatch.  Every block builds the plan it needs from topk_idx in shared
// memory (a stable counting sort of at most 4096 slots), so there is no plan
// kernel and no gather.  The down kernel does this while the gate_up kernel
// ends (programmatic launch), and waits only before it reads a.
//
// Precision.  Products accumulate in fp32.  a is rounded to bf16 between the
// kernels for bf16 storage, as the layer for many tokens does (it is an operand
// of the bf16 product); it stays fp32 for fp32 storage, whose products run in
// fp32 on the CUDA cores.
#include <algorithm>
#include <atomic>

#include "abi_internal.h"
#include "common.cuh"
#include "mx.cuh"
#include "vec.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 128;
constexpr int kMaxSlots = kMaxTokens * 32;   // k <= 32
constexpr int kMaxE = 1024;
constexpr int kMaxChunks = kMaxE + kMaxSlots / 8;
constexpr int kMaxGrid = 512;
constexpr int kNowhere = 0xffff;
// the largest plan_bytes(): every chunk, slot and expert there can be
constexpr int kMostPlanBytes = 4 * kMaxChunks + 4 * kMaxE + 6 * kMaxChunks + 4 * kMaxSlots + 64;
static_assert(kMaxChunks * 32 < kNowhere, "a slot's place fits 16 bits");

struct FewArgs {
  const void* x;
  const uint8_t* x_scale;
  const int* idx;
  const float* topk_w;
  const void* w;           // this kernel's weights, or codes
  const uint8_t* scales;   // the codes' scale bytes
  const void* bias;        // this kernel's bias, or null
  void* act;               // [Tk, I]
  float* part;             // parts of cut units: 2 per block
  float* o;                // [Tk, H] products of whole units
  void* y;
  unsigned* counters;      // this kernel's; 0 between calls
  int* err;
  int T, H, I, E, k, rows, act_kind, interleaved, out_fp32;   // rows: of a chunk
  float limit, alpha;
};

// ------------------------------------------------------------------ plan
// A chunk is up to `rows` (8 or 32) rows of one expert; chunks are ordered by
// expert, rows by slot.
// Its arrays lie in dynamic shared memory, sized for the call (what they do not
// take is L1 cache for the token rows).
struct Plan {
  uint16_t* slot;         // [Tk] slots in the order of the rows
  uint16_t* where;        // [Tk] a slot's chunk * 32 + row in it; kNowhere: bad id
  uint16_t* chunk_e;      // [chunks_max]
  uint16_t* chunk_first;  // [chunks_max]
  uint16_t* chunk_rows;   // [chunks_max]
  uint32_t* span;         // [chunks_max] down kernel: a unit's blocks, see combine
  uint32_t* off;          // [E] scratch: the experts' first chunk << 16 | first row
  int chunks;
};
struct PlanSmall {
  uint32_t warp[8];
  int chunks;
  int last[2];
};

__host__ __device__ __forceinline__ int chunks_max(int Tk, int E, int rows) {
  return (Tk < E ? Tk : E) + Tk / rows;
}
__host__ __device__ __forceinline__ int plan_bytes(int Tk, int E, int rows) {
  const int c = (chunks_max(Tk, E, rows) + 1) & ~1, s = (Tk + 1) & ~1;
  return (4 * c + 4 * (Tk <= 32 ? 0 : E) + 2 * 3 * c + 2 * 2 * s + 15) & ~15;
}
__device__ __forceinline__ Plan plan_at(void* base, int Tk, int E, int rows) {
  const int c = (chunks_max(Tk, E, rows) + 1) & ~1, s = (Tk + 1) & ~1;
  Plan p;
  p.span = static_cast<uint32_t*>(base);
  p.off = p.span + c;
  p.chunk_e = reinterpret_cast<uint16_t*>(p.off + (Tk <= 32 ? 0 : E));
  p.chunk_first = p.chunk_e + c;
  p.chunk_rows = p.chunk_first + c;
  p.slot = p.chunk_rows + c;
  p.where = p.slot + s;
  p.chunks = 0;
  return p;
}

// One warp, a slot per lane: positions by counting.
__device__ __forceinline__ void build_plan_warp(const Plan& p, PlanSmall& ps,
                                                const int* __restrict__ idx, int Tk, int E,
                                                int rows, int* err) {
  const int lane = threadIdx.x & 31;
  int e = lane < Tk ? __ldg(idx + lane) : E;
  if (lane < Tk && (e < 0 || e >= E)) {
    record_error(err, kErrBadIndex);
    e = E;                                     // sorts last
  }
  const unsigned same = __match_any_sync(0xffffffffu, e);
  const int rank = __popc(same & ((1u << lane) - 1u));
  const int pos_e = e * 32 + lane;             // order of the rows
  const bool head = e < E && rank % rows == 0; // a chunk's first row
  const int head_key = head ? pos_e : 0x7fffffff;
  int pos = 0, heads = 0;
  for (int i = 0; i < Tk; ++i) {
    const int o = __shfl_sync(0xffffffffu, pos_e, i), h = __shfl_sync(0xffffffffu, head_key, i);
    pos += o < pos_e;
    heads += h <= pos_e;
  }
  if (lane < Tk) p.where[lane] = static_cast<uint16_t>(e < E ? (heads - 1) * 32 + rank % rows : kNowhere);
  if (e < E) p.slot[pos] = static_cast<uint16_t>(lane);
  if (head) {
    p.chunk_e[heads - 1] = static_cast<uint16_t>(e);
    p.chunk_first[heads - 1] = static_cast<uint16_t>(pos);
    p.chunk_rows[heads - 1] = static_cast<uint16_t>(min(rows, __popc(same) - rank));
  }
  const unsigned hb = __ballot_sync(0xffffffffu, head);
  if (lane == 0) ps.chunks = __popc(hb);
}

// All blocks build the same plan.
__device__ __forceinline__ void build_plan(Plan& p, PlanSmall& ps, const int* __restrict__ idx, int Tk,
                                           int E, int rows, int* err) {
  const int tid = threadIdx.x, lane = tid & 31;
  if (Tk <= 32) {
    if (tid < 32) build_plan_warp(p, ps, idx, Tk, E, rows, err);
    __syncthreads();
    p.chunks = ps.chunks;
    return;
  }
  for (int e = tid; e < E; e += kThreads) p.off[e] = 0;
  for (int s = tid; s < Tk; s += kThreads) {
    const int e = __ldg(idx + s);
    const bool ok = e >= 0 && e < E;
    if (!ok) record_error(err, kErrBadIndex);
    p.slot[s] = static_cast<uint16_t>(ok ? e : kNowhere);   // the expert, for now
  }
  __syncthreads();
  if (tid < 32) {
    for (int s0 = 0; s0 < Tk; s0 += 32) {
      const int s = s0 + lane;
      const int e = s < Tk ? p.slot[s] : kNowhere;
      const unsigned same = __match_any_sync(0xffffffffu, e);
      const int before = __popc(same & ((1u << lane) - 1u));
      uint32_t base = 0;
      if (e != kNowhere) base = p.off[e];
      __syncwarp();
      if (e != kNowhere) {
        p.where[s] = static_cast<uint16_t>(base + before);   // the row within the expert, for now
        if (before == 0) p.off[e] = base + __popc(same);
      }
      __syncwarp();
    }
  }
  __syncthreads();
  // exclusive scan over the experts, four per thread
  uint32_t v[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = tid * 4 + i;
    const uint32_t c = e < E ? p.off[e] : 0;
    v[i] = sum;
    sum += c | (((c + rows - 1) / rows) << 16);
  }
  uint32_t inc = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) ps.warp[tid >> 5] = inc;
  // the slots' experts move to registers: their array takes the sorted slots
  uint16_t mine[kMaxSlots / kThreads];
#pragma unroll
  for (int i = 0; i < kMaxSlots / kThreads; ++i)
    if (tid + i * kThreads < Tk) mine[i] = p.slot[tid + i * kThreads];
  __syncthreads();
  uint32_t base = inc - sum;
  for (int w = 0; w < (tid >> 5); ++w) base += ps.warp[w];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = tid * 4 + i;
    if (e < E) {
      const uint32_t b = base + v[i];
      const uint32_t end = base + (i < 3 ? v[i + 1] : sum);
      p.off[e] = b;
      const int first = b & 0xffffu, c0 = b >> 16, n = static_cast<int>(end & 0xffffu) - first;
      for (int c = 0; c * rows < n; ++c) {
        p.chunk_e[c0 + c] = static_cast<uint16_t>(e);
        p.chunk_first[c0 + c] = static_cast<uint16_t>(first + c * rows);
        p.chunk_rows[c0 + c] = static_cast<uint16_t>(min(rows, n - c * rows));
      }
      if (e == E - 1) ps.chunks = static_cast<int>(end >> 16);
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMaxSlots / kThreads; ++i) {
    const int s = tid + i * kThreads;
    if (s < Tk) {
      int at = kNowhere;
      if (mine[i] != kNowhere) {
        const uint32_t o = p.off[mine[i]];
        const int r = p.where[s];
        p.slot[(o & 0xffffu) + r] = static_cast<uint16_t>(s);
        at = (static_cast<int>(o >> 16) + r / rows) * 32 + r % rows;
      }
      p.where[s] = static_cast<uint16_t>(at);
    }
  }
  __syncthreads();
  p.chunks = ps.chunks;
}

// Adds to a counter after the block's earlier writes, and before its later reads.
__device__ __forceinline__ unsigned join_add(unsigned* p, unsigned v) {
  unsigned old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

// ------------------------------------------------------------------ products
// Each kind of weight: FG column groups of WF columns by KG shares of the
// contraction make the block's eight warps; a step takes STEP values of the
// contraction per warp.  Lane (g, t) = (lane / 4, lane % 4) holds weight columns
// of row group g and every fourth part of the contraction, in whatever order
// suits the loads: the token side uses the same order.

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weights: read once, never written by the layer.
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Token rows and activations.  The down kernel reads what the gate_up kernel
// wrote while it was already running, so these are plain loads in program order,
// after its wait.
__device__ __forceinline__ uint32_t ld_u32(const void* p) {
  uint32_t v;
  asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_u64(const void* p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_u128(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Two e4m3 codes times a power-of-two scale as bf16 (exact but for results below
// bf16's normal range).
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t two, float scale) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xffffu), __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  return pack_bf16(f.x * scale, f.y * scale);
}

// A token row (or a slot's activations) as the product reads it.
template <bool X8>
struct Row {
  const void* p = nullptr;             // null: no such row, zeros
  const uint8_t* scale = nullptr;
  __device__ __forceinline__ uint2 bf16x4(int k) const {
    if (!p) return make_uint2(0, 0);
    if (!X8) return ld_u64(static_cast<const __nv_bfloat16*>(p) + k);
    const uint32_t c = ld_u32(static_cast<const uint8_t*>(p) + k);
    const float s = mx_scale(__ldg(scale + (k >> 5)));
    return make_uint2(e4m3_pair(c, s), e4m3_pair(c >> 16, s));
  }
  __device__ __forceinline__ uint4 bf16x8(int k) const {
    if (!p) return make_uint4(0, 0, 0, 0);
    if (!X8) return ld_u128(static_cast<const __nv_bfloat16*>(p) + k);
    const uint2 c = ld_u64(static_cast<const uint8_t*>(p) + k);
    const float s = mx_scale(__ldg(scale + (k >> 5)));
    return make_uint4(e4m3_pair(c.x, s), e4m3_pair(c.x >> 16, s), e4m3_pair(c.y, s),
                      e4m3_pair(c.y >> 16, s));
  }
  __device__ __forceinline__ float4 f32x4(int k) const {
    if (!X8) {
      const uint4 v = ld_u128(static_cast<const float*>(p) + k);
      return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                         __uint_as_float(v.w));
    }
    const uint32_t c = ld_u32(static_cast<const uint8_t*>(p) + k);
    const float s = mx_scale(__ldg(scale + (k >> 5)));
    const float2 lo = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(c & 0xffffu), __NV_E4M3)));
    const float2 hi = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(c >> 16), __NV_E4M3)));
    return make_float4(lo.x * s, lo.y * s, hi.x * s, hi.y * s);
  }
};

// A block of 32 values of a token row as it lies in memory, for use a little later.
template <bool X8>
struct RawBlock {
  uint4 v[X8 ? 2 : 4];
  uint32_t byte;
  __device__ __forceinline__ void load(const Row<X8>& r, int b, bool ok) {
    const bool in = ok && r.p;
#pragma unroll
    for (int i = 0; i < (X8 ? 2 : 4); ++i)
      v[i] = in ? ld_u128(static_cast<const uint8_t*>(r.p) + (X8 ? 32 : 64) * static_cast<int64_t>(b) + 16 * i)
                : make_uint4(0, 0, 0, 0);
    byte = X8 && in ? __ldg(r.scale + b) : 127u;
  }
  __device__ __forceinline__ uint4 bf16x8(int q) const {
    if (!X8) return v[q % (X8 ? 2 : 4)];
    const uint4& c = v[(q >> 1) % 2];
    const uint32_t lo = q & 1 ? c.z : c.x, hi = q & 1 ? c.w : c.y;
    const float s = mx_scale(byte);
    return make_uint4(e4m3_pair(lo, s), e4m3_pair(lo >> 16, s), e4m3_pair(hi, s), e4m3_pair(hi >> 16, s));
  }
};

// bf16 weights [K, ld], columns innermost.  A lane loads 16 bytes (8 columns) of
// four rows of the contraction; pairs along the contraction, as the instruction
// wants them, come from two rows by byte permutes.  Columns 2 i and 2 i + 1 of
// the lane are rows g and g + 8 of instruction i.
struct Bf16 {
  using Store = __nv_bfloat16;
  static constexpr int WF = 64, FG = 2, KG = 4, STEP = 16;
  static constexpr int PITCH = FG * WF + 1;   // of the results [row][column] in shared memory
  static constexpr bool kRowPerLane = true;   // lane (g, t) reads rows g, g + 8, ...
  template <int NT, bool X8>
  static __device__ __forceinline__ void run(const void* w, const uint8_t*, int64_t ld, int col,
                                             int ncol, int K, int s0, int s1, int kg,
                                             const Row<X8>* rows, int, float* red) {
    constexpr int U = NT <= 2 ? 2 : 1;   // steps per buffer; two buffers take turns
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float acc[4][NT][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][n][q] = 0.f;
    const bool col_ok = 8 * g < ncol;
    const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(w) + col + 8 * g;
    uint4 v[2][U][4];
    uint2 xb[2][U][NT];
    auto load = [&](int buf, int s) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = ((s + u) * KG + kg) * STEP + 4 * t;
        const bool ok = s + u < s1 && k < K;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          v[buf][u][r] = ok && col_ok ? ldg_stream(base + (k + r) * ld) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int n = 0; n < NT; ++n) xb[buf][u][n] = ok ? rows[n].bf16x4(k) : make_uint2(0, 0);
      }
    };
    auto multiply = [&](int buf) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t* w0 = &v[buf][u][0].x;
        const uint32_t* w1 = &v[buf][u][1].x;
        const uint32_t* w2 = &v[buf][u][2].x;
        const uint32_t* w3 = &v[buf][u][3].x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a0 = __byte_perm(w0[i], w1[i], 0x5410), a1 = __byte_perm(w0[i], w1[i], 0x7632);
          const uint32_t a2 = __byte_perm(w2[i], w3[i], 0x5410), a3 = __byte_perm(w2[i], w3[i], 0x7632);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(acc[i][n], a0, a1, a2, a3, xb[buf][u][n].x, xb[buf][u][n].y);
        }
      }
    };
    load(0, s0);
    for (int s = s0; s < s1; s += 2 * U) {
      load(1, s + U);
      multiply(0);
      load(0, s + 2 * U);
      multiply(1);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float* d = red + (8 * n + 2 * t) * PITCH + 8 * g + 2 * i;
        d[0] = acc[i][n][0], d[PITCH] = acc[i][n][1];
        d[1] = acc[i][n][2], d[PITCH + 1] = acc[i][n][3];
      }
  }
};

// fp32 weights [K, ld]: the same loads (4 columns per lane), products on the
// CUDA cores in fp32; the four lanes of a group hold shares of the contraction.
struct F32 {
  using Store = float;
  static constexpr int WF = 32, FG = 2, KG = 4, STEP = 16;
  static constexpr int PITCH = FG * WF + 1;   // of the results [row][column] in shared memory
  static constexpr bool kRowPerLane = false;   // every lane reads all rows
  template <int NT, bool X8>
  static __device__ __forceinline__ void run(const void* w, const uint8_t*, int64_t ld, int col,
                                             int ncol, int K, int s0, int s1, int kg,
                                             const Row<X8>* rows, int nrows, float* red) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const bool col_ok = 4 * g < ncol;
    float acc[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[n][c] = 0.f;
    const float* base = static_cast<const float*>(w) + col + 4 * g;
    for (int s = s0; s < s1; ++s) {
      const int k = (s * KG + kg) * STEP + 4 * t;
      const bool ok = k < K;
      float v[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint4 q = ok && col_ok ? ldg_stream(base + (k + r) * ld) : make_uint4(0, 0, 0, 0);
        v[r][0] = __uint_as_float(q.x), v[r][1] = __uint_as_float(q.y);
        v[r][2] = __uint_as_float(q.z), v[r][3] = __uint_as_float(q.w);
      }
#pragma unroll
      for (int n = 0; n < 8; ++n)
        if (n < nrows && ok) {
          const float4 x = rows[n].f32x4(k);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            acc[n][c] = fmaf(x.w, v[3][c], fmaf(x.z, v[2][c], fmaf(x.y, v[1][c], fmaf(x.x, v[0][c], acc[n][c]))));
        }
    }
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[n][c] += __shfl_xor_sync(0xffffffffu, acc[n][c], 1);
        acc[n][c] += __shfl_xor_sync(0xffffffffu, acc[n][c], 2);
        if ((n >> 1) == t) red[n * PITCH + 4 * g + c] = acc[n][c];
      }
  }
};

// Microscaled e2m1 weights: codes [N, K/2] and scale bytes [N, K/32], the
// contraction innermost.  A lane loads whole blocks of 32 (16 bytes) of columns
// g, g + 8, g + 16 and g + 24, so each load has one scale.  Two codes four apart
// in a word lie 16 bits apart: their sign and magnitude bits are moved to bit 15
// and bits 8..6 of both halves at once, which reads as the value times 2^-126 in
// bf16 (0.5 is a subnormal there), and one exact bf16 product by 2^(126 + q)
// gives the weight.  Scales above 2 would need a larger factor than bf16 has
// and take a second product.
struct Mx {
  using Store = __nv_bfloat16;
  static constexpr int WF = 32, FG = 4, KG = 2, STEP = 128;
  static constexpr int PITCH = FG * WF + 1;   // of the results [row][column] in shared memory
  static constexpr bool kRowPerLane = true;
  static __device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  // Codes j and j + 4 of a word as bf16 values times 2^-126.
  template <int J>
  static __device__ __forceinline__ uint32_t spread(uint32_t w) {
    const uint32_t sign = J == 3 ? w : w << (12 - 4 * J);
    const uint32_t mag = J < 2 ? w << (6 - 4 * J) : w >> (4 * J - 6);
    return (sign & 0x80008000u) | (mag & 0x01c001c0u);
  }
  template <int NT, bool X8>
  static __device__ __forceinline__ void run(const void* w, const uint8_t* scales, int64_t, int col,
                                             int ncol, int K, int s0, int s1, int kg,
                                             const Row<X8>* rows, int, float* red) {
    // the token rows' loads go ahead with the weights' where registers allow (16
    // for a step's weights, 16 for a row tile's tokens, twice); two buffers take
    // turns
    constexpr bool EARLY = NT == 1;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int nb = K >> 5;
    const int64_t cld = K >> 1;
    float acc[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[m][n][q] = 0.f;
    const uint8_t* cp = static_cast<const uint8_t*>(w) + (static_cast<int64_t>(col) + g) * cld;
    const uint8_t* sp = scales + (static_cast<int64_t>(col) + g) * nb;
    uint4 v[2][4];
    uint32_t f[2][4];
    RawBlock<X8> x[2][EARLY ? NT : 1];
    auto load = [&](int buf, int s) {
      const int b = (s * KG + kg) * 4 + t;
      const bool ok = s < s1 && b < nb;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool in = ok && 8 * r < ncol;
        v[buf][r] = in ? ldg_stream(cp + 8 * r * cld + 16 * b) : make_uint4(0, 0, 0, 0);
        f[buf][r] = in ? __ldg(sp + static_cast<int64_t>(8 * r) * nb + b) : 0u;
      }
      if (EARLY)
#pragma unroll
        for (int n = 0; n < NT; ++n) x[buf][n].load(rows[n], b, ok);
    };
    auto multiply = [&](int buf, int s) {
      const int b = (s * KG + kg) * 4 + t;
      const bool ok = s < s1 && b < nb;
      bool large = false;
#pragma unroll
      for (int r = 0; r < 4; ++r) large = large || f[buf][r] > 128u;
      if (__any_sync(0xffffffffu, large))
        step<NT, X8, EARLY, true>(v[buf], f[buf], x[buf], b, ok, rows, acc);
      else
        step<NT, X8, EARLY, false>(v[buf], f[buf], x[buf], b, ok, rows, acc);
    };
    load(0, s0);
    for (int s = s0; s < s1; s += 2) {
      load(1, s + 1);
      multiply(0, s);
      if (s + 1 >= s1) break;
      load(0, s + 2);
      multiply(1, s + 1);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float* d = red + (8 * n + 2 * t) * PITCH + 16 * m + g;
        d[0] = acc[m][n][0], d[PITCH] = acc[m][n][1];
        d[8] = acc[m][n][2], d[PITCH + 8] = acc[m][n][3];
      }
  }
  template <int NT, bool X8, bool EARLY, bool LARGE>
  static __device__ __forceinline__ void step(const uint4 (&v)[4], const uint32_t (&f)[4],
                                              const RawBlock<X8>* x, int b, bool ok,
                                              const Row<X8>* rows, float (&acc)[2][NT][4]) {
    uint32_t f1[4], f2[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      f1[r] = ((LARGE ? min(f[r], 128u) : f[r]) + 126u) * 0x00800080u;
      if (LARGE)
        f2[r] = f[r] == 255u ? 0x7fc07fc0u : (f[r] > 128u ? (f[r] - 1u) * 0x00800080u : 0x3f803f80u);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t xb[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 xv = EARLY ? x[n].bf16x8(q) : (ok ? rows[n].bf16x8(32 * b + 8 * q) : make_uint4(0, 0, 0, 0));
        xb[n][0] = __byte_perm(xv.x, xv.z, 0x5410);   // values 0 and 4
        xb[n][1] = __byte_perm(xv.x, xv.z, 0x7632);   // 1 and 5
        xb[n][2] = __byte_perm(xv.y, xv.w, 0x5410);   // 2 and 6
        xb[n][3] = __byte_perm(xv.y, xv.w, 0x7632);   // 3 and 7
      }
      uint32_t a[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t wd = q == 0 ? v[r].x : (q == 1 ? v[r].y : (q == 2 ? v[r].z : v[r].w));
        a[r][0] = mul2(spread<0>(wd), f1[r]);
        a[r][1] = mul2(spread<1>(wd), f1[r]);
        a[r][2] = mul2(spread<2>(wd), f1[r]);
        a[r][3] = mul2(spread<3>(wd), f1[r]);
        if (LARGE) {
#pragma unroll
          for (int j = 0; j < 4; ++j) a[r][j] = mul2(a[r][j], f2[r]);
        }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma16816(acc[m][n], a[2 * m][0], a[2 * m + 1][0], a[2 * m][1], a[2 * m + 1][1], xb[n][0], xb[n][1]);
          mma16816(acc[m][n], a[2 * m][2], a[2 * m + 1][2], a[2 * m][3], a[2 * m + 1][3], xb[n][2], xb[n][3]);
        }
    }
  }
};

// ------------------------------------------------------------------ kernels
__device__ __forceinline__ float load_elem(const __nv_bfloat16* p, int64_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ float load_elem(const float* p, int64_t i) { return p[i]; }

__device__ __forceinline__ float sigmoid_exact(float v) { return 1.f / (1.f + expf(-v)); }

// A NaN stays a NaN through the clamps.
__device__ __forceinline__ float activate(const FewArgs& a, float gate, float up) {
  if (a.act_kind == MOE_ACT_SWIGLU) return gate * sigmoid_exact(gate) * up;
  const float gc = gate > a.limit ? a.limit : gate;
  const float uc = up > a.limit ? a.limit : (up < -a.limit ? -a.limit : up);
  return (uc + 1.f) * gc * sigmoid_exact(a.alpha * gc);
}

// All units' steps cut into `grid` runs, the first `more` of them one step longer.
struct Runs {
  int grid, len, more;
  __device__ __forceinline__ Runs(int steps, int blocks) {
    // no more runs than steps: a unit's blocks are consecutive and each has a share
    grid = min(blocks, steps);
    len = grid ? steps / grid : 0;
    more = steps - len * grid;
  }
  __device__ __forceinline__ int begin(int c) const { return c * len + min(c, more); }
  __device__ __forceinline__ int block_of(int s) const {
    const int head = more * (len + 1);
    return s < head ? s / (len + 1) : more + (s - head) / len;
  }
};

// The products of one unit's share for `tiles` row tiles, in the smallest
// instance that holds them.
template <class W, int NT, bool X8>
__device__ __forceinline__ void run_tiles(int tiles, const void* w, const uint8_t* scales, int64_t ld,
                                          int col, int ncol, int K, int s0, int s1, int kg,
                                          const Row<X8>* rows, int nrows, float* red) {
  if constexpr (NT >= 4) {
    if (tiles > 2) {
      W::template run<4, X8>(w, scales, ld, col, ncol, K, s0, s1, kg, rows, nrows, red);
      return;
    }
  }
  if constexpr (NT >= 2) {
    if (tiles > 1) {
      W::template run<2, X8>(w, scales, ld, col, ncol, K, s0, s1, kg, rows, nrows, red);
      return;
    }
  }
  W::template run<1, X8>(w, scales, ld, col, ncol, K, s0, s1, kg, rows, nrows, red);
}

// Floats of `red`: the shares' results, or the 256 threads' sums of the combine.
template <class W>
__host__ __device__ __forceinline__ int red_floats(int rows) {
  const int n = (W::KG * W::PITCH * rows + 3) & ~3;
  return n > 4 * kThreads ? n : 4 * kThreads;
}

// The activation of a unit's results, red[row][column], into its rows of a.act.
template <class W>
__device__ __forceinline__ void finish_gate_up(const FewArgs& a, const Plan& p, const float* red,
                                               int chunk, int tile) {
  using S = typename W::Store;
  constexpr int OUT = W::FG * W::WF / 2;
  const int first = p.chunk_first[chunk], nrows = p.chunk_rows[chunk];
  const S* b = a.bias ? static_cast<const S*>(a.bias) + static_cast<int64_t>(p.chunk_e[chunk]) * 2 * a.I : nullptr;
  for (int i = threadIdx.x; i < OUT * nrows; i += kThreads) {
    const int f = i % OUT, r = i / OUT;
    const int feature = tile * OUT + f;
    if (feature >= a.I) continue;
    const float* q = red + r * W::PITCH;
    float gate = q[a.interleaved ? 2 * f : f];
    float up = q[a.interleaved ? 2 * f + 1 : f + OUT];
    if (b) {
      gate += load_elem(b, a.interleaved ? 2 * feature : feature);
      up += load_elem(b, a.interleaved ? 2 * feature + 1 : a.I + feature);
    }
    static_cast<S*>(a.act)[static_cast<int64_t>(p.slot[first + r]) * a.I + feature] =
        static_cast<S>(activate(a, gate, up));
  }
}

__device__ __forceinline__ void add4(float4& v, const float4& o) {
  v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
}
__device__ __forceinline__ float4 ldcg4(const float* p) { return __ldcg(reinterpret_cast<const float4*>(p)); }

template <class S>
__device__ __forceinline__ void store_y(const FewArgs& a, int tok, int c, const float4& y) {
  if (c >= a.H) return;
  const int64_t at = static_cast<int64_t>(tok) * a.H + c;
  if (a.out_fp32 || sizeof(S) == 4)
    *reinterpret_cast<float4*>(static_cast<float*>(a.y) + at) = y;
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.y) + at) =
        make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
}

// y of one column tile from every chunk's products: whole units' in a.o, cut
// ones' in their blocks' parts.
template <class W>
__device__ __forceinline__ void combine_tile(const FewArgs& a, const Plan& p, const Runs& runs, int KS,
                                             int tile, float* red) {
  using S = typename W::Store;
  constexpr int CW = W::FG * W::WF, V = CW / 4;
  const int UNIT = a.rows * CW;
  // the blocks of each chunk's unit: first | last << 15 | whether the first one's
  // part is its second
  for (int c = threadIdx.x; c < p.chunks; c += kThreads) {
    const int b0 = (tile * p.chunks + c) * KS;
    const int f0 = runs.block_of(b0), f1 = runs.block_of(b0 + KS - 1);
    p.span[c] = f0 | (f1 << 15) | (runs.begin(f0) < b0 ? 1u << 30 : 0u);
  }
  __syncthreads();
  // With few tokens a token's choices are shared out over `groups` threads (every
  // groups-th choice each) whose sums are added in order.
  const int items = a.T * V;
  const int groups = max(1, min(a.k, kThreads / items));
  float4* sums = reinterpret_cast<float4*>(red);
  for (int i = threadIdx.x; i < items * groups; i += kThreads) {
    const int f = i % V * 4, tok = i / V % a.T, group = i / items;
    const int c = tile * CW + f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < a.H) {
#pragma unroll 4
      for (int j = group; j < a.k; j += groups) {
        const int slot = tok * a.k + j;
        const int at = p.where[slot];
        if (at == kNowhere) continue;
        const float w = __ldg(a.topk_w + slot);
        const uint32_t sp = p.span[at >> 5];
        const int f0 = sp & 0x7fff, n = static_cast<int>((sp >> 15) & 0x7fff) - f0;
        const int q = (at & 31) * CW + f;
        const float* head = n ? a.part + (2 * static_cast<int64_t>(f0) + (sp >> 30)) * UNIT + q
                              : a.o + static_cast<int64_t>(slot) * a.H + c;
        const float* next = a.part + 2 * static_cast<int64_t>(f0 + 1) * UNIT + q;
        float4 v = ldcg4(head), o[3], bias = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int b = 0; b < 3; ++b)
          o[b] = b < n ? ldcg4(next + 2 * static_cast<int64_t>(b) * UNIT) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.bias) {
          const S* b = static_cast<const S*>(a.bias) + static_cast<int64_t>(p.chunk_e[at >> 5]) * a.H + c;
          bias = make_float4(load_elem(b, 0), load_elem(b, 1), load_elem(b, 2), load_elem(b, 3));
        }
#pragma unroll
        for (int b = 0; b < 3; ++b) add4(v, o[b]);
        for (int b = 3; b < n; ++b) add4(v, ldcg4(next + 2 * static_cast<int64_t>(b) * UNIT));
        add4(v, bias);
        y.x = fmaf(w, v.x, y.x), y.y = fmaf(w, v.y, y.y);
        y.z = fmaf(w, v.z, y.z), y.w = fmaf(w, v.w, y.w);
      }
    }
    if (groups == 1)
      store_y<S>(a, tok, c, y);
    else
      sums[i] = y;
  }
  if (groups > 1) {
    __syncthreads();
    for (int i = threadIdx.x; i < items; i += kThreads) {
      float4 y = sums[i];
      for (int g = 1; g < groups; ++g) add4(y, sums[g * items + i]);
      store_y<S>(a, i / V, tile * CW + i % V * 4, y);
    }
  }
  __syncthreads();   // p.span and red are free again
}

// PHASE 0: gate_up and activation; a cut unit is finished by the last of its
// blocks.  PHASE 1: down and combine; a column tile is finished by the last of
// its blocks.  Units are ordered by tile, then chunk: a run covers few tiles, and
// experts with many rows and with few mix in every run.  A block counts itself in
// at the end of its run, once, for the pieces at its two ends; the pieces between
// are its own alone.
template <class W, int PHASE, int NT, bool X8>
__global__ void __launch_bounds__(kThreads, 2) few_kernel(const __grid_constant__ FewArgs a) {
  using S = typename W::Store;
  constexpr int CW = W::FG * W::WF;            // weight columns of a unit
  const int UNIT = a.rows * CW;                // results of a unit, [row][column]
  const int SHARE = a.rows * W::PITCH;         // one share's results in shared memory
  constexpr int OUT = PHASE == 0 ? CW / 2 : CW;
  extern __shared__ float4 red4[];
  float* red = reinterpret_cast<float*>(red4);
  __shared__ PlanSmall ps;
  Plan p = plan_at(red + red_floats<W>(a.rows), a.T * a.k, a.E, a.rows);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int fg = warp % W::FG, kg = warp / W::FG;
  const int me = blockIdx.x;
  if (PHASE == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  build_plan(p, ps, a.idx, a.T * a.k, a.E, a.rows, PHASE == 0 ? a.err : nullptr);

  const int K = PHASE == 0 ? a.H : a.I;                // contraction
  const int N = PHASE == 0 ? 2 * a.I : a.H;            // weight columns
  const int tiles = ((PHASE == 0 ? a.I : a.H) + OUT - 1) / OUT;
  const int KS = (K + W::KG * W::STEP - 1) / (W::KG * W::STEP);
  const int chunks = p.chunks;
  const Runs runs(chunks * tiles * KS, gridDim.x);
  if (PHASE == 1) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (me >= runs.grid) {
    // no row at all (every id out of range): y is still written
    if (PHASE == 1 && runs.grid == 0) {
      for (int64_t i = me * static_cast<int64_t>(kThreads) + tid; i < static_cast<int64_t>(a.T) * a.H;
           i += static_cast<int64_t>(gridDim.x) * kThreads) {
        if (a.out_fp32)
          static_cast<float*>(a.y)[i] = 0.f;
        else
          static_cast<S*>(a.y)[i] = static_cast<S>(0.f);
      }
    }
    return;
  }
  const int begin = runs.begin(me), end = runs.begin(me + 1);

  for (int s = begin; s < end;) {
    const int unit = s / KS;
    const int u0 = unit * KS;
    const int ks0 = s - u0;
    const int ks1 = min(KS, end - u0);
    const int chunk = unit % chunks, tile = unit / chunks;
    const int e = p.chunk_e[chunk], first = p.chunk_first[chunk], nrows = p.chunk_rows[chunk];

    // this warp's columns
    int col, ncol;
    if (PHASE == 0 && !a.interleaved) {
      constexpr int HALF = W::FG / 2;
      const int o = tile * OUT + (fg % HALF) * W::WF;
      col = (fg / HALF) * a.I + o;
      ncol = a.I - o;
    } else {
      col = tile * CW + fg * W::WF;
      ncol = N - col;
    }
    // the biases that the finishing block will want (128-byte lines)
    if (a.bias && lane == 0 && kg == 0 && ncol > 0)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const S*>(a.bias) + static_cast<int64_t>(e) * N + col));
    Row<X8> rows[W::kRowPerLane ? NT : 8];
#pragma unroll
    for (int i = 0; i < (W::kRowPerLane ? NT : 8); ++i) {
      const int r = W::kRowPerLane ? 8 * i + (lane >> 2) : i;
      if (r < nrows) {
        const int slot = p.slot[first + r];
        const int64_t row = PHASE == 0 ? slot / a.k : slot;
        if (X8) {
          rows[i].p = static_cast<const uint8_t*>(a.x) + row * K;
          rows[i].scale = a.x_scale + row * (K >> 5);
        } else {
          rows[i].p = static_cast<const S*>(a.x) + row * K;
        }
      }
    }
    if (ncol > 0) {
      const int64_t we = static_cast<int64_t>(e) * K * N;   // weights of the experts before
      const void* w = sizeof(S) == 4 ? static_cast<const void*>(static_cast<const float*>(a.w) + we)
                      : W::STEP == 128
                          ? static_cast<const void*>(static_cast<const uint8_t*>(a.w) + we / 2)
                          : static_cast<const void*>(static_cast<const __nv_bfloat16*>(a.w) + we);
      run_tiles<W, NT, X8>((nrows + 7) >> 3, w, W::STEP == 128 ? a.scales + we / 32 : nullptr, N, col,
                           ncol, K, ks0, ks1, kg, rows, nrows, red + kg * SHARE + fg * W::WF);
    }
    __syncthreads();

    // add the shares of the contraction; a cut unit's sum goes to its part, a
    // whole one stays (gate_up) or goes to its rows (down)
    const bool whole = ks1 - ks0 == KS;
    float* part = a.part + (2 * static_cast<int64_t>(me) + (begin >= u0 ? 0 : 1)) * UNIT;
    for (int i = tid; i < nrows * CW; i += kThreads) {
      const int f = i % CW, r = i / CW, q = r * W::PITCH + f;
      float v = red[q];
#pragma unroll
      for (int j = 1; j < W::KG; ++j) v += red[j * SHARE + q];
      if (!whole)
        part[i] = v;
      else if (PHASE == 0)
        red[q] = v;
      else if (tile * OUT + f < a.H)
        a.o[static_cast<int64_t>(p.slot[first + r]) * a.H + tile * OUT + f] = v;
    }
    __syncthreads();
    if (PHASE == 0 && whole) {
      finish_gate_up<W>(a, p, red, chunk, tile);
      __syncthreads();
    }
    // a tile that lies in this run alone
    if (PHASE == 1 && chunk == chunks - 1 && ks1 == KS && begin <= tile * chunks * KS)
      combine_tile<W>(a, p, runs, KS, tile, red);
    s = u0 + ks1;
  }

  // the pieces at the run's ends: piece 0 its first unit (tile), 1 its last
  const int per = PHASE == 0 ? KS : chunks * KS;       // steps of a unit (tile)
  const int p0 = begin / per, p1 = (end - 1) / per;
  if (tid < 2) {
    const int piece = tid ? p1 : p0;
    const int lo = max(begin, piece * per), hi = min(end, (piece + 1) * per);
    int last = 0;
    if (hi - lo < per && (tid == 0 || p1 != p0)) {
      // a unit's counter is its first block's (a block is the first of at most one cut unit)
      unsigned* c = a.counters + (PHASE == 0 ? runs.block_of(piece * per) : piece);
      last = join_add(c, hi - lo) + (hi - lo) == static_cast<unsigned>(per);
      if (last) *c = 0;
    }
    ps.last[tid] = last;
  }
  __syncthreads();
  for (int i = 0; i < 2; ++i) {
    if (!ps.last[i]) continue;
    const int piece = i ? p1 : p0;
    if (PHASE == 1) {
      combine_tile<W>(a, p, runs, KS, piece, red);
      continue;
    }
    const int chunk = piece % chunks;
    const int nrows = p.chunk_rows[chunk];
    const int c0 = runs.block_of(piece * KS), c1 = runs.block_of(piece * KS + KS - 1);
    const float* head = a.part + (2 * static_cast<int64_t>(c0) + (runs.begin(c0) >= piece * KS ? 0 : 1)) * UNIT;
    for (int j = tid; j < nrows * CW; j += kThreads) {
      float v = __ldcg(head + j);
#pragma unroll 4
      for (int c = c0 + 1; c <= c1; ++c) v += __ldcg(a.part + 2 * static_cast<int64_t>(c) * UNIT + j);
      red[j / CW * W::PITCH + j % CW] = v;
    }
    __syncthreads();
    finish_gate_up<W>(a, p, red, chunk, piece / chunks);
    __syncthreads();
  }
}

template <class W, int PHASE, int NT, bool X8>
cudaError_t launch(const FewArgs& a, int grid, cudaStream_t st) {
  const int smem = red_floats<W>(a.rows) * 4 + plan_bytes(a.T * a.k, a.E, a.rows);
  const int most = red_floats<W>(8 * NT) * 4 + kMostPlanBytes;
  static std::atomic<uint64_t> ready{0};   // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(few_kernel<W, PHASE, NT, X8>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = PHASE == 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, few_kernel<W, PHASE, NT, X8>, a);
}

template <class W, int PHASE, bool X8>
cudaError_t launch_nt(const FewArgs& a, int nt, int grid, cudaStream_t st) {
  if constexpr (W::kRowPerLane) {
    if (nt > 1) return launch<W, PHASE, 4, X8>(a, grid, st);
  }
  return launch<W, PHASE, 1, X8>(a, grid, st);
}

// Row tiles of 8 tokens per unit, at most four (registers): as many as hold an
// expert's rows when every token names it once, so its weights are read once.  A
// unit runs only the tiles that its rows fill.
int row_tiles(const moe_shape* s) {
  return s->dtype == MOE_FP32 ? 1 : static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(4, (s->T + 7) / 8)));
}

struct FewLayout {
  size_t counters0, counters1, act, part, o, total;
};
FewLayout few_layout(const moe_shape* s) {
  FewLayout L;
  size_t off = 256;   // the error word
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = abi_align256(off + bytes);
    return at;
  };
  const size_t Tk = static_cast<size_t>(s->T) * s->k;
  L.counters0 = take(sizeof(unsigned) * kMaxGrid);
  L.counters1 = take(sizeof(unsigned) * ((s->H + 63) / 64));
  L.act = take((s->dtype == MOE_FP32 ? 4 : 2) * Tk * s->I);
  L.part = take(sizeof(float) * 2 * kMaxGrid * 128 * 8 * row_tiles(s));
  L.o = take(sizeof(float) * Tk * s->H);
  L.total = off;
  return L;
}

// Few tokens, and steps that 32 bits count: the smallest units are 32 outputs by
// 64 values of the contraction.
bool few_size_ok(const moe_shape* s) {
  const int64_t wide = std::max(s->H, s->I) / 32 + 1, deep = std::max(s->H, s->I) / 64 + 1;
  return s->T <= kMaxTokens &&
         std::min<int64_t>(s->T * s->k, s->E + s->T * s->k / 8) * wide * deep < (1ll << 31);
}
bool few_shape_ok(const moe_shape* s) { return abi_shape_ok(s) && few_size_ok(s); }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_few_workspace_size(const moe_shape* shape) {
  return few_shape_ok(shape) ? few_layout(shape).total : 0;
}

moe_status moe_ffn_few(const moe_shape* s, const void* x, const uint8_t* x_scale,
                       const int32_t* topk_idx, const float* topk_w, const void* w_gate_up,
                       const void* w_down, const moe_mx_weights_t* mx, const moe_bias_t* bias,
                       void* y, void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!abi_shape_ok(s) || !ws || (reinterpret_cast<uintptr_t>(ws) & 255)) return MOE_ERR_INVALID_ARG;
  if (mx ? (w_gate_up || w_down) : (!w_gate_up || !w_down)) return MOE_ERR_INVALID_ARG;
  if (mx) {
    if (!mx->codes_gate_up || !mx->scales_gate_up || !mx->codes_down || !mx->scales_down ||
        !abi_aligned16(mx->codes_gate_up) || !abi_aligned16(mx->codes_down) || s->H % 32 || s->I % 32)
      return MOE_ERR_INVALID_ARG;
    if (s->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  }
  if (x_scale && s->H % 32) return MOE_ERR_INVALID_ARG;
  if (s->T == 0) return MOE_OK;
  if (!x || !topk_idx || !topk_w || !y) return MOE_ERR_INVALID_ARG;
  for (const void* q : {x, w_gate_up, w_down, static_cast<const void*>(y)})
    if (!abi_aligned16(q)) return MOE_ERR_INVALID_ARG;
  if (bias && (!abi_aligned16(bias->b_gate_up) || !abi_aligned16(bias->b_down)))
    return MOE_ERR_INVALID_ARG;
  if (!few_size_ok(s)) return MOE_ERR_UNSUPPORTED;
  const FewLayout L = few_layout(s);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  int sms = 0;
  const moe_status ds = abi_device_sms(&sms);
  if (ds != MOE_OK) return ds;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int grid = std::min(kMaxGrid, 2 * sms);
  char* base = static_cast<char*>(ws);

  FewArgs a = {};
  a.x = x;
  a.x_scale = x_scale;
  a.idx = topk_idx;
  a.topk_w = topk_w;
  a.w = mx ? mx->codes_gate_up : w_gate_up;
  a.scales = mx ? mx->scales_gate_up : nullptr;
  a.bias = bias ? bias->b_gate_up : nullptr;
  a.act = base + L.act;
  a.part = reinterpret_cast<float*>(base + L.part);
  a.o = reinterpret_cast<float*>(base + L.o);
  a.y = y;
  a.counters = reinterpret_cast<unsigned*>(base + L.counters0);
  a.err = reinterpret_cast<int*>(base);
  a.T = static_cast<int>(s->T);
  a.H = s->H, a.I = s->I, a.E = s->E, a.k = s->k;
  a.act_kind = s->act;
  a.interleaved = s->gate_up_layout == MOE_GATE_UP_INTERLEAVED;
  a.out_fp32 = s->out_fp32;
  a.limit = s->clamp_limit;
  a.alpha = s->alpha;
  const int nt = row_tiles(s);
  a.rows = 8 * nt;

  cudaError_t e = abi_tracked(kAbiFewGateUp, 1, st, [&] {
    if (s->dtype == MOE_FP32)
      return x_scale ? launch_nt<F32, 0, true>(a, nt, grid, st) : launch_nt<F32, 0, false>(a, nt, grid, st);
    if (mx)
      return x_scale ? launch_nt<Mx, 0, true>(a, nt, grid, st) : launch_nt<Mx, 0, false>(a, nt, grid, st);
    return x_scale ? launch_nt<Bf16, 0, true>(a, nt, grid, st) : launch_nt<Bf16, 0, false>(a, nt, grid, st);
  });
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  a.x = a.act;
  a.x_scale = nullptr;
  a.w = mx ? mx->codes_down : w_down;
  a.scales = mx ? mx->scales_down : nullptr;
  a.bias = bias ? bias->b_down : nullptr;
  a.counters = reinterpret_cast<unsigned*>(base + L.counters1);
  e = abi_tracked(kAbiFewDown, 1, st, [&] {
    if (s->dtype == MOE_FP32) return launch_nt<F32, 1, false>(a, nt, grid, st);
    if (mx) return launch_nt<Mx, 1, false>(a, nt, grid, st);
    return launch_nt<Bf16, 1, false>(a, nt, grid, st);
  });
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
