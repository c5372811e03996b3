// The whole expert layer for a few tokens, in two kernels:
//
//   gate_up:  a[s]  = act(x[s / k] Wgu[e_s] (+ b_gate_up))      for every slot s
//   down:     y[t]  = sum_j w[t,j] (a[t k + j] Wd[e] (+ b_down))
//
// (A small one before them clears the joins' counters and rewrites e4m3 tokens, or any
// tokens for 4-bit weights.)
// With a few rows per expert the layer reads each touched expert's weights once
// and does next to nothing with them: it is bound by HBM, not by the tensor
// cores.  So the weights are operands of warp-level matrix instructions (weights on
// the 16-row side, up to 8 tokens per instruction on the other): bf16 and fp32 ones
// go from global memory straight into registers, 4-bit ones through a ring of TMA
// copies per warp, and everything else is arranged to keep loads in flight and every
// SM busy to the end:
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
// Precision.  Products accumulate in fp32.  a is rounded between the kernels, being
// an operand of the next product: to bf16 with bf16 weights, as the layer for many
// tokens does; to fp16 with a power of two per 32 values (11 bits, see kTokenTop) with
// 4-bit weights.  fp32 weights keep it in fp32 and multiply on the CUDA cores in fp32.
//
// Measured, of the bytes of the touched experts' weights (a copy reaches 6.76 TB/s):
// 16 tokens on 256 bf16 experts of 4096 x 2048 (5.1 GB) 745 to 847 us by machine and
// pass, 6.1 to 6.9 TB/s; one token on four of 2880 x 2880 (199 MB) 47 us, of which 36 us
// stream at 5.5 TB/s and the rest is start, joins and the step between the kernels; 32
// tokens on 64 4-bit experts of 8192 x 2048 (1.7 GB) 366 to 380 us, 4.5 TB/s, bound by
// instructions.
#include <cuda.h>

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
constexpr int kPrefetchSteps = 6;
constexpr int kMaxCW = 256;       // weight columns of a unit, at most
constexpr int kNowhere = 0xffff;
constexpr uint64_t kDrainNs = 200000000ull;   // for copies in flight after a wait ran out
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
  const void* w_next;      // gate_up: the down kernel's weights and bias
  const uint8_t* scales_next;
  const void* bias_next;
  void* act;               // [Tk, I]: storage type; fp16 with 4-bit weights, and
  uint8_t* act_scale;      // [Tk, I/32] its blocks' scale bytes, and
  int* act_top;            // [Tk] the largest of each row's
  const int* top;          // of the fp16 rows in x
  float* part;             // parts of cut units: 2 per block
  float* o;                // [Tk, H] products of whole units
  void* y;
  unsigned* counters;      // this kernel's, cleared by the kernel before both
  int* err;
  int T, H, I, E, k, rows, act_kind, interleaved, out_fp32;   // rows: of a chunk
  float limit, alpha;
  uint64_t timeout_ns;
  CUtensorMap codes;       // 4-bit weights: this kernel's [E, N, K/2]
};

// ------------------------------------------------------------------ plan
// A chunk is up to `rows` (8 or 16) rows of one expert; chunks are ordered by
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

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Weights: read once, never written by the layer.
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Token rows and activations.  A kernel may start before the one that writes them
// has ended, so these are plain loads in program order, after its wait.
__device__ __forceinline__ uint32_t ld_u8(const void* p) {
  uint32_t v;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_u16(const void* p) {
  uint32_t v;
  asm volatile("ld.global.u16 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
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

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Waits for the kernel before (returns at once when it has ended).
__device__ __forceinline__ void wait_for_rows() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A token row (or a slot's activations) as the product reads it.
struct Row {
  const void* p;
  int row;    // of fp16 rows: which, and
  int top;    // its byte, the largest of its blocks'
};

// bf16 weights [K, ld], columns innermost.  A lane loads 16 bytes (8 columns) of
// four rows of the contraction; pairs along the contraction, as the instruction
// wants them, come from two rows by byte permutes.  Columns 2 i and 2 i + 1 of
// the lane are rows g and g + 8 of instruction i.  Past the contraction's end both
// are zero; columns past the end and rows that a unit does not have are computed
// from others' and never read.
//
// Four groups of columns side by side make a block's rows 512 bytes (gate_up: two
// times 256): with two, 16 tokens on 256 experts take 4% longer in gate_up.
struct Bf16 {
  using Store = __nv_bfloat16;
  static constexpr int WF = 64, FG = 4, KG = 2, STEP = 16;
  static constexpr int PITCH = FG * WF + 1;   // of the results [row][column] in shared memory
  static constexpr bool kHalfRows = false;
  static constexpr int kRing = 0;
  static constexpr bool kRowPerLane = true;   // lane (g, t) reads rows g, g + 8, ...
  static constexpr int kMaxTiles = 2;
  // The weights of step s of a unit, all columns: 32 rows of four 128-byte lines.
  static __device__ __forceinline__ void prefetch(const void* w, const uint8_t*, int64_t first, int64_t ld,
                                                  int col, int K, int s) {
    const int k = s * KG * STEP + (threadIdx.x / FG), c = col + (threadIdx.x % FG) * 64;
    if (threadIdx.x < FG * KG * STEP && k < K && c < ld)
      prefetch_l2(static_cast<const __nv_bfloat16*>(w) + first + k * ld + c);
  }
  template <int NT>
  static __device__ __forceinline__ void run(const void* w, int64_t ld, int col, int ncol, int K, int s0, int s1, int kg,
                                             const Row* rows, int nrows, float* red) {
    constexpr int U = NT == 1 ? 2 : 1;   // steps per buffer; two buffers take turns
    const bool both = NT > 1 && nrows > 8;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float acc[4][NT][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][n][q] = 0.f;
    const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(w) + col + (8 * g < ncol ? 8 * g : 0);
    uint4 v[2][U][4];
    uint2 xb[2][U][NT];
    auto load_w = [&](int buf, int s) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = ((s + u) * KG + kg) * STEP + 4 * t;
        const bool ok = s + u < s1 && k < K;
        const __nv_bfloat16* p = base + k * ld;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[buf][u][r] = ok ? ldg_stream(p + r * ld) : make_uint4(0, 0, 0, 0);
      }
    };
    auto load_x = [&](int buf, int s) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = ((s + u) * KG + kg) * STEP + 4 * t;
        const bool ok = s + u < s1 && k < K;
#pragma unroll
        for (int n = 0; n < NT; ++n)
          if (n == 0 || both)
            xb[buf][u][n] = ok ? ld_u64(static_cast<const __nv_bfloat16*>(rows[n].p) + k) : make_uint2(0, 0);
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
          for (int n = 0; n < NT; ++n)
            if (n == 0 || both) mma16816(acc[i][n], a0, a1, a2, a3, xb[buf][u][n].x, xb[buf][u][n].y);
        }
      }
    };
    load_w(0, s0);
    wait_for_rows();
    load_x(0, s0);
    for (int s = s0; s < s1; s += 2 * U) {
      load_w(1, s + U);
      load_x(1, s + U);
      multiply(0);
      load_w(0, s + 2 * U);
      load_x(0, s + 2 * U);
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
// Bound by HBM up to a row or two per expert (one token on 4 experts of 2880 x 2880:
// 88 us, 4.5 TB/s), by instructions beyond (16 tokens on 16: 381 us, 4.2 TB/s).
struct F32 {
  using Store = float;
  static constexpr int WF = 32, FG = 2, KG = 4, STEP = 16;
  static constexpr int PITCH = FG * WF + 1;   // of the results [row][column] in shared memory
  static constexpr bool kHalfRows = false;
  static constexpr int kRing = 0;
  static constexpr bool kRowPerLane = false;   // every lane reads all rows
  static constexpr int kMaxTiles = 1;
  static __device__ __forceinline__ void prefetch(const void* w, const uint8_t*, int64_t first, int64_t ld,
                                                  int col, int K, int s) {
    const int k = s * KG * STEP + (threadIdx.x >> 1), c = col + (threadIdx.x & 1) * 32;
    if (threadIdx.x < 2 * KG * STEP && k < K && c < ld)
      prefetch_l2(static_cast<const float*>(w) + first + k * ld + c);
  }
  template <int NT>
  static __device__ __forceinline__ void run(const void* w, int64_t ld, int col, int ncol, int K, int s0, int s1, int kg,
                                             const Row* rows, int nrows, float* red) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const bool col_ok = 4 * g < ncol;
    float acc[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[n][c] = 0.f;
    const float* base = static_cast<const float*>(w) + col + 4 * g;
    uint4 v[2][4];   // two buffers take turns
    auto load = [&](int buf, int s) {
      const int k = (s * KG + kg) * STEP + 4 * t;
      const bool ok = s < s1 && k < K && col_ok;
      const float* p = base + k * ld;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[buf][r] = ok ? ldg_stream(p + r * ld) : make_uint4(0, 0, 0, 0);
    };
    auto multiply = [&](int buf, int s) {
      const int k = (s * KG + kg) * STEP + 4 * t;
      if (s >= s1 || k >= K) return;
      // four rows' loads at a time (rows that are not there repeat the first)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (4 * half >= nrows) break;
        uint4 x[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) x[n] = ld_u128(static_cast<const float*>(rows[4 * half + n].p) + k);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          float* s4 = acc[4 * half + n];
          const uint32_t* q = &x[n].x;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float xr = __uint_as_float(q[r]);
            const uint4& wr = v[buf][r];
            const float2 lo = fma2(make_float2(xr, xr), make_float2(__uint_as_float(wr.x), __uint_as_float(wr.y)),
                                   make_float2(s4[0], s4[1]));
            const float2 hi = fma2(make_float2(xr, xr), make_float2(__uint_as_float(wr.z), __uint_as_float(wr.w)),
                                   make_float2(s4[2], s4[3]));
            s4[0] = lo.x, s4[1] = lo.y, s4[2] = hi.x, s4[3] = hi.y;
          }
        }
      }
    };
    load(0, s0);
    wait_for_rows();
    for (int s = s0; s < s1; s += 2) {
      load(1, s + 1);
      multiply(0, s);
      load(0, s + 2);
      multiply(1, s + 1);
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

// Where fp16 holds the largest of a token row's values and of a block of 32
// activations, as a power of two.  A token row has one scale: its values down to 2^-29
// of the largest keep bf16's bits, and smaller ones are rounded at 2^-39 of it.  Blocks
// of activations are brought to their row's power of two by a factor in fp16, whose own
// range ends at 2^-24, so a block with its largest at 2^7 may lie 2^31 below the row's
// largest before it is lost, and its values are rounded at 2^-32 of the block's
// largest: an activation has fp16's 11 bits or an error of at most 2^-31 of its row's
// largest.  (With 2^14 for both, blocks more than 2^24 below were lost.)
constexpr int kTokenTop = 14, kActTop = 7;

// Microscaled e2m1 weights: codes [N, K/2] and scale bytes [N, K/32], the
// contraction innermost; token rows in fp16 with a power of two per row (and
// possibly per block of 32).
//
// At HBM's rate an SM gets some 44 weights a clock and issues 128 operations, half
// of them logic and conversions, so decoding must be cheap: a conversion e2m1 ->
// fp16 makes two weights, and one fp16 product scales them, two instructions per
// two weights (half of all that a step takes).  A lane takes whole blocks (16 bytes)
// of columns g, g + 8, g + 16 and g + 24, so each has one scale 2^q.  The codes come
// by TMA, two steps ahead and across the ends of units: with two steps in registers
// instead, 32 tokens on 64 experts took 465 us, not 365, and a ring of four smaller
// steps takes 427.  What is left to wait for are tokens and scale bytes at a unit's
// start.  fp16 holds 2^q times a code exactly only near 1, so a column's weights are
// scaled by 2^(q - ref), ref being the scale of the first block that the warp sees of
// that column (or, where that holds zeros, of the first that does not: new_ref), and
// the sums by 2^ref at the end.  A step with a block outside 2^-14 .. 2^13 of its
// column's ref (or a NaN scale) takes a path that multiplies the blocks one by one and
// scales sums.
struct Mx {
  using Store = __nv_bfloat16;
  static constexpr int WF = 32, FG = 4, KG = 2, STEP = 256;
  static constexpr int PITCH = FG * WF + 1;   // of the results [row][column] in shared memory
  static constexpr int kMaxTiles = 2;
  static constexpr bool kRowPerLane = true, kHalfRows = true;
  // A warp's ring of steps in shared memory: 32 columns of 128 bytes each.
  static constexpr int kRing = 2, kSlotBytes = WF * STEP / 2;

  static __device__ __forceinline__ void mma(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
  // The eight codes of a word as fp16 pairs.
  static __device__ __forceinline__ void decode(uint32_t w, uint32_t (&v)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
        : "r"(w));
  }
  static __device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t word(const uint4& v, int q) {
    return q == 0 ? v.x : (q == 1 ? v.y : (q == 2 ? v.z : v.w));
  }
  // 2^d for d <= 15 in both halves of fp16, 0 below its range.
  static __device__ __forceinline__ uint32_t pow2_half(int d) {
    const uint32_t h = d >= -14 ? (d + 15) << 10 : (d >= -24 ? 1u << (d + 24) : 0u);
    return h * 0x00010001u;
  }

  // fp16 rows lie as the lanes read them: of each 256 values (a step of a warp) the
  // blocks 2 t of all lanes come before the blocks 2 t + 1, and the 16-byte chunks q
  // of a half's four blocks side by side.
  static __host__ __device__ __forceinline__ int pitch(int K) { return (K + STEP - 1) / STEP * STEP; }
  static __host__ __device__ __forceinline__ int scale_pitch(int K) { return (K / 32 + 1) & ~1; }
  // Where chunk i (values 8 i .. 8 i + 7) of a row is.
  static __device__ __forceinline__ int chunk_at(int i) {
    const int b = i >> 2;
    return (i & ~31) | (b & 1) << 4 | (i & 3) << 2 | ((b >> 1) & 3);
  }
  static __device__ __forceinline__ uint4 row_vec(const void* p, int q) {
    return ld_u128(static_cast<const char*>(p) + q * 64);
  }
  // What brings an activation block with this scale byte to the row's power of two,
  // which has the largest block where fp16's tokens are too.
  static constexpr int kActUp = kTokenTop - kActTop;
  static __device__ __forceinline__ uint32_t row_factor(uint32_t p, int top) {
    return p == 255u ? 0x7e007e00u : pow2_half(static_cast<int>(p) - top + kActUp);
  }

  // The codes of step s of a unit, KG lines of each column, and the lines of their
  // scales.
  static __device__ __forceinline__ void prefetch(const void* w, const uint8_t* scales, int64_t first,
                                                  int64_t ld, int col, int K, int s) {
    static_assert(FG * WF * KG == kThreads, "a line per thread");
    const int64_t c = col + threadIdx.x / KG;
    const int k = (s * KG + threadIdx.x % KG) * STEP;
    if (c >= ld || k >= K) return;
    prefetch_l2(static_cast<const uint8_t*>(w) + first / 2 + c * (K >> 1) + k / 2);
    if (threadIdx.x % KG == 0) prefetch_l2(scales + first / 32 + c * (K >> 5) + k / 32);
  }
  // Token rows times the row's factor for a block (gate_up's have one scale).
  template <int PHASE>
  static __device__ __forceinline__ uint4 scaled(uint4 x, uint32_t f) {
    if (PHASE == 0) return x;
    return make_uint4(mul2(x.x, f), mul2(x.y, f), mul2(x.z, f), mul2(x.w, f));
  }
  // `ring` has the codes: wait() returns the shared address of the next step's,
  // release() gives their place to a later step's.
  template <int NT, int PHASE, class Ring>
  static __device__ __forceinline__ void run(Ring& ring, const uint8_t* scales, int col, int K, int s0,
                                             int s1, int kg, const void* x_rows, const uint8_t* x_scales,
                                             const Row* rows, int nrows, float* red) {
    // A step is two halves: lane t takes the blocks 2 t and 2 t + 1 of a column's
    // eight.  Scale bytes, and with one row tile the tokens, are loaded a step ahead;
    // with two there are no registers for that.  Codes past the end are zeros,
    // whatever their scale and tokens (the last step's).
    constexpr bool EARLY = NT == 1;
    const bool both = NT > 1 && nrows > 8;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int nb = K >> 5;
    float acc[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[m][n][q] = 0.f;
    int b = (s0 * KG + kg) * 8 + 2 * t;         // the blocks whose loads are next: b, b + 1
    const uint8_t* sp = scales + (static_cast<int64_t>(col) + g) * nb + b;
    // two scale bytes in one load where every pair is aligned
    const bool pairs = ((nb | static_cast<int>(reinterpret_cast<uintptr_t>(scales))) & 1) == 0;
    const char* xp = static_cast<const char*>(x_rows) +
                     2 * (static_cast<int64_t>(rows[0].row) * pitch(K) + (s0 * KG + kg) * STEP + 8 * t);
    uint32_t bytes[4], bytes_next[4], xs = 0, xs_next = 0;
    uint4 x[2][EARLY ? 4 : 1];
#pragma unroll
    for (int r = 0; r < 4; ++r) bytes_next[r] = 127 * 0x101, x[0][r % (EARLY ? 4 : 1)] = x[1][r % (EARLY ? 4 : 1)] = make_uint4(0, 0, 0, 0);
    auto load_bytes = [&]() {
      if (pairs) {
        if (b < nb) {
#pragma unroll
          for (int r = 0; r < 4; ++r) bytes_next[r] = ld_u16(sp + r * 8 * nb);
        }
      } else if (b < nb) {
        const int d = b + 1 < nb;               // past the end: the last block's
#pragma unroll
        for (int r = 0; r < 4; ++r) bytes_next[r] = ld_u8(sp + r * 8 * nb) | ld_u8(sp + r * 8 * nb + d) << 8;
      }
    };
    auto load_x = [&](int u) {
      if (EARLY && b + u < nb) {
#pragma unroll
        for (int q = 0; q < 4; ++q) x[u][q % (EARLY ? 4 : 1)] = row_vec(xp + u * 256, q);
      }
    };
    auto load_xs = [&]() {
      if (EARLY && PHASE == 1 && b < nb) {
        xs_next = ld_u16(x_scales + rows[0].row * scale_pitch(K) + b);
        if (b + 1 == nb) xs_next = (xs_next & 0xffu) * 0x101u;
      }
    };
    load_bytes();
    wait_for_rows();
    load_x(0);
    load_x(1);
    load_xs();
    int ref[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
      ref[r] = min(240, static_cast<int>(__shfl_sync(0xffffffffu, bytes_next[r] & 0xffu, lane & 28)));
    // half u of a step, its codes at shared address `at`
    auto half = [&](int u, int s, uint32_t at) {
      uint4 v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = ld_shared_v4(at + r * 8 * (STEP / 2));
      // 2^(q - ref) in fp16, in range for -14 .. 13 (ref <= 240: a NaN's 255 is not)
      uint32_t f[4];
      auto factors = [&]() {
        bool out = false;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t d = (u ? bytes[r] >> 8 : bytes[r] & 0xffu) - ref[r] + 14;
          out = out || d > 27u;
          f[r] = d * 0x04000400u + 0x04000400u;
        }
        return out;
      };
      // the same, with any finite factor for a block of zeros, which needs none
      auto factors_but_zeros = [&]() {
        factors();
        bool out = false;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t byte = u ? bytes[r] >> 8 : bytes[r] & 0xffu;
          if (byte - ref[r] + 14 > 27u) {
            out = out || !zeros(v[r]) || byte == 255u;
            f[r] = 0x3c003c00u;
          }
        }
        return __any_sync(0xffffffffu, out);
      };
      bool far = false;
      if (__builtin_expect(__any_sync(0xffffffffu, factors()), 0)) {
        far = factors_but_zeros();
        if (far) {
          new_ref<NT>(v, bytes, u, ref, acc);
          far = factors_but_zeros();
        }
      }
      uint32_t fx[NT];
      const void* xp[NT];
      const int here = (s * KG + kg) * 8 + 2 * t + u;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        fx[n] = 0;
        // past the end: block 0, which every row has
        xp[n] = static_cast<const __half*>(x_rows) + rows[n].row * pitch(K) +
                (here < nb ? (s * KG + kg) * STEP + u * (STEP / 2) + 8 * t : 0);
        if (PHASE == 1) {
          const uint32_t byte =
              EARLY ? (u ? xs >> 8 : xs & 0xffu) : ld_u8(x_scales + rows[n].row * scale_pitch(K) + (here < nb ? here : 0));
          fx[n] = row_factor(byte, rows[n].top);
        }
      }
      if (__builtin_expect(far, 0)) {
        far_step<NT, PHASE, EARLY>(v, bytes, u, x[u], xp, fx, ref, acc);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t a[4][4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            decode(word(v[r], q), a[r]);
#pragma unroll
            for (int j = 0; j < 4; ++j) a[r][j] = mul2(a[r][j], f[r]);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (n > 0 && !both) continue;
            const uint4 xv = scaled<PHASE>(EARLY ? x[u][q % (EARLY ? 4 : 1)] : row_vec(xp[n], q), fx[n]);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              mma(acc[m][n], a[2 * m][0], a[2 * m + 1][0], a[2 * m][1], a[2 * m + 1][1], xv.x, xv.y);
              mma(acc[m][n], a[2 * m][2], a[2 * m + 1][2], a[2 * m][3], a[2 * m + 1][3], xv.z, xv.w);
            }
          }
        }
      }
      load_x(u);
    };
    // the copies' swizzle has chunk j of row g at j ^ (g & 7): no bank conflicts
    const uint32_t mine = g * (STEP / 2) + ((2 * t) ^ g) * 16;
    for (int s = s0; s < s1; ++s) {
#pragma unroll
      for (int r = 0; r < 4; ++r) bytes[r] = bytes_next[r];
      xs = xs_next;
      b = s + 1 < s1 ? b + KG * 8 : nb;        // (no loads after the last)
      sp += KG * 8;
      xp += KG * 2 * STEP;
      load_bytes();
      load_xs();
      const uint32_t at = ring.wait() + mine;
      half(0, s, at);
      half(1, s, at ^ 16u);
      ring.release();
    }
    // the sums' powers of two: the columns' refs and the token rows' tops
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int t0 = __shfl_sync(0xffffffffu, rows[n].top, 8 * t) - (PHASE == 1 ? kActUp : 0);
      const int t1 = __shfl_sync(0xffffffffu, rows[n].top, 8 * t + 4) - (PHASE == 1 ? kActUp : 0);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int lo = ref[2 * m], hi = ref[2 * m + 1];
        float* d = red + (8 * n + 2 * t) * PITCH + 16 * m + g;
        d[0] = times_scales(acc[m][n][0], lo, t0), d[PITCH] = times_scales(acc[m][n][1], lo, t1);
        d[8] = times_scales(acc[m][n][2], hi, t0), d[PITCH + 8] = times_scales(acc[m][n][3], hi, t1);
      }
    }
  }
  // v * 2^(a - 127) * 2^(b - 127); b = 255: NaN.  One scale after the other could leave
  // fp32's range on the way to a result inside it, so each factor has half of the
  // exponent (2^-126 at the least: below 2^-252 no sum leaves anything).
  static __device__ __forceinline__ float times_scales(float v, int a, int b) {
    const int e = a + b, half = e >> 1;
    const float f = __uint_as_float(static_cast<uint32_t>(max(half, 1)) << 23);
    const float g = __uint_as_float(b == 255 ? 0x7fc00000u : static_cast<uint32_t>(max(e - half, 1)) << 23);
    return v * f * g;
  }

  static __device__ __forceinline__ bool zeros(const uint4& codes) {
    return ((codes.x | codes.y | codes.z | codes.w) & 0x77777777u) == 0;
  }
  // A step with far scales first moves the columns' refs where they do not serve.  A
  // column whose sums are still 0 (its blocks so far were zeros, to which the quantiser
  // gives the byte 0, or met zeros) takes the largest scale of the blocks here that hold
  // something.  One that has sums rises only as far as far_step needs: with
  // 2^(q - ref) <= 2^90 the sums of 2^13 blocks (below 2^23 each) are inside fp32.  The
  // sums lose bits by that only where a column's scales lie more than 2^150 apart.
  template <int NT>
  static __device__ __forceinline__ void new_ref(const uint4 (&v)[4], const uint32_t (&bytes)[4], int u,
                                                 int (&ref)[4], float (&acc)[2][NT][4]) {
    constexpr int kMost = 90;
    // a byte per column: the largest scale byte of the group's blocks, plus one; and a
    // bit per column: whether the group has sums
    uint32_t tops = 0, held = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = r >> 1, q = 2 * (r & 1);
      const uint32_t byte = bytes[r] >> 8 * u & 0xffu;
      if (!zeros(v[r]) && byte != 255u) tops |= (byte + 1) << 8 * r;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (acc[m][n][q] != 0.f || acc[m][n][q + 1] != 0.f) held |= 1u << r;
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      tops = __vmaxu4(tops, __shfl_xor_sync(0xffffffffu, tops, d));
      held |= __shfl_xor_sync(0xffffffffu, held, d);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = r >> 1, q = 2 * (r & 1);
      const int top = static_cast<int>(tops >> 8 * r & 0xffu) - 1;
      int to = ref[r];
      if (top >= 0) to = held >> r & 1 ? max(to, top - kMost) : min(top, 240);
      const float down = pow2(min(0, ref[r] - to));
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n][q] *= down, acc[m][n][q + 1] *= down;
      ref[r] = to;
    }
  }
  // 2^e for e <= 127, 0 below fp32's range.
  static __device__ __forceinline__ float pow2(int e) {
    return __uint_as_float(e >= -126 ? static_cast<uint32_t>(e + 127) << 23 : (e >= -149 ? 1u << (e + 149) : 0u));
  }

  // A step with far scales: the four lanes' blocks one after the other, codes as
  // they are, each block's sums scaled by 2^(q - ref) in fp32.
  template <int NT, int PHASE, bool EARLY>
  static __device__ __forceinline__ void far_step(const uint4 (&v)[4], const uint32_t (&bytes)[4], int u,
                                                  const uint4* x, const void* const (&xp)[NT],
                                                  const uint32_t (&fx)[NT], const int (&ref)[4],
                                                  float (&acc)[2][NT][4]) {
    const int lane = threadIdx.x & 31, t = lane & 3;
#pragma unroll 1
    for (int turn = 0; turn < 4; ++turn) {
      float f[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t byte = __shfl_sync(0xffffffffu, bytes[r], (lane & 28) | turn) >> 8 * u & 0xffu;
        f[r] = byte == 255u ? __uint_as_float(0x7fc00000u) : pow2(static_cast<int>(byte) - ref[r]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float c[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m) c[m][0] = c[m][1] = c[m][2] = c[m][3] = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t a[4][4];
#pragma unroll
          for (int r = 0; r < 4; ++r) decode(t == turn ? word(v[r], q) : 0u, a[r]);
          uint4 xv = scaled<PHASE>(EARLY ? x[q] : row_vec(xp[n], q), fx[n]);
          if (t != turn) xv = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            mma(c[m], a[2 * m][0], a[2 * m + 1][0], a[2 * m][1], a[2 * m + 1][1], xv.x, xv.y);
            mma(c[m], a[2 * m][2], a[2 * m + 1][2], a[2 * m][3], a[2 * m + 1][3], xv.z, xv.w);
          }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          acc[m][n][0] += c[m][0] * f[2 * m], acc[m][n][1] += c[m][1] * f[2 * m];
          acc[m][n][2] += c[m][2] * f[2 * m + 1], acc[m][n][3] += c[m][3] * f[2 * m + 1];
        }
      }
    }
  }
};

// Values with a common scale of 2^p as fp16: p such that the largest magnitude (its
// fp32 bits) lies in [2^top, 2^(top + 1)), see kTokenTop.  Returns the scale's byte; 255
// (NaN) where one is an infinity or a NaN.
__device__ __forceinline__ uint32_t half_block_byte(uint32_t amax_bits, int top) {
  if (amax_bits >= 0x7f800000u) return 255u;
  return static_cast<uint32_t>(max(0, static_cast<int>(amax_bits >> 23) - top));
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight values of e4m3 codes (times their block's scale) or bf16.
template <bool X8>
__device__ __forceinline__ void load_row8(const void* x, const uint8_t* x_scale, int64_t i, float (&v)[8]) {
  if (!X8) {
    load8(static_cast<const __nv_bfloat16*>(x) + 8 * i, v);
    return;
  }
  const uint2 c = __ldg(static_cast<const uint2*>(x) + i);
  const float f = mx_scale(__ldg(x_scale + (i >> 2)));
  const uint32_t q[4] = {c.x, c.x >> 16, c.y, c.y >> 16};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 h = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(q[j] & 0xffffu), __NV_E4M3)));
    v[2 * j] = h.x * f, v[2 * j + 1] = h.y * f;
  }
}

// The counters of both products' joins are cleared by the call itself: a workspace may
// hold anything that earlier calls of other shapes and kinds left in it.
__device__ __forceinline__ void clear_counters(unsigned* counters, int n) {
  for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) counters[i] = 0;
}

// What is left to do before the products where tokens are taken as they are.
__global__ void __launch_bounds__(256) few_clear_kernel(unsigned* counters, int n) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  clear_counters(counters, n);
}

// e4m3 token rows in the storage type (bf16: exact but below its normal range).
template <class S>
__global__ void __launch_bounds__(256) few_rows_kernel(const void* __restrict__ x,
                                                       const uint8_t* __restrict__ x_scale, int vecs,
                                                       S* __restrict__ out, unsigned* counters,
                                                       int ncounters) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  clear_counters(counters, ncounters);
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= vecs) return;
  float v[8];
  load_row8<true>(x, x_scale, i, v);
  store8(out + 8 * static_cast<int64_t>(i), v);
}

// Token rows, a block each, in fp16 with a power of two per row, for 4-bit weights.
// Also clears what the gate_up kernel collects the activations' tops in.
template <bool X8>
__global__ void __launch_bounds__(256) few_half_rows_kernel(const void* __restrict__ x,
                                                            const uint8_t* __restrict__ x_scale, int H,
                                                            __half* __restrict__ out,
                                                            int* __restrict__ top,
                                                            int* __restrict__ act_top, int Tk,
                                                            unsigned* counters, int ncounters) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  clear_counters(counters, ncounters);
  __shared__ uint32_t part[8];
  const int row = blockIdx.x, n = H / 8;
  const int64_t base = static_cast<int64_t>(row) * n;
  for (int i = row * 256 + threadIdx.x; i < Tk; i += gridDim.x * 256) act_top[i] = 0;
  constexpr int kHeld = 4;   // of a thread's vectors, loaded once
  float held[kHeld][8];
  uint32_t amax = 0;
#pragma unroll
  for (int h = 0; h < kHeld; ++h) {
#pragma unroll
    for (int j = 0; j < 8; ++j) held[h][j] = 0.f;
    const int i = threadIdx.x + h * 256;
    if (i < n) load_row8<X8>(x, x_scale, base + i, held[h]);
  }
#pragma unroll
  for (int h = 0; h < kHeld; ++h)
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(held[h][j]) & 0x7fffffffu);
  for (int i = threadIdx.x + kHeld * 256; i < n; i += 256) {
    float v[8];
    load_row8<X8>(x, x_scale, base + i, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7fffffffu);
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) amax = max(amax, part[w]);
  const uint32_t byte = half_block_byte(amax, kTokenTop);
  const float f = mx_inv_scale(byte);
  uint4* row_out = reinterpret_cast<uint4*>(out) + row * static_cast<int64_t>(Mx::pitch(H) / 8);
  auto put = [&](int i, const float (&v)[8]) {
    uint4 u;
    u.x = pack_half(v[0] * f, v[1] * f), u.y = pack_half(v[2] * f, v[3] * f);
    u.z = pack_half(v[4] * f, v[5] * f), u.w = pack_half(v[6] * f, v[7] * f);
    row_out[Mx::chunk_at(i)] = u;
  };
#pragma unroll
  for (int h = 0; h < kHeld; ++h)
    if (threadIdx.x + h * 256 < n) put(threadIdx.x + h * 256, held[h]);
  for (int i = threadIdx.x + kHeld * 256; i < n; i += 256) {
    float v[8];
    load_row8<X8>(x, x_scale, base + i, v);
    put(i, v);
  }
  if (threadIdx.x == 0) top[row] = static_cast<int>(byte);
}

// ------------------------------------------------------------------ kernels
__device__ __forceinline__ float load_elem(const __nv_bfloat16* p, int64_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ float load_elem(const float* p, int64_t i) { return p[i]; }

// A NaN stays a NaN through the clamps.  Both kinds share one sigmoid.
__device__ __forceinline__ float activate(const FewArgs& a, float gate, float up) {
  float z = gate;
  if (a.act_kind != MOE_ACT_SWIGLU) {
    gate = gate > a.limit ? a.limit : gate;
    up = (up > a.limit ? a.limit : (up < -a.limit ? -a.limit : up)) + 1.f;
    z = a.alpha * gate;
  }
  return up * gate * (1.f / (1.f + expf(-z)));
}

// n / d for n >= 0 and quotients below 2^22, by the reciprocal (a handful of
// instructions: what a block runs once it has to fetch first).
__device__ __forceinline__ int quotient(int n, int d, float inv) {
  int q = static_cast<int>(static_cast<float>(n) * inv);
  const int r = n - q * d;
  q += r >= d;
  q -= r < 0;
  return q;
}

// All units' steps cut into `grid` runs of `len` steps, the last one shorter.
struct Runs {
  int grid, len, steps;
  float inv;
  __device__ __forceinline__ Runs(int steps_, int blocks) : steps(steps_) {
    len = max(1, (steps + blocks - 1) / blocks);
    grid = (steps + len - 1) / len;
    inv = 1.f / static_cast<float>(len);
  }
  __device__ __forceinline__ int begin(int c) const { return min(c * len, steps); }
  __device__ __forceinline__ int block_of(int s) const { return quotient(s, len, inv); }
};

// Floats of `red`: the shares' results, or the 256 threads' sums of the combine.
template <class W>
__host__ __device__ __forceinline__ int red_floats(int rows) {
  const int n = (W::KG * W::PITCH * rows + 3) & ~3;
  return n > 4 * kThreads ? n : 4 * kThreads;
}

template <class W>
__host__ __device__ constexpr int ring_slot() {
  if constexpr (W::kRing > 0) return W::kSlotBytes;
  return 0;
}
// Bytes of the warps' rings, their barriers and the way to a multiple of 1024.
template <class W>
__host__ __device__ constexpr int ring_bytes() {
  return W::kRing ? kThreads / 32 * W::kRing * (ring_slot<W>() + 8) + 1008 : 0;
}

// The biases of this thread's output in a unit: thread i has output i % OUT of every
// kThreads / OUT-th row.
template <class W>
__device__ __forceinline__ float2 unit_bias(const FewArgs& a, int e, int tile) {
  using S = typename W::Store;
  constexpr int OUT = W::FG * W::WF / 2;
  const int feature = tile * OUT + threadIdx.x % OUT;
  if (!a.bias || feature >= a.I) return make_float2(0.f, 0.f);
  const S* b = static_cast<const S*>(a.bias) + static_cast<int64_t>(e) * 2 * a.I;
  return make_float2(load_elem(b, a.interleaved ? 2 * feature : feature),
                     load_elem(b, a.interleaved ? 2 * feature + 1 : a.I + feature));
}

// The activation of a unit's results, the sums of `shares` of red[share][row][column],
// into its rows of a.act.
template <class W, int SHARES>
__device__ __forceinline__ void finish_gate_up(const FewArgs& a, const Plan& p, const float* red,
                                               int chunk, int tile, float2 bias) {
  using S = typename W::Store;
  constexpr int OUT = W::FG * W::WF / 2;
  static_assert(kThreads % OUT == 0 && OUT % 32 == 0, "a warp has 32 outputs of a row");
  const int first = p.chunk_first[chunk], nrows = p.chunk_rows[chunk];
  const int f = threadIdx.x % OUT, feature = tile * OUT + f;
  if (feature >= a.I) return;
  for (int r = threadIdx.x / OUT; r < nrows; r += kThreads / OUT) {
    const float* q = red + r * W::PITCH;
    const int at_gate = a.interleaved ? 2 * f : f, at_up = a.interleaved ? 2 * f + 1 : f + OUT;
    float gate = q[at_gate], up = q[at_up];
#pragma unroll
    for (int j = 1; j < SHARES; ++j) {
      q += a.rows * W::PITCH;
      gate += q[at_gate], up += q[at_up];
    }
    gate += bias.x, up += bias.y;
    const float v = activate(a, gate, up);
    const int64_t slot = p.slot[first + r];
    if constexpr (!W::kHalfRows) {
      static_cast<S*>(a.act)[slot * a.I + feature] = static_cast<S>(v);
    } else {
      // a warp has the 32 values of one block (I is a multiple of 32)
      const uint32_t byte =
          half_block_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7fffffffu), kActTop);
      static_cast<__half*>(a.act)[slot * W::pitch(a.I) + 8 * W::chunk_at(feature >> 3) + (feature & 7)] =
          __float2half_rn(v * mx_inv_scale(byte));
      if ((threadIdx.x & 31) == 0) {
        a.act_scale[slot * W::scale_pitch(a.I) + (feature >> 5)] = static_cast<uint8_t>(byte);
        if (byte != 255u) atomicMax(a.act_top + slot, static_cast<int>(byte));
      }
    }
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

// Four of a bias row's values.
__device__ __forceinline__ float4 bias4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
}
__device__ __forceinline__ float4 bias4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// y of one column tile from every chunk's products: whole units' in a.o, cut
// ones' in their blocks' parts.  A block runs this once or twice, so most of its
// time is the fetch of its instructions: it is kept small.
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
  // With few tokens a token's choices are shared out over 2^shift threads (every
  // 2^shift-th choice each) whose sums are added in order.
  const int items = a.T * V;
  int shift = 0;
  while ((items << (shift + 1)) <= kThreads && (1 << shift) < a.k) ++shift;
  float4* sums = reinterpret_cast<float4*>(red);
#pragma unroll 1
  for (int i = threadIdx.x; i < items << shift; i += kThreads) {
    const int f = i % V * 4, tok = i / V >> shift, group = (i / V) & ((1 << shift) - 1);
    const int c = tile * CW + f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int j = group; j < a.k && c < a.H; j += 1 << shift) {
      const int slot = tok * a.k + j;
      const int at = p.where[slot];
      if (at == kNowhere) continue;
      const float w = __ldg(a.topk_w + slot);
      const uint32_t sp = p.span[at >> 5];
      const int f0 = sp & 0x7fff;
      int n = static_cast<int>((sp >> 15) & 0x7fff) - f0;
      const float* next = a.part + 2 * static_cast<int64_t>(f0) * UNIT + (at & 31) * CW + f;
      float4 v = ldcg4(n ? next + (sp >> 30) * UNIT : a.o + static_cast<int64_t>(slot) * a.H + c);
      float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.bias) bias = bias4(static_cast<const S*>(a.bias) + static_cast<int64_t>(p.chunk_e[at >> 5]) * a.H + c);
#pragma unroll 1
      for (; n > 0; n -= 3) {   // three parts' loads at a time
        float4 o[3];
#pragma unroll
        for (int b = 0; b < 3; ++b) {
          next += 2 * UNIT;
          o[b] = b < n ? ldcg4(next) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int b = 0; b < 3; ++b) add4(v, o[b]);
      }
      add4(v, bias);
      y.x = fmaf(w, v.x, y.x), y.y = fmaf(w, v.y, y.y);
      y.z = fmaf(w, v.z, y.z), y.w = fmaf(w, v.w, y.w);
    }
    if (shift == 0)
      store_y<S>(a, tok, c, y);
    else
      sums[i] = y;
  }
  if (shift > 0) {
    __syncthreads();
    for (int i = threadIdx.x; i < items; i += kThreads) {
      const int at = (i / V << shift) * V + i % V;
      float4 y = sums[at];
      for (int g = 1; g < 1 << shift; ++g) add4(y, sums[at + g * V]);
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
template <class W, int PHASE, int NT>
__global__ void __launch_bounds__(kThreads, 2) few_kernel(const __grid_constant__ FewArgs a) {
  using S = typename W::Store;
  constexpr int CW = W::FG * W::WF;            // weight columns of a unit
  const int UNIT = a.rows * CW;                // results of a unit, [row][column]
  const int SHARE = a.rows * W::PITCH;         // one share's results in shared memory
  constexpr int OUT = PHASE == 0 ? CW / 2 : CW;
  extern __shared__ float4 dynamic[];          // results, plan
  float* const reds = reinterpret_cast<float*>(dynamic);
  float* red = reds;
  __shared__ PlanSmall ps;
  Plan p = plan_at(reds + 2 * red_floats<W>(a.rows), a.T * a.k, a.E, a.rows);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int fg = warp % W::FG, kg = warp / W::FG;
  uint32_t slots = 0, bars = 0;                // this warp's ring
  if (W::kRing > 0) {
    slots = (smem_u32(dynamic) + red_floats<W>(a.rows) * 8 + plan_bytes(a.T * a.k, a.E, a.rows) + 1023) & ~1023u;
    bars = slots + kThreads / 32 * W::kRing * ring_slot<W>() + warp * W::kRing * 8;
    slots += warp * W::kRing * ring_slot<W>();
    if (lane == 0) {
      for (int i = 0; i < W::kRing; ++i) mbar_init(bars + 8 * i, 1);
      fence_barrier_init();
    }
    __syncwarp();
  }
  const int me = blockIdx.x;
  if (PHASE == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  build_plan(p, ps, a.idx, a.T * a.k, a.E, a.rows, PHASE == 0 ? a.err : nullptr);

  const int K = PHASE == 0 ? a.H : a.I;                // contraction
  const int N = PHASE == 0 ? 2 * a.I : a.H;            // weight columns
  const int tiles = ((PHASE == 0 ? a.I : a.H) + OUT - 1) / OUT;
  const int KS = (K + W::KG * W::STEP - 1) / (W::KG * W::STEP);
  const int chunks = p.chunks;
  const Runs runs(chunks * tiles * KS, gridDim.x);
  const float inv_KS = 1.f / static_cast<float>(KS), inv_chunks = 1.f / static_cast<float>(chunks);
  if (me >= runs.grid) {
    wait_for_rows();
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
  // this warp's first weight column in a tile, and how many there are from it on
  auto columns = [&](int tile, int* col, int* ncol) {
    if (PHASE == 0 && !a.interleaved) {
      constexpr int HALF = W::FG / 2;
      const int o = tile * OUT + (fg % HALF) * W::WF;
      *col = (fg / HALF) * a.I + o;
      *ncol = a.I - o;
    } else {
      *col = tile * CW + fg * W::WF;
      *ncol = N - *col;
    }
  };

  // The ring runs through all of the block's steps, whatever unit they are of.
  constexpr uint32_t kSlots = W::kRing ? W::kRing : 1;   // a power of two
  struct Ring {
    int next, left;            // the step to load next; steps left of its unit, or -1:
                               // a copy did not come in time, no more are made
    int k, col, e;             // where its codes are
    uint32_t used;             // steps taken out
  } at = {begin, 0, 0, 0, 0, 0};
  auto load_next = [&](uint32_t slot) {
    while (at.left == 0) {
      if (at.next >= end) return;
      const int unit = quotient(at.next, KS, inv_KS), tile = quotient(unit, chunks, inv_chunks);
      int ncol;
      columns(tile, &at.col, &ncol);
      const int stop = min(end, (unit + 1) * KS);
      if (ncol <= 0) {
        at.next = stop;
        continue;
      }
      at.left = stop - at.next;
      at.k = ((at.next - unit * KS) * W::KG + kg) * (W::STEP / 2);
      at.e = p.chunk_e[unit - tile * chunks];
      // the first of the unit's scale bytes, a column per lane
      prefetch_l2(a.scales + (static_cast<int64_t>(at.e) * N + min(at.col + lane, N - 1)) * (K >> 5) +
                  min(at.k >> 4, (K >> 5) - 1));
    }
    if (lane == 0) {
      mbar_arrive_expect_tx(bars + 8 * slot, ring_slot<W>());
      tma_load_3d(slots + slot * ring_slot<W>(), &a.codes, bars + 8 * slot, at.k, at.col, at.e);
    }
    ++at.next, --at.left;
    at.k += W::KG * W::STEP / 2;
  };
  struct {
    decltype(load_next)& load;
    Ring& at;
    uint32_t slots, bars;
    uint64_t timeout_ns;
    int* err;
    __device__ __forceinline__ uint32_t wait() {
      const uint32_t slot = at.used % kSlots, phase = at.used / kSlots & 1;
      if (__builtin_expect(!__all_sync(0xffffffffu, mbar_try_wait(bars + 8 * slot, phase)), 0)) {
        if (!__all_sync(0xffffffffu, at.left >= 0 && mbar_wait(bars + 8 * slot, phase, timeout_ns))) {
          record_error(err, kErrTimeout);
          at.left = -1;
        }
      }
      return slots + slot * ring_slot<W>();
    }
    __device__ __forceinline__ void release() {
      __syncwarp();
      if (at.left < 0) return;
      load(at.used % kSlots);
      ++at.used;
    }
  } ring = {load_next, at, slots, bars, a.timeout_ns, a.err};
  if (W::kRing > 0)
    for (int i = 0; i < W::kRing; ++i) load_next(i);

  for (int s = begin; s < end;) {
    const int unit = quotient(s, KS, inv_KS);
    const int u0 = unit * KS;
    const int ks0 = s - u0;
    const int ks1 = min(KS, end - u0);
    const int tile = quotient(unit, chunks, inv_chunks), chunk = unit - tile * chunks;
    const int e = p.chunk_e[chunk], first = p.chunk_first[chunk], nrows = p.chunk_rows[chunk];

    int col, ncol;
    columns(tile, &col, &ncol);
    // the biases that the finishing block will want (128-byte lines)
    if (a.bias && lane == 0 && kg == 0 && ncol > 0)
      prefetch_l2(static_cast<const S*>(a.bias) + static_cast<int64_t>(e) * N + col);
    Row rows[W::kRowPerLane ? NT : 8];
#pragma unroll
    for (int i = 0; i < (W::kRowPerLane ? NT : 8); ++i) {
      const int r = W::kRowPerLane ? 8 * i + (lane >> 2) : i;
      const int slot = p.slot[first + (r < nrows ? r : 0)];
      const int64_t row = PHASE == 0 ? slot / a.k : slot;
      if constexpr (!W::kHalfRows) {
        rows[i].p = static_cast<const S*>(a.x) + row * K;
      } else {
        rows[i].row = static_cast<int>(row);
        wait_for_rows();
        rows[i].top = static_cast<int>(ld_u32(a.top + row));
      }
    }
    if (ncol > 0) {
      const int64_t we = static_cast<int64_t>(e) * K * N;   // weights of the experts before
      float* out = red + kg * SHARE + fg * W::WF;
      if constexpr (W::kRing > 0)
        W::template run<NT, PHASE>(ring, a.scales + we / 32, col, K, ks0, ks1, kg, a.x, a.x_scale, rows, nrows,
                                    out);
      else
        W::template run<NT>(static_cast<const S*>(a.w) + we, N, col, ncol, K, ks0, ks1, kg, rows, nrows, out);
    }
    const bool whole = ks1 - ks0 == KS;
    float2 bias = make_float2(0.f, 0.f);
    if (PHASE == 0 && whole) bias = unit_bias<W>(a, e, tile);
    __syncthreads();

    // A whole unit of gate_up is finished here; else the shares of the contraction
    // are added, a cut unit's into its part, a whole one's into its rows of o.
    if (PHASE == 0 && whole) {
      finish_gate_up<W, W::KG>(a, p, red, chunk, tile, bias);
    } else {
      float* part = a.part + (2 * static_cast<int64_t>(me) + (begin >= u0 ? 0 : 1)) * UNIT;
      for (int i = tid; i < nrows * CW; i += kThreads) {
        const int f = i % CW, r = i / CW, q = r * W::PITCH + f;
        float v = red[q];
#pragma unroll
        for (int j = 1; j < W::KG; ++j) v += red[j * SHARE + q];
        if (!whole)
          part[i] = v;
        else if (tile * OUT + f < a.H)
          a.o[static_cast<int64_t>(p.slot[first + r]) * a.H + tile * OUT + f] = v;
      }
    }
    // the next unit's results go to the other half of `red`, so that they need not
    // wait for these to be read
    red = red == reds ? reds + red_floats<W>(a.rows) : reds;
    // a tile that lies in this run alone
    if (PHASE == 1 && chunk == chunks - 1 && ks1 == KS && begin <= tile * chunks * KS) {
      __syncthreads();
      combine_tile<W>(a, p, runs, KS, tile, red);
    }
    s = u0 + ks1;
  }
  if (W::kRing > 0 && at.left < 0)   // no copy is in flight when the block ends
    for (uint32_t i = at.used; i < at.used + kSlots; ++i)
      mbar_wait(bars + 8 * (i % kSlots), i / kSlots & 1, kDrainNs);
  __syncthreads();

  wait_for_rows();   // (warps without columns have not yet)

  // the pieces at the run's ends: piece 0 its first unit (tile), 1 its last
  const int per = PHASE == 0 ? KS : chunks * KS;       // steps of a unit (tile)
  const float inv_per = PHASE == 0 ? inv_KS : inv_KS * inv_chunks;
  const int p0 = quotient(begin, per, inv_per), p1 = quotient(end - 1, per, inv_per);
  int last = 0;
  if (tid < 2) {
    const int piece = tid ? p1 : p0;
    const int lo = max(begin, piece * per), hi = min(end, (piece + 1) * per);
    if (hi - lo < per && (tid == 0 || p1 != p0)) {
      // a unit's counter is its first block's (a block is the first of at most one cut unit)
      unsigned* c = a.counters + (PHASE == 0 ? runs.block_of(piece * per) : piece);
      last = join_add(c, hi - lo) + (hi - lo) == static_cast<unsigned>(per);
    }
    ps.last[tid] = last;
  }
  // Until the last blocks are done HBM has little to do: the first steps of what
  // this block's number does in the down kernel go to L2 meanwhile.
  if (PHASE == 0) {
    const int tiles2 = (a.H + CW - 1) / CW, KS2 = (a.I + W::KG * W::STEP - 1) / (W::KG * W::STEP);
    const Runs next(chunks * tiles2 * KS2, gridDim.x);
    const int from = next.begin(me), to = me < next.grid ? min(next.begin(me + 1), from + kPrefetchSteps / (W::kRing ? 2 : 1)) : 0;
    const float inv_KS2 = 1.f / static_cast<float>(KS2);
#pragma unroll 1
    for (int s = from; s < to; ++s) {
      const int unit = quotient(s, KS2, inv_KS2), tile = quotient(unit, chunks, inv_chunks);
      const int e = p.chunk_e[unit - tile * chunks];
      W::prefetch(a.w_next, a.scales_next, static_cast<int64_t>(e) * a.I * a.H, a.H, tile * CW, a.I,
                  s - unit * KS2);
      if (a.bias_next && s == from && tid < CW / 32 && tile * CW + tid * 32 < a.H)
        prefetch_l2(static_cast<const S*>(a.bias_next) + static_cast<int64_t>(e) * a.H + tile * CW + tid * 32);
    }
    if (tid < a.T * a.k && me < 32) prefetch_l2(a.topk_w + tid);
  }
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    if (!ps.last[i]) continue;
    const int piece = i ? p1 : p0;
    if (PHASE == 1) {
      combine_tile<W>(a, p, runs, KS, piece, red);
      continue;
    }
    const int tile = quotient(piece, chunks, inv_chunks), chunk = piece - tile * chunks;
    const int nrows = p.chunk_rows[chunk];
    const int c0 = runs.block_of(piece * KS), c1 = runs.block_of(piece * KS + KS - 1);
    const float* head = a.part + (2 * static_cast<int64_t>(c0) + (runs.begin(c0) >= piece * KS ? 0 : 1)) * UNIT;
    const float2 bias = unit_bias<W>(a, p.chunk_e[chunk], tile);
#pragma unroll 1
    for (int j = tid * 4; j < nrows * CW; j += kThreads * 4) {
      float4 v = ldcg4(head + j);
#pragma unroll 2
      for (int c = c0 + 1; c <= c1; ++c) add4(v, ldcg4(a.part + 2 * static_cast<int64_t>(c) * UNIT + j));
      float* d = red + j / CW * W::PITCH + j % CW;
      d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
    }
    __syncthreads();
    finish_gate_up<W, 1>(a, p, red, chunk, tile, bias);
    __syncthreads();
  }
}

// May start while the kernel before it, which writes its rows, ends.
template <class W, int PHASE, int NT>
cudaError_t launch(const FewArgs& a, int grid, cudaStream_t st) {
  const int smem = red_floats<W>(a.rows) * 8 + plan_bytes(a.T * a.k, a.E, a.rows) + ring_bytes<W>();
  const int most = red_floats<W>(8 * NT) * 8 + kMostPlanBytes + ring_bytes<W>();
  static std::atomic<uint64_t> ready{0};   // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(few_kernel<W, PHASE, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
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
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_kernel<W, PHASE, NT>, a);
}

template <class W, int PHASE>
cudaError_t launch_nt(const FewArgs& a, int nt, int grid, cudaStream_t st) {
  if constexpr (W::kMaxTiles > 1) {
    if (nt > 1) return launch<W, PHASE, W::kMaxTiles>(a, grid, st);
  }
  return launch<W, PHASE, 1>(a, grid, st);
}

// The kernel before the products: x as gate_up wants it (x_scale: e4m3, half: fp16;
// H % 32 == 0), counters cleared.
cudaError_t launch_rows(const moe_shape* s, const void* x, const uint8_t* x_scale, bool half, void* out,
                        int* top, int* act_top, unsigned* counters, int ncounters, cudaStream_t st) {
  const int T = static_cast<int>(s->T), Tk = T * s->k;
  const int vecs = T * (s->H / 8), grid = (vecs + 255) / 256;
  if (half && x_scale)
    few_half_rows_kernel<true><<<T, 256, 0, st>>>(x, x_scale, s->H, static_cast<__half*>(out), top, act_top, Tk, counters, ncounters);
  else if (half)
    few_half_rows_kernel<false><<<T, 256, 0, st>>>(x, x_scale, s->H, static_cast<__half*>(out), top, act_top, Tk, counters, ncounters);
  else if (!x_scale)
    few_clear_kernel<<<1, 256, 0, st>>>(counters, ncounters);
  else if (s->dtype == MOE_FP32)
    few_rows_kernel<float><<<grid, 256, 0, st>>>(x, x_scale, vecs, static_cast<float*>(out), counters, ncounters);
  else
    few_rows_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(x, x_scale, vecs, static_cast<__nv_bfloat16*>(out), counters, ncounters);
  return cudaGetLastError();
}

// Row tiles of 8 tokens per unit.  Two where an expert may have more than 8 rows,
// so that its weights are read and decoded once for 16.  4-bit weights take two only
// from 8 rows per expert on: the kernel for one tile has its tokens' loads ahead.
// (One and two tiles, 32 experts of 2880 x 2880, top-4: 48 tokens 146 and 171 us, 64
// tokens 187 and 185, 96 tokens 246 and 210.)  fp32: one.
int row_tiles(const moe_shape* s, bool mx) {
  if (s->dtype == MOE_FP32 || s->T <= 8) return 1;
  return mx && s->T * s->k < 8ll * s->E ? 1 : 2;
}

struct FewLayout {
  size_t counters0, counters1, rows, top, act, act_scale, act_top, part, o, total;
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
  L.rows = take((s->dtype == MOE_FP32 ? 4 : 2) * static_cast<size_t>(s->T) * Mx::pitch(s->H));
  L.top = take(sizeof(int) * static_cast<size_t>(s->T));
  L.act_top = take(sizeof(int) * Tk);
  L.act_scale = take(Tk * Mx::scale_pitch(s->I));
  L.act = take((s->dtype == MOE_FP32 ? 4 : 2) * Tk * Mx::pitch(s->I));
  L.part = take(sizeof(float) * 2 * kMaxGrid * kMaxCW * (s->T <= 8 ? 8 : 16));
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
  a.w_next = mx ? mx->codes_down : w_down;
  a.scales_next = mx ? mx->scales_down : nullptr;
  a.bias_next = bias ? bias->b_down : nullptr;
  a.act = base + L.act;
  a.act_scale = reinterpret_cast<uint8_t*>(base + L.act_scale);
  a.act_top = reinterpret_cast<int*>(base + L.act_top);
  a.top = reinterpret_cast<const int*>(base + L.top);
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
  a.timeout_ns = abi_wait_timeout_ns();
  CUtensorMap down_codes;
  if (mx && !(abi_map_bytes(&a.codes, mx->codes_gate_up, s->H / 2, 2 * static_cast<uint64_t>(s->I), s->E,
                            Mx::STEP / 2, Mx::WF, CU_TENSOR_MAP_SWIZZLE_128B) &&
              abi_map_bytes(&down_codes, mx->codes_down, s->I / 2, s->H, s->E, Mx::STEP / 2, Mx::WF,
                            CU_TENSOR_MAP_SWIZZLE_128B)))
    return MOE_ERR_CUDA;
  const int nt = row_tiles(s, mx != nullptr);
  a.rows = 8 * nt;

  if (x_scale || mx) a.x = base + L.rows;
  cudaError_t e = abi_tracked(kAbiFewRows, 1, st, [&] {
    return launch_rows(s, x, x_scale, mx != nullptr, base + L.rows, reinterpret_cast<int*>(base + L.top), a.act_top,
                       a.counters, static_cast<int>((L.rows - L.counters0) / sizeof(unsigned)), st);
  });
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  e = abi_tracked(kAbiFewGateUp, 1, st, [&] {
    if (s->dtype == MOE_FP32) return launch_nt<F32, 0>(a, nt, grid, st);
    if (mx) return launch_nt<Mx, 0>(a, nt, grid, st);
    return launch_nt<Bf16, 0>(a, nt, grid, st);
  });
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  a.x = a.act;
  a.x_scale = a.act_scale;
  a.top = a.act_top;
  if (mx) a.codes = down_codes;
  a.w = mx ? mx->codes_down : w_down;
  a.scales = mx ? mx->scales_down : nullptr;
  a.bias = bias ? bias->b_down : nullptr;
  a.counters = reinterpret_cast<unsigned*>(base + L.counters1);
  e = abi_tracked(kAbiFewDown, 1, st, [&] {
    if (s->dtype == MOE_FP32) return launch_nt<F32, 1>(a, nt, grid, st);
    if (mx) return launch_nt<Mx, 1>(a, nt, grid, st);
    return launch_nt<Bf16, 1>(a, nt, grid, st);
  });
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
