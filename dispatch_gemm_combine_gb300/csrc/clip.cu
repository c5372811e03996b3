// The global norm of a list of gradients, and clipping by it:
//   norm = sqrt(sum over all tensors of g^2),  coef = min(1, max_norm / (norm + 1e-6)),
//   dst = coef * src.
//
// Two passes over memory, both HBM-bound: one reads every gradient, the other
// reads it again and writes it scaled.  The second walks the chunks from the
// last to the first, so it starts with what the first left in the L2 cache, and
// where nothing is clipped an entry that is scaled in place is not touched.
// The list is a kernel argument (kBatch tensors per launch), so it needs no
// device memory and a captured graph holds its own copy.
//
// The sum: each thread squares and adds the few dozen values of one chunk in
// fp32; from there on sums are pairs of fp32 values (the sum and what it rounded
// off), in a fixed order: every block of the second pass adds all blocks' sums by
// index, so nothing but those sums goes from one kernel to the other.  (Doubles in
// their place take 2 us more on a short list: this GPU adds few a clock.)
// Squares of fp32 values leave fp32's range beyond 2^64 and below 2^-63, so
// three sums run side by side, of g^2, (2^-80 g)^2 and (2^80 g)^2, and the
// final step takes the one in range; the arithmetic is a tenth of what the
// loads leave room for.
//
// Measured: 796 M fp32 values in 1.41 ms, 6.8 TB/s of what two reads and a write
// move; a dozen small tensors in 13 us, two launches.
#include <algorithm>
#include <cmath>

#include "abi_internal.h"
#include "vec.cuh"

namespace moe {
namespace {

constexpr int kBatch = 96;           // tensors per launch (a 2.9 KB kernel argument)
constexpr int kChunk = 8192;         // elements of one block's step
constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 8;
constexpr int kMaxBlocks = kBlocksPerSm * 256;   // of any device
constexpr float kUp = 0x1p80f;
constexpr float kDown = 0x1p-80f;

struct GradTable {
  const void* src[kBatch];
  void* dst[kBatch];
  long long n[kBatch];
  int chunk0[kBatch + 1];   // first chunk of each tensor
  uint8_t bf16[kBatch];
  uint8_t vec[kBatch];      // 16-byte accesses: src and dst are aligned for them
  int count;
};

// A sum as its rounded value and the rest.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair operator+(const Pair& a, const Pair& b) {
  const float s = a.hi + b.hi;
  if (!isfinite(s)) return {s, 0.f};
  const float v = s - a.hi;
  const float e = ((a.hi - (s - v)) + (b.hi - v)) + (a.lo + b.lo);
  const float hi = s + e;
  return {hi, e - (hi - s)};
}
struct Sums {
  Pair mid, big, small;
};
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return {a.mid + b.mid, a.big + b.big, a.small + b.small};
}

// The whole warp asks for the same chunk; a lane looks at every 32nd tensor (one
// round of loads in place of a search's seven, each waiting for the one before).
__device__ __forceinline__ int tensor_of_chunk(const GradTable& t, int chunk) {
  int k = 0;
  for (int i = threadIdx.x & 31; i - static_cast<int>(threadIdx.x & 31) < t.count; i += 32)
    k += __popc(__ballot_sync(0xffffffffu, i < t.count && t.chunk0[i + 1] <= chunk));
  return k;
}

struct Acc {
  float mid = 0.f, big = 0.f, small = 0.f;
  __device__ __forceinline__ void add(float g) {
    const float b = g * kDown, s = g * kUp;
    mid = fmaf(g, g, mid);
    big = fmaf(b, b, big);
    small = fmaf(s, s, small);
  }
};

__device__ __forceinline__ float elem(const float* p, long long i) { return __ldg(p + i); }
__device__ __forceinline__ float elem(const __nv_bfloat16* p, long long i) {
  return __bfloat162float(p[i]);
}

template <typename E>
__device__ __forceinline__ void sum_chunk(const E* p, int n, bool vec, Acc& acc) {
  constexpr int W = 16 / sizeof(E);
  int done = 0;
  if (vec) {
    const uint4* q = reinterpret_cast<const uint4*>(p);
    const int nv = n / W;
    constexpr int U = 4;
    int i = threadIdx.x;
    for (; i + (U - 1) * kThreads < nv; i += U * kThreads) {
      uint4 u[U];
#pragma unroll
      for (int j = 0; j < U; ++j) u[j] = __ldg(q + i + j * kThreads);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (sizeof(E) == 4) {
            acc.add(__uint_as_float(w[k]));
          } else {
            acc.add(bf16_lo(w[k]));
            acc.add(bf16_hi(w[k]));
          }
        }
      }
    }
    for (; i < nv; i += kThreads) {
      const uint4 u = __ldg(q + i);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (sizeof(E) == 4) {
          acc.add(__uint_as_float(w[k]));
        } else {
          acc.add(bf16_lo(w[k]));
          acc.add(bf16_hi(w[k]));
        }
      }
    }
    done = nv * W;
  }
  for (int i = done + threadIdx.x; i < n; i += kThreads) acc.add(elem(p, i));
}

__device__ __forceinline__ Pair warp_sum(Pair v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    v = v + Pair{__shfl_xor_sync(0xffffffffu, v.hi, d), __shfl_xor_sync(0xffffffffu, v.lo, d)};
  return v;
}

// Sum over the block in a fixed order; valid in thread 0.
__device__ __forceinline__ Sums block_sums(Sums v, Sums* part) {
  v = {warp_sum(v.mid), warp_sum(v.big), warp_sum(v.small)};
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < kThreads / 32; ++w) v = v + part[w];
  return v;
}

// sqrt(v) with the rest taken in: one step of Newton's iteration on fp32's root.
__device__ __forceinline__ float root(const Pair& v) {
  const float s = sqrtf(v.hi);
  return s > 0.f && isfinite(s) ? s + (fmaf(-s, s, v.hi) + v.lo) / (2.f * s) : s;
}

// `first`: this launch's place in the blocks' sums.
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ GradTable t,
                                                             int first, Sums* sums) {
  __shared__ Sums part[kThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Sums s{};
  const int chunks = t.chunk0[t.count];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int k = tensor_of_chunk(t, c);
    const long long i0 = static_cast<long long>(c - t.chunk0[k]) * kChunk;
    const int n = static_cast<int>(min(static_cast<long long>(kChunk), t.n[k] - i0));
    Acc a;
    if (t.bf16[k])
      sum_chunk(static_cast<const __nv_bfloat16*>(t.src[k]) + i0, n, t.vec[k], a);
    else
      sum_chunk(static_cast<const float*>(t.src[k]) + i0, n, t.vec[k], a);
    s = s + Sums{{a.mid, 0.f}, {a.big, 0.f}, {a.small, 0.f}};
  }
  const Sums b = block_sums(s, part);
  if (threadIdx.x == 0) sums[first + blockIdx.x] = b;
}

// (norm, coef) of all blocks' sums, the same in every thread of every block.
__device__ __forceinline__ float2 norm_and_coef(const Sums* sums, int blocks, float max_norm) {
  __shared__ Sums part[kThreads / 32];
  __shared__ float2 result;
  Sums v{};
  for (int i = threadIdx.x; i < blocks; i += kThreads) {
    const float2* q = reinterpret_cast<const float2*>(sums + i);
    const float2 m = __ldcg(q), b = __ldcg(q + 1), s = __ldcg(q + 2);
    v = v + Sums{{m.x, m.y}, {b.x, b.y}, {s.x, s.y}};
  }
  v = block_sums(v, part);
  if (threadIdx.x == 0) {
    // |g| <= 2^-20 throughout where the middle sum is below 2^-40, so the
    // scaled-up squares stay in range there
    float norm;
    if (!isfinite(v.mid.hi))
      norm = root(v.big) * 0x1p80f;
    else if (v.mid.hi < 0x1p-40f)
      norm = root(v.small) * 0x1p-80f;
    else
      norm = root(v.mid);
    const float c = max_norm / (norm + 1e-6f);
    result = make_float2(norm, isfinite(norm) && c < 1.f ? c : 1.f);
  }
  __syncthreads();
  return result;
}

template <typename E>
__device__ __forceinline__ void scale_chunk(const E* p, E* d, int n, bool vec, float c) {
  constexpr int W = 16 / sizeof(E);
  const bool copy = c == 1.f;   // bits and all: a product would rewrite a NaN's
  int done = 0;
  if (vec) {
    const uint4* q = reinterpret_cast<const uint4*>(p);
    uint4* o = reinterpret_cast<uint4*>(d);
    const int nv = n / W;
    constexpr int U = 4;
    for (int i0 = threadIdx.x; i0 < nv; i0 += U * kThreads) {
      uint4 u[U];
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (i0 + j * kThreads < nv) u[j] = q[i0 + j * kThreads];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (i0 + j * kThreads >= nv) break;
        uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
        for (int k = 0; k < 4 && !copy; ++k)
          w[k] = sizeof(E) == 4 ? __float_as_uint(__uint_as_float(w[k]) * c)
                                : pack_bf16(bf16_lo(w[k]) * c, bf16_hi(w[k]) * c);
        o[i0 + j * kThreads] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    done = nv * W;
  }
  for (int i = done + threadIdx.x; i < n; i += kThreads)
    d[i] = copy ? p[i] : static_cast<E>(static_cast<float>(p[i]) * c);
}

// `out`: where the norm and the factor go, or null.  Five blocks per SM: with the 54
// registers that the compiler would take four fit (796 M values: 28 us more); with six
// or eight, those for the loads in flight are short (97 and 430 us more).
__global__ void __launch_bounds__(kThreads, 5) grad_scale_kernel(const __grid_constant__ GradTable t,
                                                              const Sums* sums, int blocks,
                                                              float max_norm, float* out) {
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the sums are there
  const float2 result = norm_and_coef(sums, blocks, max_norm);
  const float c = result.y;
  if (out && blockIdx.x == 0 && threadIdx.x == 0) out[0] = result.x, out[1] = c;
  const int chunks = t.chunk0[t.count];
  for (int r = blockIdx.x; r < chunks; r += gridDim.x) {
    const int ch = chunks - 1 - r;
    const int k = tensor_of_chunk(t, ch);
    if (!t.dst[k] || (c == 1.f && t.dst[k] == t.src[k])) continue;
    const long long i0 = static_cast<long long>(ch - t.chunk0[k]) * kChunk;
    const int n = static_cast<int>(min(static_cast<long long>(kChunk), t.n[k] - i0));
    if (t.bf16[k])
      scale_chunk(static_cast<const __nv_bfloat16*>(t.src[k]) + i0,
                  static_cast<__nv_bfloat16*>(t.dst[k]) + i0, n, t.vec[k], c);
    else
      scale_chunk(static_cast<const float*>(t.src[k]) + i0, static_cast<float*>(t.dst[k]) + i0, n,
                  t.vec[k], c);
  }
}

bool grads_ok(const moe_grad_t* g, int64_t n) {
  if (n < 0 || (n > 0 && !g)) return false;
  for (int64_t i = 0; i < n; ++i) {
    if (g[i].n < 0 || (g[i].dtype != MOE_BF16 && g[i].dtype != MOE_FP32)) return false;
    if (g[i].n > 0) {
      const uintptr_t align = g[i].dtype == MOE_FP32 ? 3 : 1;
      if (!g[i].src || (reinterpret_cast<uintptr_t>(g[i].src) & align) ||
          (reinterpret_cast<uintptr_t>(g[i].dst) & align))
        return false;
      if (g[i].n > (static_cast<int64_t>(1) << 42)) return false;
    }
  }
  return true;
}

// The tensors from g[i] on that go into one launch: at most kBatch of them and
// fewer than 2^31 chunks.  A tensor larger than that is not split.
int64_t fill_table(const moe_grad_t* g, int64_t n, int64_t i, GradTable* t) {
  int64_t chunks = 0;
  t->count = 0;
  t->chunk0[0] = 0;
  for (; i < n && t->count < kBatch; ++i) {
    if (g[i].n == 0) continue;
    const int64_t c = (g[i].n + kChunk - 1) / kChunk;
    if (t->count > 0 && chunks + c >= (1ll << 31) - 1) break;
    const int k = t->count++;
    t->src[k] = g[i].src;
    t->dst[k] = g[i].dst;
    t->n[k] = g[i].n;
    t->bf16[k] = g[i].dtype == MOE_BF16;
    t->vec[k] = ((reinterpret_cast<uintptr_t>(g[i].src) | reinterpret_cast<uintptr_t>(g[i].dst)) &
                 15) == 0;
    chunks += c;
    t->chunk0[t->count] = static_cast<int>(chunks);
  }
  return i;
}

int grid_of(const GradTable& t, int sms) {
  return static_cast<int>(std::min<int64_t>(t.chunk0[t.count],
                                            std::min(kMaxBlocks, sms * kBlocksPerSm)));
}

size_t sums_bytes(int64_t n) {
  const int64_t launches = std::max<int64_t>(1, (n + kBatch - 1) / kBatch);
  return abi_align256(sizeof(Sums) * kMaxBlocks * static_cast<size_t>(launches));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_grad_clip_workspace_size(const moe_grad_t* grads, int64_t n) {
  if (!grads_ok(grads, n)) return 0;
  // the error word's place, the blocks' sums; a launch that ends early for its
  // chunks leaves the next one its tensors
  int64_t launches = 0;
  GradTable t;
  for (int64_t i = 0; i < n; ++launches) i = fill_table(grads, n, i, &t);
  return 256 + sums_bytes(std::max<int64_t>(1, launches) * kBatch);
}

moe_status moe_grad_clip(const moe_grad_t* grads, int64_t n, float max_norm, float* norm_out,
                         void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!grads_ok(grads, n) || !(max_norm >= 0.f) || !norm_out || !ws ||
      (reinterpret_cast<uintptr_t>(ws) & 255) || (reinterpret_cast<uintptr_t>(norm_out) & 3))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_grad_clip_workspace_size(grads, n)) return MOE_ERR_WORKSPACE;
  int sms = 0;
  const moe_status ds = abi_device_sms(&sms);
  if (ds != MOE_OK) return ds;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Sums* sums = reinterpret_cast<Sums*>(static_cast<char*>(ws) + 256);
  GradTable t;
  int blocks = 0;
  for (int64_t i = 0; i < n;) {
    i = fill_table(grads, n, i, &t);
    if (!t.count) continue;
    const int grid = grid_of(t, sms);
    const cudaError_t e = abi_tracked(kAbiGradNorm, 1, st, [&] {
      grad_norm_kernel<<<grid, kThreads, 0, st>>>(t, blocks, sums);
      return cudaGetLastError();
    });
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    blocks += grid;
  }
  bool scale = false;
  for (int64_t i = 0; i < n; ++i) scale = scale || (grads[i].n > 0 && grads[i].dst);
  // Where there is nothing to scale, one block for the norm (0 of no element).
  bool first = true;
  for (int64_t i = scale ? 0 : n; i < n || first;) {
    t.count = 0;
    t.chunk0[0] = 0;
    i = fill_table(grads, n, i, &t);
    if (scale && !t.count) continue;
    // (the first may start while the norm's last blocks end)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(std::max(1, grid_of(t, sms)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = first && blocks > 0 ? 1 : 0;
    float* out = first ? norm_out : nullptr;
    const cudaError_t e = abi_tracked(kAbiGradScale, 1, st, [&] {
      return cudaLaunchKernelEx(&cfg, grad_scale_kernel, t, static_cast<const Sums*>(sums), blocks, max_norm, out);
    });
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    first = false;
  }
  return MOE_OK;
}

}  // extern "C"
