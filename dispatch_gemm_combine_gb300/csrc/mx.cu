// Expert weights in microscaled 4-bit: quantisation of w [E, K, N] in blocks of
// 32 along K (the contraction of x @ w), and the way back.
//
// The codes are laid out with K innermost, [E, N, K/2], as a product that
// streams them wants them, so both directions transpose.  A block of 256
// threads owns 32 C columns by 256 rows: warp w the rows [32 w, 32 w + 32) of
// every column, lane l the columns C l .. C l + C - 1 (8 bytes: C = 4 in bf16, 2 in
// fp32).  A warp's access to w is 256 bytes of one row, 32 of them in flight per
// lane; a lane then holds C whole blocks of 32, so the scale needs no
// exchange.  The codes pass through shared memory to reach global memory as
// 128-byte rows.  Both directions are HBM-bound: 2 + 17/32 bytes per bf16 weight.
// Measured: 16 x 2880 x 5760 bf16 there and back in 225 us, 6.0 TB/s.
#include "abi_internal.h"
#include "mx.cuh"
#include "vec.cuh"

namespace moe {
namespace {

constexpr int kTileK = 256;
constexpr int kRowPad = kTileK / 2 + 16;   // bytes between the columns' codes in shared memory

struct MxDims {
  int64_t K, N;
  int tiles_k, tiles_n;
};

// C neighbouring values of a row, 8 bytes.
template <typename E>
struct Cols {
  static constexpr int C = 8 / sizeof(E);
  static constexpr int kTileN = 32 * C;
  uint2 u;
  __device__ __forceinline__ void load(const E* p) { u = __ldg(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ float get(int c) const {
    if (sizeof(E) == 4) return __uint_as_float(c ? u.y : u.x);
    const uint32_t w = c >> 1 ? u.y : u.x;
    return c & 1 ? bf16_hi(w) : bf16_lo(w);
  }
};
__device__ __forceinline__ void store_cols(__nv_bfloat16* p, const float* v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}
__device__ __forceinline__ void store_cols(float* p, const float* v) {
  *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
}

template <typename E>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const E* __restrict__ w, MxDims d,
                                                          uint8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  constexpr int C = Cols<E>::C, TN = Cols<E>::kTileN;
  __shared__ alignas(16) uint8_t sc[TN * kRowPad];
  __shared__ uint8_t ss[TN][8];
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
  const int tn = blockIdx.x % d.tiles_n;
  const int64_t rest = blockIdx.x / d.tiles_n;
  const int tk = static_cast<int>(rest % d.tiles_k);
  const int64_t e = rest / d.tiles_k;
  const int64_t n0 = static_cast<int64_t>(tn) * TN, n = n0 + C * lane;
  const int64_t k0 = static_cast<int64_t>(tk) * kTileK, k = k0 + 32 * wp;
  if (k < d.K && n < d.N) {
    const E* p = w + (e * d.K + k) * d.N + n;
    Cols<E> v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i].load(p + i * d.N);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < 32; ++i) amax = max(amax, __float_as_uint(v[i].get(c)) & 0x7fffffffu);
      const uint32_t byte = mx_scale_byte(amax, 0x400000u, 2);
      const float inv = mx_inv_scale(byte);
      uint32_t q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        q[j] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          q[j] |= e2m1_pair(v[8 * j + 2 * i].get(c) * inv, v[8 * j + 2 * i + 1].get(c) * inv) << (8 * i);
        if (byte == 255u) q[j] = 0;
      }
      *reinterpret_cast<uint4*>(sc + (C * lane + c) * kRowPad + 16 * wp) = make_uint4(q[0], q[1], q[2], q[3]);
      ss[C * lane + c][wp] = static_cast<uint8_t>(byte);
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = threadIdx.x; i < TN * 8; i += 256) {
    const int c = i >> 3, b = i & 7;   // column, block of 32
    if (n0 + c < d.N && k0 + 32 * b < d.K) {
      const int64_t row = e * d.N + n0 + c;
      *reinterpret_cast<uint4*>(codes + row * (d.K / 2) + k0 / 2 + 16 * b) =
          *reinterpret_cast<const uint4*>(sc + c * kRowPad + 16 * b);
      scales[row * (d.K / 32) + k0 / 32 + b] = ss[c][b];
    }
  }
}

template <typename E>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales,
                                                            MxDims d, E* __restrict__ w) {
  constexpr int C = Cols<E>::C, TN = Cols<E>::kTileN;
  __shared__ alignas(16) uint8_t sc[TN * kRowPad];
  __shared__ uint8_t ss[TN][8];
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
  const int tn = blockIdx.x % d.tiles_n;
  const int64_t rest = blockIdx.x / d.tiles_n;
  const int tk = static_cast<int>(rest % d.tiles_k);
  const int64_t e = rest / d.tiles_k;
  const int64_t n0 = static_cast<int64_t>(tn) * TN, n = n0 + C * lane;
  const int64_t k0 = static_cast<int64_t>(tk) * kTileK, k = k0 + 32 * wp;
#pragma unroll
  for (int i = threadIdx.x; i < TN * 8; i += 256) {
    const int c = i >> 3, b = i & 7;
    if (n0 + c < d.N && k0 + 32 * b < d.K) {
      const int64_t row = e * d.N + n0 + c;
      *reinterpret_cast<uint4*>(sc + c * kRowPad + 16 * b) =
          __ldg(reinterpret_cast<const uint4*>(codes + row * (d.K / 2) + k0 / 2 + 16 * b));
      ss[c][b] = scales[row * (d.K / 32) + k0 / 32 + b];
    }
  }
  __syncthreads();
  if (k >= d.K || n >= d.N) return;
  float f[C];
#pragma unroll
  for (int c = 0; c < C; ++c) f[c] = mx_scale(ss[C * lane + c][wp]);
  E* p = w + (e * d.K + k) * d.N + n;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t q[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
      q[c] = *reinterpret_cast<const uint32_t*>(sc + (C * lane + c) * kRowPad + 16 * wp + 4 * j);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo[C], hi[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float2 a = e2m1_values((q[c] >> (8 * i)) & 0xffu);
        lo[c] = a.x * f[c], hi[c] = a.y * f[c];
      }
      store_cols(p + (8 * j + 2 * i) * d.N, lo);
      store_cols(p + (8 * j + 2 * i + 1) * d.N, hi);
    }
  }
}

// The tiles of a launch, or 0 for dimensions that the calls refuse.
int64_t mx_tiles(int64_t E, int64_t K, int64_t N, int32_t dtype, MxDims* d) {
  const int kTileN = dtype == MOE_FP32 ? Cols<float>::kTileN : Cols<__nv_bfloat16>::kTileN;
  if (E < 0 || K < 32 || N < 8 || K % 32 || N % 8 || K > (1ll << 31) || N > (1ll << 31)) return 0;
  d->K = K, d->N = N;
  d->tiles_k = static_cast<int>((K + kTileK - 1) / kTileK);
  d->tiles_n = static_cast<int>((N + kTileN - 1) / kTileN);
  const int64_t per = static_cast<int64_t>(d->tiles_k) * d->tiles_n;
  if (E > ((1ll << 31) - 1) / per) return 0;
  return E * per;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_mx_quantize(const void* w, int32_t dtype, int64_t E, int64_t K, int64_t N,
                           uint8_t* codes, uint8_t* scales, moe_stream_t stream) {
  MxDims d;
  const int64_t tiles = mx_tiles(E, K, N, dtype, &d);
  if ((tiles == 0 && E != 0) || (E == 0 && mx_tiles(1, K, N, dtype, &d) == 0) ||
      (dtype != MOE_BF16 && dtype != MOE_FP32))
    return MOE_ERR_INVALID_ARG;
  if (E == 0) return MOE_OK;
  if (!w || !codes || !scales || !abi_aligned16(w) || !abi_aligned16(codes))
    return MOE_ERR_INVALID_ARG;
  int sms = 0;
  const moe_status ds = abi_device_sms(&sms);
  if (ds != MOE_OK) return ds;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(tiles);
  const cudaError_t r = abi_tracked(kAbiMxQuantize, 1, st, [&] {
    if (dtype == MOE_FP32)
      mx_quantize_kernel<float><<<grid, 256, 0, st>>>(static_cast<const float*>(w), d, codes, scales);
    else
      mx_quantize_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(w), d, codes, scales);
    return cudaGetLastError();
  });
  return r == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t E, int64_t K,
                             int64_t N, int32_t dtype, void* w, moe_stream_t stream) {
  MxDims d;
  const int64_t tiles = mx_tiles(E, K, N, dtype, &d);
  if ((tiles == 0 && E != 0) || (E == 0 && mx_tiles(1, K, N, dtype, &d) == 0) ||
      (dtype != MOE_BF16 && dtype != MOE_FP32))
    return MOE_ERR_INVALID_ARG;
  if (E == 0) return MOE_OK;
  if (!w || !codes || !scales || !abi_aligned16(w) || !abi_aligned16(codes))
    return MOE_ERR_INVALID_ARG;
  int sms = 0;
  const moe_status ds = abi_device_sms(&sms);
  if (ds != MOE_OK) return ds;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(tiles);
  const cudaError_t r = abi_tracked(kAbiMxDequantize, 1, st, [&] {
    if (dtype == MOE_FP32)
      mx_dequantize_kernel<float><<<grid, 256, 0, st>>>(codes, scales, d, static_cast<float*>(w));
    else
      mx_dequantize_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(codes, scales, d, static_cast<__nv_bfloat16*>(w));
    return cudaGetLastError();
  });
  return r == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
