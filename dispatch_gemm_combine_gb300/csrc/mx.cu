// Expert weights in microscaled 4-bit: quantisation of w [E, K, N] in blocks of
// 32 along K (the contraction of x @ w), and the way back.
//
// The codes are laid out with K innermost, [E, N, K/2], as a product that
// streams them wants them, so both directions transpose.  A block of 256
// threads owns 64 columns by 256 rows: warp w the rows [32 w, 32 w + 32) of
// every column, lane l the columns 2 l and 2 l + 1.  A warp's access to w is 64
// neighbouring columns of one row (128 bytes in bf16), 32 of them in flight per
// lane; a lane then holds two whole blocks of 32, so the scale needs no
// exchange.  The codes pass through shared memory to reach global memory as
// 128-byte rows.  Both directions are HBM-bound: 2 + 17/32 bytes per bf16 weight.
#include "abi_internal.h"
#include "mx.cuh"
#include "vec.cuh"

namespace moe {
namespace {

constexpr int kTileN = 64;
constexpr int kTileK = 256;
constexpr int kRowPad = kTileK / 2 + 16;   // bytes between the columns' codes in shared memory

struct MxDims {
  int64_t K, N;
  int tiles_k, tiles_n;
};

__device__ __forceinline__ float2 load_pair(const __nv_bfloat16* p) {
  const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p));
  return make_float2(bf16_lo(w), bf16_hi(w));
}
__device__ __forceinline__ float2 load_pair(const float* p) {
  return __ldg(reinterpret_cast<const float2*>(p));
}
__device__ __forceinline__ void store_pair(__nv_bfloat16* p, float2 v) {
  *reinterpret_cast<uint32_t*>(p) = pack_bf16(v.x, v.y);
}
__device__ __forceinline__ void store_pair(float* p, float2 v) {
  *reinterpret_cast<float2*>(p) = v;
}

template <typename E>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const E* __restrict__ w, MxDims d,
                                                          uint8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  __shared__ alignas(16) uint8_t sc[kTileN * kRowPad];
  __shared__ uint8_t ss[kTileN][8];
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
  const int tn = blockIdx.x % d.tiles_n;
  const int64_t rest = blockIdx.x / d.tiles_n;
  const int tk = static_cast<int>(rest % d.tiles_k);
  const int64_t e = rest / d.tiles_k;
  const int64_t n0 = static_cast<int64_t>(tn) * kTileN, n = n0 + 2 * lane;
  const int64_t k0 = static_cast<int64_t>(tk) * kTileK, k = k0 + 32 * wp;
  if (k < d.K && n < d.N) {
    const E* p = w + (e * d.K + k) * d.N + n;
    float2 v[32];
    uint32_t ax = 0, ay = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = load_pair(p + i * d.N);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      ax = max(ax, __float_as_uint(v[i].x) & 0x7fffffffu);
      ay = max(ay, __float_as_uint(v[i].y) & 0x7fffffffu);
    }
    const uint32_t bx = mx_scale_byte(ax, 0x400000u, 2), by = mx_scale_byte(ay, 0x400000u, 2);
    const float ix = mx_inv_scale(bx), iy = mx_inv_scale(by);
    uint32_t cx[4], cy[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      cx[q] = 0, cy[q] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 a = v[8 * q + 2 * j], b = v[8 * q + 2 * j + 1];
        cx[q] |= e2m1_pair(a.x * ix, b.x * ix) << (8 * j);
        cy[q] |= e2m1_pair(a.y * iy, b.y * iy) << (8 * j);
      }
      if (bx == 255u) cx[q] = 0;
      if (by == 255u) cy[q] = 0;
    }
    *reinterpret_cast<uint4*>(sc + (2 * lane) * kRowPad + 16 * wp) = make_uint4(cx[0], cx[1], cx[2], cx[3]);
    *reinterpret_cast<uint4*>(sc + (2 * lane + 1) * kRowPad + 16 * wp) = make_uint4(cy[0], cy[1], cy[2], cy[3]);
    ss[2 * lane][wp] = static_cast<uint8_t>(bx);
    ss[2 * lane + 1][wp] = static_cast<uint8_t>(by);
  }
  __syncthreads();
#pragma unroll
  for (int i = threadIdx.x; i < kTileN * 8; i += 256) {
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
  __shared__ alignas(16) uint8_t sc[kTileN * kRowPad];
  __shared__ uint8_t ss[kTileN][8];
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
  const int tn = blockIdx.x % d.tiles_n;
  const int64_t rest = blockIdx.x / d.tiles_n;
  const int tk = static_cast<int>(rest % d.tiles_k);
  const int64_t e = rest / d.tiles_k;
  const int64_t n0 = static_cast<int64_t>(tn) * kTileN, n = n0 + 2 * lane;
  const int64_t k0 = static_cast<int64_t>(tk) * kTileK, k = k0 + 32 * wp;
#pragma unroll
  for (int i = threadIdx.x; i < kTileN * 8; i += 256) {
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
  const uint4 ux = *reinterpret_cast<const uint4*>(sc + (2 * lane) * kRowPad + 16 * wp);
  const uint4 uy = *reinterpret_cast<const uint4*>(sc + (2 * lane + 1) * kRowPad + 16 * wp);
  const float fx = mx_scale(ss[2 * lane][wp]), fy = mx_scale(ss[2 * lane + 1][wp]);
  const uint32_t cx[4] = {ux.x, ux.y, ux.z, ux.w}, cy[4] = {uy.x, uy.y, uy.z, uy.w};
  E* p = w + (e * d.K + k) * d.N + n;
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = e2m1_values((cx[q] >> (8 * j)) & 0xffu);
      const float2 b = e2m1_values((cy[q] >> (8 * j)) & 0xffu);
      const int i = 8 * q + 2 * j;
      store_pair(p + i * d.N, make_float2(a.x * fx, b.x * fy));
      store_pair(p + (i + 1) * d.N, make_float2(a.y * fx, b.y * fy));
    }
}

// The tiles of a launch, or 0 for dimensions that the calls refuse.
int64_t mx_tiles(int64_t E, int64_t K, int64_t N, MxDims* d) {
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
  const int64_t tiles = mx_tiles(E, K, N, &d);
  if ((tiles == 0 && E != 0) || (E == 0 && mx_tiles(1, K, N, &d) == 0) ||
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
  const int64_t tiles = mx_tiles(E, K, N, &d);
  if ((tiles == 0 && E != 0) || (E == 0 && mx_tiles(1, K, N, &d) == 0) ||
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
