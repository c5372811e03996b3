// Helpers that more than one translation unit of the C ABI shares: the
// shape check, the per-device capability cache and launch accounting
// (the launch counter and the optional event timer of moe.h).  Not part of
// the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

// moe_shape validity, as every entry point checks it.
bool abi_shape_ok(const moe_shape* s);

// SM count of the current device, or MOE_ERR_UNSUPPORTED if it is not an
// sm_103 part (cached per device).
moe_status abi_device_sms(int* sms);

// The limit of a kernel's wait for its own copies (moe_set_wait_timeout_ns).
uint64_t abi_wait_timeout_ns();

// A tensor map over bytes [d2, d1, d0], contiguous, d0 a multiple of 16; boxes of
// [1, b1, b0].  False if it cannot be made.
bool abi_map_bytes(CUtensorMap* m, const void* base, uint64_t d0, uint64_t d1, uint64_t d2,
                   uint32_t b0, uint32_t b1, CUtensorMapSwizzle sw);

// The plan kernels (launch_plan) and a memset, counted by
// moe_kernel_launch_count() and bracketed by the event timer when it is on.
cudaError_t abi_tracked_plan(const int* idx, int64_t Tk, int E, int* counts, int* offsets,
                             int* perm, int* inv, int* poff, int* blkhist, int* err,
                             cudaStream_t st);
cudaError_t abi_tracked_memset(void* p, int value, size_t bytes, cudaStream_t st);

// Kernel kinds of the operators outside api.cu, for the launch counter and the
// event timer (their names: api.cu).
enum AbiKind : int {
  kAbiNormFwd = 0, kAbiNormBwd, kAbiGradNorm, kAbiGradScale, kAbiMxQuantize, kAbiMxDequantize,
  kAbiFewGateUp, kAbiFewDown, kAbiFewRows, kNumAbiKinds
};

// Launch accounting around a launcher of `nkernels` kernels, as moe.h
// describes it (an event pair is recorded when the timer is on).
struct AbiTrack {
  int kind;
  cudaEvent_t a, b;
};
AbiTrack abi_track_begin(AbiKind kind, cudaStream_t st);
void abi_track_end(const AbiTrack& t, int nkernels, cudaStream_t st);

template <typename F>
cudaError_t abi_tracked(AbiKind kind, int nkernels, cudaStream_t st, F&& launch) {
  const AbiTrack t = abi_track_begin(kind, st);
  const cudaError_t e = launch();
  abi_track_end(t, nkernels, st);
  return e;
}

inline bool abi_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline size_t abi_align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

}  // namespace moe
