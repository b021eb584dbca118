// Shared by the paged-cache operators: argument checks, the even division of
// attention work over workers, and bounded waits.
#pragma once

#include <cuda.h>  // CUtensorMap types
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <string>
#include <utility>

#include "graph.h"
#include "mk.h"

namespace mk {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool page_size_ok(int p) { return p >= 16 && p <= 256 && (p & (p - 1)) == 0; }

// An error left by the caller's earlier work stays the caller's: reported,
// not cleared, and nothing is launched.
inline int pending_error(const char* who) {
  const cudaError_t e = cudaPeekAtLastError();
  if (e == cudaSuccess) return MK_OK;
  return fail(MK_ERR_CUDA, std::string(who) + ": an earlier CUDA error is pending: " + cudaGetErrorString(e));
}

// SMs of the current device.
inline int device_sms(const char* who, int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return fail(MK_ERR_CUDA, std::string(who) + ": no current device");
  return MK_OK;
}

// Let kernel `fn` use `bytes` of dynamic shared memory, once per device (`done`: that kernel's own record).
template <typename Fn>
cudaError_t allow_smem(Fn fn, int bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done->load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launch with programmatic dependent launch: the kernel's CTAs may start before the kernel ahead of it in the
// stream has ended, and wait for it themselves (wait_dependency) before they touch global memory.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

inline int launch_result(cudaError_t e, const char* who) {
  if (e == cudaSuccess) e = cudaGetLastError();
  else (void)cudaGetLastError();
  if (e == cudaSuccess) return MK_OK;
  return fail(MK_ERR_CUDA, std::string(who) + ": launch: " + cudaGetErrorString(e));
}

// First code wins; the caller clears the word.
__device__ __forceinline__ void set_status(int32_t* status, int code) {
  if (status) atomicCAS(status, MK_DEV_OK, code);
}

// Smallest b in [0, n) with off[b + 1] > i, for a non-decreasing off with
// off[0] <= i < off[n].
__device__ __forceinline__ int upper_row(const int32_t* off, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (off[mid + 1] > i) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

}  // namespace mk
