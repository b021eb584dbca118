// Shared by the paged-cache operators: argument checks, the even division of
// attention work over workers, and bounded waits.
#pragma once

#include <cuda.h>  // CUtensorMap types
#include <cuda_runtime.h>

#include <cstdint>
#include <string>

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
