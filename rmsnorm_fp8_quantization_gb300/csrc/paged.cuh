// What the kernels around the paged key/value cache share: the sticky
// bad-index flag, the search for a token's sequence, and divisions by sizes
// known to the host.
#pragma once

#include <cstdint>

#include "gbn_device.cuh"
#include "gbnorm.h"

namespace gbn {

// Sticky device-side error bits of one translation unit (read and cleared by
// gbn_device_error through read_paged_error below).
static __device__ unsigned int g_paged_error;

__device__ __forceinline__ void flag_bad_index() {
  if ((*reinterpret_cast<volatile unsigned int*>(&g_paged_error) & GBN_DEVICE_ERR_BAD_INDEX) == 0u)
    atomicOr(&g_paged_error, GBN_DEVICE_ERR_BAD_INDEX);
}
__device__ __forceinline__ void flag_wait_timeout() {
  atomicOr(&g_paged_error, GBN_DEVICE_ERR_COPY_TIMEOUT);
}

static inline cudaError_t read_paged_error(unsigned int* v, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(v, g_paged_error, sizeof(unsigned int));
  if (e != cudaSuccess || !clear || *v == 0u) return e;
  const unsigned int zero = 0u;
  return cudaMemcpyToSymbol(g_paged_error, &zero, sizeof(unsigned int));
}

// Number of entries of the sorted cu[1..n] that are <= t, found by one warp:
// each round every lane probes one of 32 evenly spaced entries, so 1024
// sequences take two dependent loads (a binary search would take ten).
// All lanes call it and get the same answer; reads stay within cu[1..n]
// whatever the values are.
__device__ __forceinline__ int warp_find_sequence(const int32_t* cu, int n, int64_t t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;  // the answer lies in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5;
    const int at = lo + (lane + 1) * step;  // probes cu[lo+step], cu[lo+2 step], ...
    const bool below = at <= hi && static_cast<int64_t>(cu[at]) <= t;
    const int c = __popc(__ballot_sync(0xFFFFFFFFu, below));
    lo += c * step;
    if (step == 1) break;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

}  // namespace gbn
