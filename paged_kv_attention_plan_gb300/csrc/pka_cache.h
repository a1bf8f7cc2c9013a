// Internal declarations of the operators around the paged cache: rotary
// positions (rope.cu) and the pages themselves (pages.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "pka.h"

namespace pka {

// Whether the enums, counts and scales of *p are in range (plan.cpp).
bool params_valid(const pka_params* p);

// Whether an int32 array starts where none can (null does not).
inline bool unaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) != 0; }

#ifdef __CUDACC__
// Note a violation that a kernel found (and stepped around) in the device
// error word: the largest code stays, whichever thread comes first.
__device__ __forceinline__ void note_error(int32_t* err, pka_status code) {
  if (err) atomicMax(err, static_cast<int32_t>(code));
}

// The last index r in [0, n) with ptr[r] <= x (ptr nondecreasing, n >= 1; 0
// when ptr[0] > x), found by a whole warp: each round compares 32 evenly
// spaced entries, so 1,024 requests take two dependent loads instead of ten.
__device__ __forceinline__ int warp_find(const int32_t* __restrict__ ptr, int n, int64_t x,
                                         int lane) {
  int lo = 0;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int64_t at = (int64_t)lane * step;
    const bool le = at < n && ptr[lo + at] <= x;
    const int below = max(__popc(__ballot_sync(0xffffffffu, le)) - 1, 0);
    lo += below * step;
    n = min(step, n - below * step);
  }
  return lo;
}
#endif

}  // namespace pka
