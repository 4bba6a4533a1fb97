// paged_search.cuh -- which sequence of a ragged batch a token belongs to.
#pragma once

#include <cstdint>

namespace fa {

// the last b with cu[b] <= t, by 32-way search over cu[0 .. B-1]; the whole
// warp asks for one t
__device__ __forceinline__ int find_sequence(const int* __restrict__ cu, int B, int t, int lane) {
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const uint32_t yes = __ballot_sync(0xffffffffu, i < n && cu[lo + i] <= t);
    const int last = yes == 0u ? 0 : 31 - __clz(yes);
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

}  // namespace fa
