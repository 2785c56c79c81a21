// Device helpers over row offsets (cu arrays), shared by the attention and
// cache kernels.
#pragma once

#include "common.hpp"

namespace qg {

// The last row b in [0, rows) with key(b) <= x, for ascending key with
// key(0) <= x, searched by the whole wave: every lane probes one of 64 evenly
// spaced rows, so up to 64 rows take one round of loads and 4096 take two.
// Any key values give a result in [0, rows).
template <typename F>
__device__ __forceinline__ int find_row(int rows, int x, F&& key) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = rows;  // the answer is in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) >> 6;
    const int at = lo + lane * step;
    const uint64_t m = __ballot(at < hi && key(at) <= x);
    const int n = m ? 63 - __builtin_clzll(m) : 0;  // the last probe that holds
    lo += n * step;
    hi = lo + step < hi ? lo + step : hi;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

}  // namespace qg
