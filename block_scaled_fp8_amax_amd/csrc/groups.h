// Rows of routed experts, as the kernels of the MXFP4 experts find them.
// The offsets are not checked on the host: group g's rows are [lo, hi) with
// lo = off[g] and hi = off[g + 1] clamped into [0, total_m] and hi >= lo.
#pragma once

#include "device.h"

namespace fp8blk {

__device__ __forceinline__ int clamp_to(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

__device__ __forceinline__ void rows_of_group(const int32_t* offsets, int g, int total_m, int* lo, int* hi) {
  *lo = clamp_to(offsets[g], 0, total_m);
  *hi = clamp_to(offsets[g + 1], *lo, total_m);
}

// Row tile `tile` (of `per` rows) counted over all groups: its group, first
// row and last row; false where there are fewer.
__device__ __forceinline__ bool row_tile(const int32_t* offsets, int groups, int total_m, int per, int tile, int* g,
                                         int* first, int* last) {
  if (!offsets) {
    *g = 0;
    *first = tile * per;
    *last = total_m - *first < per ? total_m : *first + per;
    return *first < total_m;
  }
  for (int e = 0; e < groups; ++e) {
    int lo, hi;
    rows_of_group(offsets, e, total_m, &lo, &hi);
    const int tiles = (hi - lo + per - 1) / per;
    if (tile < tiles) {
      *g = e;
      *first = lo + tile * per;
      *last = hi - *first < per ? hi : *first + per;
      return true;
    }
    tile -= tiles;
  }
  return false;
}

}  // namespace fp8blk
