// Operands of v_mfma_scale_f32_16x16x128_f8f6f4, as the products of the MXFP4
// experts take them.
#pragma once

#include "device.h"

namespace fp8blk {

__device__ __forceinline__ v8i frag(u32x4 lo) { return (v8i){(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, 0, 0, 0, 0}; }
__device__ __forceinline__ v8i frag(u32x4 lo, u32x4 hi) {
  return (v8i){(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

__device__ __forceinline__ v8i frag(v8i f) { return f; }

// The codes with |a| >= 2 (bit 6 of a byte).
__device__ __forceinline__ v8i large_codes(v8i c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t m = ((uint32_t)c[i] >> 6) & 0x01010101u;
    c[i] &= (int)((m << 8) - m);
  }
  return c;
}

}  // namespace fp8blk
