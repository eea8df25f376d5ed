// What the kernels of the experts' gradients share: operands in LDS whose summed
// places lie apart, as in memory, and their reads.
#pragma once

#include <type_traits>

#include "groups.h"

namespace fp8blk {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// f(0), ..., f(N - 1) with compile-time arguments.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    each<N, I + 1>(f);
  }
}

constexpr int kPlaces = 64;   // of a stage

// Whether `tiles`, one to a CU and turn, keep three quarters of the CUs busy.
inline bool fills_turns(int64_t tiles, int num_cu) {
  const int64_t turns = (tiles + num_cu - 1) / num_cu;
  return 4 * tiles >= 3 * turns * num_cu;
}

// 16-byte pieces of a row of 128 bytes lie at piece ^ turn(row), 32-byte pieces
// of a place at piece ^ spread(place).
__device__ __forceinline__ int turn(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int spread(int place) { return (place & 3) | ((place >> 1) & 4); }

// 4 places by 16 columns of 16 lanes, turned: lane i of the 16 gives the
// address of 4 columns 4 (i % 4) of place i / 4 and gets the 4 places of
// column i.
__device__ __forceinline__ u32x2 read_turned(uint32_t lds) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) v4s lds_v4s;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(uintptr_t)lds));
}

}  // namespace fp8blk
