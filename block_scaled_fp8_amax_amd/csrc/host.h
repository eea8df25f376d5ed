// Host helpers shared by the entry points (abi.cpp, abi_moe.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8blk.h"

namespace fp8blk {

struct DeviceInfo {
  bool ok = false;
  bool supported = false;
  int num_cu = 0;
};

// Properties of the current device, read once per device.
int current_device(DeviceInfo** out);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// a * b <= lim for non-negative a, b, without overflowing int64.
inline bool product_at_most(int64_t a, int64_t b, int64_t lim) { return b == 0 || a <= lim / b; }

inline int hip_status(hipError_t e) { return e == hipSuccess ? FP8_OK : FP8_ERR_HIP; }

}  // namespace fp8blk
