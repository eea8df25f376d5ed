// MXFP4 codec (gfx950): bf16 <-> E2M1 codes with an E8M0 scale per 32
// elements of a row.
//   X from the block's amax by the rule, code = e2m1(x 2^-X)
// v_cvt_scalef32_pk_fp4_bf16 divides by the power of two and rounds once
// (nearest even, saturating at 6, sign kept; checked for every bf16 at scales
// over the whole range), and its inverse multiplies exactly.
#include "device.h"
#include "launch.h"

namespace fp8blk {

namespace {

// E8M0 code of a block from its bf16 amax bits.  With amax = (1 + m/128)
// 2^(E-127) and 6 = 1.5 * 2^2: floor is E - 2, ceil one more where m > 64
// (the mantissa of 1.5).  Both at least 0: X = -127, also for amax = 0.
// Subnormal amax: floor(log2 amax) - 2 and the smallest X are below -127.
template <bool FLOOR>
__device__ __forceinline__ uint32_t mx4_code(uint32_t amax) {
  const int c = (int)(amax >> 7) - 2 + (!FLOOR && (amax & 0x7F) > 0x40 ? 1 : 0);
  return (uint32_t)(c < 0 ? 0 : c);
}

constexpr int kThreads = 256;

// This thread among all of a launch, whose workgroups fill two dimensions.
__device__ __forceinline__ uint64_t thread_of_launch() {
  return ((uint64_t)blockIdx.y * gridDim.x + blockIdx.x) * kThreads + threadIdx.x;
}

// A lane takes 8 elements (16 bytes), four lanes a block.  Bound by memory:
// 131072 x 7168 with fake-quant values, 4.2 GB: 659 us, 6.5 TB/s; two or four
// times the elements a lane 760, codes stored through the caches 674.
template <bool FLOOR, bool DQ>
__global__ __launch_bounds__(kThreads) void mxfp4_quant_kernel(const u32x4* __restrict__ x, uint64_t chunks,
                                                              uint32_t* __restrict__ q, uint8_t* __restrict__ scale,
                                                              u32x4* __restrict__ xdq) {
  const uint64_t c = thread_of_launch();
  const u32x4 v = c < chunks ? __builtin_nontemporal_load(x + c) : (u32x4){0u, 0u, 0u, 0u};
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const uint32_t code = mx4_code<FLOOR>(group_max<4>(absmax_bits<4>(w)));
  const float s = e8m0_val(code);
  uint32_t o = 0;
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(v2bf, w[0]), s, 0);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(v2bf, w[1]), s, 1);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(v2bf, w[2]), s, 2);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(v2bf, w[3]), s, 3);
  if (c >= chunks) return;
  __builtin_nontemporal_store(o, q + c);
  if ((threadIdx.x & 3) == 0) scale[c >> 2] = (uint8_t)code;
  if constexpr (DQ) {
    const u32x4 d = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(o, s, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(o, s, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(o, s, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(o, s, 3))};
    __builtin_nontemporal_store(d, xdq + c);
  }
}

// E8M0 as fp32, 255 as NaN.
__device__ __forceinline__ float e8m0_or_nan(uint32_t code) {
  return code == 255 ? __uint_as_float(0x7FC00000u) : e8m0_val(code);
}

// Two times 8 elements a lane (114688 x 2048, 595 MB: 91 us, 6.5 TB/s; once
// 102, four times 96).
constexpr int kTimes = 2;

__global__ __launch_bounds__(kThreads) void mxfp4_dequant_kernel(const uint32_t* __restrict__ q, uint64_t chunks,
                                                                const uint8_t* __restrict__ scale,
                                                                u32x4* __restrict__ x) {
  const uint64_t first = (thread_of_launch() - threadIdx.x) * kTimes + threadIdx.x;
  uint32_t w[kTimes], c8[kTimes];
#pragma unroll
  for (int u = 0; u < kTimes; ++u) {
    const uint64_t at = first + u * kThreads, c = at < chunks ? at : chunks - 1;
    w[u] = __builtin_nontemporal_load(q + c);
    c8[u] = scale[c >> 2];
  }
#pragma unroll
  for (int u = 0; u < kTimes; ++u) {
    const uint64_t c = first + u * kThreads;
    if (c >= chunks) continue;
    const float s = e8m0_or_nan(c8[u]);
    const u32x4 d = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[u], s, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[u], s, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[u], s, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[u], s, 3))};
    __builtin_nontemporal_store(d, x + c);
  }
}

// Workgroups for `threads` (fewer than 2^32 threads may be in a dimension).
dim3 grid_of(uint64_t threads) {
  const uint64_t groups = (threads + kThreads - 1) / kThreads, wide = uint64_t(1) << 20;
  return groups <= wide ? dim3((unsigned)groups) : dim3((unsigned)wide, (unsigned)((groups + wide - 1) / wide));
}

}  // namespace

hipError_t launch_mxfp4_quant(const uint16_t* x, int64_t rows, int64_t cols, bool floor_rule, uint8_t* q,
                              uint8_t* scale, uint16_t* xdq, hipStream_t stream) {
  const uint64_t chunks = (uint64_t)rows * (uint64_t)(cols / 8);
  const dim3 grid = grid_of(chunks);
  const u32x4* xv = reinterpret_cast<const u32x4*>(x);
  uint32_t* qv = reinterpret_cast<uint32_t*>(q);
  u32x4* dv = reinterpret_cast<u32x4*>(xdq);
  if (floor_rule && xdq)
    hipLaunchKernelGGL((mxfp4_quant_kernel<true, true>), grid, dim3(kThreads), 0, stream, xv, chunks, qv, scale, dv);
  else if (floor_rule)
    hipLaunchKernelGGL((mxfp4_quant_kernel<true, false>), grid, dim3(kThreads), 0, stream, xv, chunks, qv, scale, dv);
  else if (xdq)
    hipLaunchKernelGGL((mxfp4_quant_kernel<false, true>), grid, dim3(kThreads), 0, stream, xv, chunks, qv, scale, dv);
  else
    hipLaunchKernelGGL((mxfp4_quant_kernel<false, false>), grid, dim3(kThreads), 0, stream, xv, chunks, qv, scale, dv);
  return hipGetLastError();
}

hipError_t launch_mxfp4_dequant(const uint8_t* q, const uint8_t* scale, int64_t rows, int64_t cols, uint16_t* x,
                                hipStream_t stream) {
  const uint64_t chunks = (uint64_t)rows * (uint64_t)(cols / 8);
  hipLaunchKernelGGL(mxfp4_dequant_kernel, grid_of((chunks + kTimes - 1) / kTimes), dim3(kThreads), 0, stream,
                     reinterpret_cast<const uint32_t*>(q), chunks, scale, reinterpret_cast<u32x4*>(x));
  return hipGetLastError();
}

}  // namespace fp8blk
