// Products of a few bf16 rows with MXFP4 matrices (gfx950), dense and
// grouped over routed experts:
//   y[i][j] = sum_k x[i][k] e2m1(c[j][k]) 2^X[j][k / 32]
// An E2M1 value times a power of two is exact in bf16, and
// v_cvt_scalef32_pk_bf16_fp4 makes it in one instruction for two weights.
// Sums are fp32.
#include "groups.h"
#include "launch.h"

namespace fp8blk {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// Eight codes of a dword times the block's scale, as an MFMA operand.
__device__ __forceinline__ v8bf decode8(uint32_t c, float s) {
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2), e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3);
  return (v8bf){a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

__device__ __forceinline__ float scale_of(uint32_t code) {
  return code == 255 ? __uint_as_float(0x7FC00000u) : e8m0_val(code);
}

// One wave per 16 weight rows and 16 rows of x, operands straight from
// memory; a step of 128 k is four 16x16x32 MFMAs, lane l's block of 32 at
// 32 (l / 16) on both sides.
__global__ __launch_bounds__(64) void mx_rows_kernel(MxRows a) {
  int g, m0, m1;
  if (!row_tile(a.offsets, (int)a.groups, (int)a.total_m, 16, (int)blockIdx.y, &g, &m0, &m1)) return;
  const int lane = (int)threadIdx.x, r = lane & 15, kg = lane >> 4;
  const int64_t K = a.k, n0 = (int64_t)blockIdx.x * 16;
  int64_t m = m0 + r < m1 ? m0 + r : m1 - 1;
  if (a.row_index) m = clamp_to(a.row_index[m], 0, (int)a.x_rows - 1);
  const int64_t n = n0 + r < a.n ? n0 + r : a.n - 1;
  const uint16_t* x = a.x + m * K;
  const uint8_t* q = a.q + (g * a.n + n) * (K / 2);
  const uint8_t* s = a.scale + (g * a.n + n) * (K / 32);
  v4f acc = {0.f, 0.f, 0.f, 0.f};
  for (int64_t k0 = 0; k0 < K; k0 += 128) {
    const int64_t k = k0 + 32 * kg;
    const bool in = k < K;
    const u32x4 c = in ? *reinterpret_cast<const u32x4*>(q + k / 2) : (u32x4){0u, 0u, 0u, 0u};
    const float sc = in ? scale_of(s[k / 32]) : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x4 xv = in ? *reinterpret_cast<const u32x4*>(x + k + 8 * i) : (u32x4){0u, 0u, 0u, 0u};
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode8(c[i], sc), __builtin_bit_cast(v8bf, xv), acc, 0, 0, 0);
    }
  }
  if (m0 + r >= m1) return;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int64_t j = n0 + 4 * kg + v;
    if (j >= a.n) continue;
    if (a.out_f32)
      reinterpret_cast<float*>(a.y)[(int64_t)(m0 + r) * a.n + j] = acc[v];
    else
      reinterpret_cast<uint16_t*>(a.y)[(int64_t)(m0 + r) * a.n + j] = (uint16_t)pack_bf16x2(acc[v], 0.f);
  }
}

}  // namespace

hipError_t launch_mx_rows(const MxRows& a, hipStream_t stream) {
  const int64_t tiles = (a.total_m + 15) / 16 + (a.offsets ? a.groups : 0);
  const dim3 grid((unsigned)((a.n + 15) / 16), (unsigned)tiles);
  hipLaunchKernelGGL(mx_rows_kernel, grid, dim3(64), 0, stream, a);
  return hipGetLastError();
}

}  // namespace fp8blk
