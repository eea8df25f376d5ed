// Gradients of the experts' products in bf16 (gfx950), grouped:
//   dgrad: dx[t][j] = sum_n dy[t][n] W[g][n][j]   (rows t of group g)
//   wgrad: dw[g][i][j] = sum_t dy[t][i] x[row(t)][j]
#include "groups.h"
#include "launch.h"

namespace fp8blk {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef unsigned short v8u16 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ void store_out(void* out, bool f32, int64_t at, float v) {
  if (f32)
    reinterpret_cast<float*>(out)[at] = v;
  else
    reinterpret_cast<uint16_t*>(out)[at] = (uint16_t)pack_bf16x2(v, 0.f);
}

// One wave per 16 x 16 outputs, operands straight from memory: lane l holds
// row l % 16 of either operand and 8 of the 32 summed places, at 8 (l / 16).
template <bool WGRAD>
__global__ __launch_bounds__(64) void grad_kernel(GroupedGrad a) {
  int g, r0, r1;
  if constexpr (WGRAD) {
    g = (int)blockIdx.z;
    rows_of_group(a.offsets, g, (int)a.total_m, &r0, &r1);
  } else {
    if (!row_tile(a.offsets, a.groups, (int)a.total_m, 16, (int)blockIdx.y, &g, &r0, &r1)) return;
  }
  const int lane = (int)threadIdx.x, r = lane & 15, kg = lane >> 4;
  const int64_t j0 = (int64_t)blockIdx.x * 16, i0 = WGRAD ? (int64_t)blockIdx.y * 16 : 0;
  const int64_t j = j0 + r < a.k ? j0 + r : a.k - 1;
  const int64_t sum = WGRAD ? r1 - r0 : a.n;
  v4f acc = {0.f, 0.f, 0.f, 0.f};
  for (int64_t s0 = 0; s0 < sum; s0 += 32) {
    v8u16 u = {0, 0, 0, 0, 0, 0, 0, 0}, v = u;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t s = s0 + 8 * kg + e;
      if (s >= sum) continue;
      if constexpr (WGRAD) {
        const int64_t t = a.row_index ? clamp_to(a.row_index[r0 + s], 0, (int)a.x_rows - 1) : r0 + s;
        u[e] = a.x[t * a.k + j];
        v[e] = a.dy[(r0 + s) * a.n + (i0 + r < a.n ? i0 + r : a.n - 1)];
      } else {
        u[e] = a.w[((int64_t)g * a.n + s) * a.k + j];
        v[e] = a.dy[(int64_t)(r0 + r < r1 ? r0 + r : r1 - 1) * a.n + s];
      }
    }
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, u), __builtin_bit_cast(v8bf, v), acc, 0, 0,
                                                  0);
  }
  const int64_t row = WGRAD ? i0 + r : r0 + r;
  if (row >= (WGRAD ? a.n : r1)) return;
#pragma unroll
  for (int v = 0; v < 4; ++v)
    if (j0 + 4 * kg + v < a.k)
      store_out(a.out, a.out_f32, ((WGRAD ? (int64_t)g * a.n : 0) + row) * a.k + j0 + 4 * kg + v, acc[v]);
}

}  // namespace

hipError_t launch_grouped_dgrad(const GroupedGrad& a, int num_cu, hipStream_t stream) {
  (void)num_cu;
  const dim3 grid((unsigned)((a.k + 15) / 16), (unsigned)((a.total_m + 15) / 16 + a.groups));
  hipLaunchKernelGGL((grad_kernel<false>), grid, dim3(64), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_grouped_wgrad(const GroupedGrad& a, int num_cu, hipStream_t stream) {
  (void)num_cu;
  const dim3 grid((unsigned)((a.k + 15) / 16), (unsigned)((a.n + 15) / 16), (unsigned)a.groups);
  hipLaunchKernelGGL((grad_kernel<true>), grid, dim3(64), 0, stream, a);
  return hipGetLastError();
}

}  // namespace fp8blk
