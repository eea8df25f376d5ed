// Products of a few bf16 rows with NVFP4 weights (gfx950), dense and
// grouped over routed experts:
//   y[i][j] = g[j] * sum_k x[i][k] e2m1(c[j][k]) e4m3(S[j][k / 16])
// An e2m1 value has 2 significant bits and an e4m3 scale 4, so their
// product is exact (also in bf16); sums are fp32 and the tensor scale
// multiplies them once.  Bound by reading the weights: 0.5625 bytes each.
#include "device.h"
#include "launch.h"

namespace fp8blk {

namespace {

constexpr int kRowsPerPass = 8;      // x rows per read of a weight row

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// One wave per weight row; lane l takes the 1x16 blocks l, l + 64, ...
template <bool OUT_F32>
__global__ __launch_bounds__(256) void matvec_kernel(MatvecArgs a) {
  const int lane = (int)(threadIdx.x & 63);
  const int64_t j = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int grp = (int)blockIdx.y;
  if (j >= a.n) return;
  int lo = 0, hi = (int)a.total_m;
  if (a.offsets) {
    lo = clampi(a.offsets[grp], 0, (int)a.total_m);
    hi = clampi(a.offsets[grp + 1], lo, (int)a.total_m);
  }
  if (lo >= hi) return;
  const int64_t wrow = (int64_t)grp * a.n + j;
  const int nb = (int)(a.k / 16);
  const u32x2* q = reinterpret_cast<const u32x2*>(a.q) + wrow * nb;
  const uint8_t* bs = a.block_scale + wrow * nb;
  const float g = a.global_scale[wrow / a.rows_per_tensor];
  for (int m0 = lo; m0 < hi; m0 += kRowsPerPass) {
    const int mr = hi - m0 < kRowsPerPass ? hi - m0 : kRowsPerPass;
    const u32x4* xr[kRowsPerPass];
    float acc[kRowsPerPass];
#pragma unroll
    for (int i = 0; i < kRowsPerPass; ++i) {
      int r = m0 + (i < mr ? i : 0);
      if (a.row_index) r = clampi(a.row_index[r], 0, (int)a.x_rows - 1);
      xr[i] = reinterpret_cast<const u32x4*>(a.x + (int64_t)r * a.k);
      acc[i] = 0.f;
    }
    for (int b = lane; b < nb; b += 64) {
      const u32x2 c = q[b];
      const float s = __builtin_amdgcn_cvt_pk_f32_fp8((int)bs[b], false)[0];
      float w[16];
      const uint32_t cw[2] = {c.x, c.y};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const v2f d0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cw[h], 1.0f, 0);
        const v2f d1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cw[h], 1.0f, 1);
        const v2f d2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cw[h], 1.0f, 2);
        const v2f d3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cw[h], 1.0f, 3);
        const float d[8] = {d0[0], d0[1], d1[0], d1[1], d2[0], d2[1], d3[0], d3[1]};
#pragma unroll
        for (int e = 0; e < 8; ++e) w[8 * h + e] = d[e] * s;
      }
#pragma unroll
      for (int i = 0; i < kRowsPerPass; ++i) {
        if (i >= mr) break;
        const u32x4 v0 = xr[i][2 * b], v1 = xr[i][2 * b + 1];
        const uint32_t xw[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          acc[i] = __builtin_fmaf(bf_lo(xw[e]), w[2 * e], acc[i]);
          acc[i] = __builtin_fmaf(bf_hi(xw[e]), w[2 * e + 1], acc[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRowsPerPass; ++i) {
      float s = acc[i];
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d, 64);
      if (lane == 0 && i < mr) {
        const int64_t at = (int64_t)(m0 + i) * a.n + j;
        if constexpr (OUT_F32)
          reinterpret_cast<float*>(a.y)[at] = s * g;
        else
          reinterpret_cast<uint16_t*>(a.y)[at] = (uint16_t)pack_bf16x2(s * g, 0.f);
      }
    }
  }
}

}  // namespace

hipError_t launch_matvec(const MatvecArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.n + 3) / 4), (unsigned)a.groups);
  if (a.out_f32)
    hipLaunchKernelGGL(matvec_kernel<true>, grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL(matvec_kernel<false>, grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace fp8blk
