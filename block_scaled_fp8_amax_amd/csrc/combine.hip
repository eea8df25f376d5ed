// Weighted combination of the experts' rows (gfx950) and its gradients:
//   y[t] = residual[t] + sum_j w[t][j] R[slot[t][j]]     (fp32, j ascending)
//   dR[slot[t][j]] = w[t][j] dy[t],  dw[t][j] = <dy[t], R[slot[t][j]]>
// Bound by reading (and writing) top_k rows per token.
#include "device.h"
#include "launch.h"

namespace fp8blk {

namespace {

constexpr int kCbThreads = 256;

// Eight consecutive elements from chunk c of a bf16 or fp32 row.
template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t chunk, float* f) {
  if constexpr (F32) {
    const v4f a = reinterpret_cast<const v4f*>(p)[2 * chunk], b = reinterpret_cast<const v4f*>(p)[2 * chunk + 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = a[i];
      f[4 + i] = b[i];
    }
  } else {
    const u32x4 v = reinterpret_cast<const u32x4*>(p)[chunk];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf_lo(w[i]);
      f[2 * i + 1] = bf_hi(w[i]);
    }
  }
}

template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t chunk, const float* f) {
  if constexpr (F32) {
    reinterpret_cast<v4f*>(p)[2 * chunk] = (v4f){f[0], f[1], f[2], f[3]};
    reinterpret_cast<v4f*>(p)[2 * chunk + 1] = (v4f){f[4], f[5], f[6], f[7]};
  } else {
    reinterpret_cast<u32x4*>(p)[chunk] = (u32x4){pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                 pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
  }
}

// One workgroup per token.
template <bool ROW_F32, bool OUT_F32>
__global__ __launch_bounds__(kCbThreads) void combine_kernel(CombineArgs a) {
  const int nch = (int)(a.n / 8);
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
  const int32_t* slot = a.slot + t * a.top_k;
  const float* wt = a.weights + t * a.top_k;
  for (int c = (int)threadIdx.x; c < nch; c += kCbThreads) {
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    if (a.residual) load8<false>(a.residual, t * nch + c, acc);
    for (int j = 0; j < a.top_k; ++j) {
      const int64_t s = slot[j];
      if (s < 0 || s >= a.total_m) continue;
      const float w = wt[j];
      float r[8];
      load8<ROW_F32>(a.rows, s * nch + c, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(w, r[i], acc[i]);
    }
    store8<OUT_F32>(a.y, t * nch + c, acc);
  }
  }
}

// One workgroup per token; the choices in turn.
template <bool DY_F32, bool ROW_F32>
__global__ __launch_bounds__(kCbThreads) void combine_bwd_kernel(CombineBwdArgs a) {
  __shared__ float red[kCbThreads / 64];
  const int nch = (int)(a.n / 8);
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x)
  for (int j = 0; j < a.top_k; ++j) {
    const int64_t s = a.slot[t * a.top_k + j];
    float dot = 0.f;
    if (s >= 0 && s < a.total_m) {
      const float w = a.weights[t * a.top_k + j];
      for (int c = (int)threadIdx.x; c < nch; c += kCbThreads) {
        float d[8], r[8];
        load8<DY_F32>(a.dy, t * nch + c, d);
        load8<ROW_F32>(a.rows, s * nch + c, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dot = __builtin_fmaf(d[i], r[i], dot);
          d[i] *= w;
        }
        store8<ROW_F32>(a.drows, s * nch + c, d);
      }
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) dot += __shfl_xor(dot, d, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = dot;
    __syncthreads();
    if (threadIdx.x == 0) a.dweights[t * a.top_k + j] = (red[0] + red[1]) + (red[2] + red[3]);
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_combine(const CombineArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)(a.tokens < kMaxGrid ? a.tokens : kMaxGrid));
  if (a.row_f32 && a.out_f32)
    hipLaunchKernelGGL((combine_kernel<true, true>), grid, dim3(kCbThreads), 0, stream, a);
  else if (a.row_f32)
    hipLaunchKernelGGL((combine_kernel<true, false>), grid, dim3(kCbThreads), 0, stream, a);
  else if (a.out_f32)
    hipLaunchKernelGGL((combine_kernel<false, true>), grid, dim3(kCbThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((combine_kernel<false, false>), grid, dim3(kCbThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_combine_bwd(const CombineBwdArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)(a.tokens < kMaxGrid ? a.tokens : kMaxGrid));
  if (a.dy_f32 && a.row_f32)
    hipLaunchKernelGGL((combine_bwd_kernel<true, true>), grid, dim3(kCbThreads), 0, stream, a);
  else if (a.dy_f32)
    hipLaunchKernelGGL((combine_bwd_kernel<true, false>), grid, dim3(kCbThreads), 0, stream, a);
  else if (a.row_f32)
    hipLaunchKernelGGL((combine_bwd_kernel<false, true>), grid, dim3(kCbThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((combine_bwd_kernel<false, false>), grid, dim3(kCbThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace fp8blk
