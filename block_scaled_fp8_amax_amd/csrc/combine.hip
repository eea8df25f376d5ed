// Weighted combination of the experts' rows (gfx950) and its gradients:
//   y[t] = residual[t] + sum_j w[t][j] R[slot[t][j]]     (fp32, j ascending)
//   dR[slot[t][j]] = w[t][j] dy[t],  dw[t][j] = <dy[t], R[slot[t][j]]>
// Bound by reading (and writing) top_k rows per token.  The rows of KB
// choices are loaded together, KB the power of two that top_k takes, eight at
// most: a load of nothing costs the address unit as much as any (635 tokens
// of one row of 7168, backward: 6.1 us, 14.2 with eight).
#include "device.h"
#include "launch.h"

namespace fp8blk {

namespace {

// Threads of a workgroup at most.  Forward, one chunk each: 16384 tokens of
// eight rows of 7168 take 412 us (5.7 TB/s) with 128; an earlier form of the
// kernel 470 with 128, 474 with 64, 493 with 192 and 500 to 520 with 256 to
// 896.  Backward, a whole token: 4093 such tokens take 201 us (4.95 TB/s)
// with 512, 200 with 256 and with 1024.
constexpr int kCbThreads = 128;
constexpr int kCbBwdThreads = 512;

typedef __amdgpu_buffer_rsrc_t Buffer;

// Row s of `rows` as a buffer; a slot that takes no part reads as zeros (a
// buffer of no length), without a branch between the loads of a batch.
template <bool F32>
__device__ __forceinline__ Buffer row_buffer(const void* rows, int64_t s, int64_t total_m, int64_t n) {
  const bool in = s >= 0 && s < total_m;
  const int64_t at = in ? s * n * (F32 ? 4 : 2) : 0;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(reinterpret_cast<const char*>(rows)) + at, 0,
                                           in ? (uint32_t)(n * (F32 ? 4 : 2)) : 0u, 0x00027000);
}

// Eight consecutive elements, chunk c of a row; bytes past the row are zeros
// and stores there are dropped.
template <bool F32, bool NT>
struct Chunk {
  static constexpr int kPolicy = NT ? 2 : 0;      // the nontemporal bit
  u32x4 v[F32 ? 2 : 1];
  __device__ __forceinline__ void load(Buffer b, int c) {
    v[0] = __builtin_amdgcn_raw_buffer_load_b128(b, (uint32_t)c * (F32 ? 32 : 16), 0, kPolicy);
    if constexpr (F32) v[1] = __builtin_amdgcn_raw_buffer_load_b128(b, (uint32_t)c * 32 + 16, 0, kPolicy);
  }
  __device__ __forceinline__ void store(Buffer b, int c) const {
    __builtin_amdgcn_raw_buffer_store_b128(v[0], b, (uint32_t)c * (F32 ? 32 : 16), 0, kPolicy);
    if constexpr (F32) __builtin_amdgcn_raw_buffer_store_b128(v[1], b, (uint32_t)c * 32 + 16, 0, kPolicy);
  }
  __device__ __forceinline__ void get(float* f) const {
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[i >> 2][i & 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf_lo(v[0][i]);
        f[2 * i + 1] = bf_hi(v[0][i]);
      }
    }
  }
  __device__ __forceinline__ void set(const float* f) {
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i >> 2][i & 3] = __float_as_uint(f[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[0][i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    }
  }
};

// A workgroup takes blockDim chunks of one token; `splits` workgroups make up
// a token.
template <bool ROW_F32, bool OUT_F32, int KB, bool NT>
__global__ __launch_bounds__(kCbThreads) void combine_kernel(CombineArgs a, int splits) {
  for (int64_t wg = blockIdx.x; wg < a.tokens * splits; wg += gridDim.x) {
    const int64_t t = wg / splits;
    const int c = (int)(wg - t * splits) * (int)blockDim.x + (int)threadIdx.x;
    const int32_t* slot = a.slot + t * a.top_k;
    const float* wt = a.weights + t * a.top_k;
    float acc[8];
    Chunk<false, NT> res;
    if (a.residual) {
      res.load(row_buffer<false>(a.residual, t, a.tokens, a.n), c);
      res.get(acc);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    }
    for (int j0 = 0; j0 < a.top_k; j0 += KB) {
      Chunk<ROW_F32, NT> r[KB];
      int64_t s[KB];
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        s[j] = j0 + j < a.top_k ? slot[j0 + j] : -1;
        r[j].load(row_buffer<ROW_F32>(a.rows, s[j], a.total_m, a.n), c);
      }
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        if (s[j] < 0 || s[j] >= a.total_m) continue;      // uniform: not even +0 is added
        const float w = wt[j0 + j];
        float f[8];
        r[j].get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(w, f[i], acc[i]);
      }
    }
    Chunk<OUT_F32, NT> y;
    y.set(acc);
    y.store(row_buffer<OUT_F32>(a.y, t, a.tokens, a.n), c);
  }
}

// One workgroup per token, KB choices at a time: dy is read once for all
// of them, and their dot products are summed over the workgroup together.
template <bool DY_F32, bool ROW_F32, int KB, bool NT>
__global__ __launch_bounds__(kCbBwdThreads) void combine_bwd_kernel(CombineBwdArgs a) {
  __shared__ float red[2][kCbBwdThreads / 64][KB];     // of this batch and the one before
  const int nch = (int)(a.n / 8), t = (int)threadIdx.x, threads = (int)blockDim.x;
  int turn = 0;
  for (int64_t tok = blockIdx.x; tok < a.tokens; tok += gridDim.x) {
    const Buffer dyb = row_buffer<DY_F32>(a.dy, tok, a.tokens, a.n);
    for (int j0 = 0; j0 < a.top_k; j0 += KB, turn ^= 1) {
      Buffer rb[KB], db[KB];
      float w[KB], dot[KB];
      int in = 0;                                      // bit j: choice j takes part
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        const int64_t s = j0 + j < a.top_k ? a.slot[tok * a.top_k + j0 + j] : -1;
        in |= (s >= 0 && s < a.total_m ? 1 : 0) << j;
        w[j] = s >= 0 && s < a.total_m ? a.weights[tok * a.top_k + j0 + j] : 0.f;
        rb[j] = row_buffer<ROW_F32>(a.rows, s, a.total_m, a.n);
        db[j] = row_buffer<ROW_F32>(a.drows, s, a.total_m, a.n);
        dot[j] = 0.f;
      }
      for (int c = t; c < nch; c += threads) {
        Chunk<DY_F32, NT> dy;
        Chunk<ROW_F32, NT> r[KB];
        dy.load(dyb, c);
#pragma unroll
        for (int j = 0; j < KB; ++j) r[j].load(rb[j], c);
        float d[8];
        dy.get(d);
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          float f[8], g[8];
          r[j].get(f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[j] = __builtin_fmaf(d[i], f[i], dot[j]);
            g[i] = w[j] * d[i];
          }
          Chunk<ROW_F32, NT> o;
          o.set(g);
          o.store(db[j], c);
        }
      }
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        dot[j] = wave_add(dot[j]);
        if ((t & 63) == 0) red[turn][t >> 6][j] = dot[j];
      }
      __syncthreads();
      if (t < KB && j0 + t < a.top_k) {
        float s = 0.f;
        for (int v = 0; v < threads / 64; ++v) s += red[turn][v][t];
        // a pair left out gets 0 whatever dy holds
        a.dweights[tok * a.top_k + j0 + t] = (in >> t) & 1 ? s : 0.f;
      }
    }
  }
}

// Whole waves for a row of n: at most `most` threads, evenly loaded.
int block_threads(int64_t n, int most) {
  const int64_t chunks = n / 8, turns = (chunks + most - 1) / most;
  const int64_t need = turns > 0 ? (chunks + turns - 1) / turns : 1;
  return (int)((need + 63) / 64 * 64);
}

template <int KB, bool NT>
void launch_combine_of(const CombineArgs& a, hipStream_t stream) {
  const int threads = a.n / 8 < kCbThreads ? block_threads(a.n, kCbThreads) : kCbThreads;
  const int splits = (int)((a.n / 8 + threads - 1) / threads);
  const int64_t wgs = a.tokens * splits;
  const dim3 grid((unsigned)(wgs < kMaxGrid ? wgs : kMaxGrid)), block((unsigned)threads);
  if (a.row_f32 && a.out_f32)
    hipLaunchKernelGGL((combine_kernel<true, true, KB, NT>), grid, block, 0, stream, a, splits);
  else if (a.row_f32)
    hipLaunchKernelGGL((combine_kernel<true, false, KB, NT>), grid, block, 0, stream, a, splits);
  else if (a.out_f32)
    hipLaunchKernelGGL((combine_kernel<false, true, KB, NT>), grid, block, 0, stream, a, splits);
  else
    hipLaunchKernelGGL((combine_kernel<false, false, KB, NT>), grid, block, 0, stream, a, splits);
}

template <int KB, bool NT>
void launch_combine_bwd_of(const CombineBwdArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)(a.tokens < kMaxGrid ? a.tokens : kMaxGrid));
  const dim3 block((unsigned)block_threads(a.n, kCbBwdThreads));
  if (a.dy_f32 && a.row_f32)
    hipLaunchKernelGGL((combine_bwd_kernel<true, true, KB, NT>), grid, block, 0, stream, a);
  else if (a.dy_f32)
    hipLaunchKernelGGL((combine_bwd_kernel<true, false, KB, NT>), grid, block, 0, stream, a);
  else if (a.row_f32)
    hipLaunchKernelGGL((combine_bwd_kernel<false, true, KB, NT>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((combine_bwd_kernel<false, false, KB, NT>), grid, block, 0, stream, a);
}

template <bool NT>
void launch_combine_nt(const CombineArgs& a, hipStream_t stream) {
  if (a.top_k == 1) launch_combine_of<1, NT>(a, stream);
  else if (a.top_k == 2) launch_combine_of<2, NT>(a, stream);
  else if (a.top_k <= 4) launch_combine_of<4, NT>(a, stream);
  else launch_combine_of<8, NT>(a, stream);
}

template <bool NT>
void launch_combine_bwd_nt(const CombineBwdArgs& a, hipStream_t stream) {
  if (a.top_k == 1) launch_combine_bwd_of<1, NT>(a, stream);
  else if (a.top_k == 2) launch_combine_bwd_of<2, NT>(a, stream);
  else if (a.top_k <= 4) launch_combine_bwd_of<4, NT>(a, stream);
  else launch_combine_bwd_of<8, NT>(a, stream);
}

}  // namespace

hipError_t launch_combine(const CombineArgs& a, hipStream_t stream) {
  const int64_t row = a.row_f32 ? 4 : 2, out = a.out_f32 ? 4 : 2, res = a.residual ? 2 : 0;
  if (a.tokens * (a.top_k * row + out + res) > kCached / a.n)
    launch_combine_nt<true>(a, stream);
  else
    launch_combine_nt<false>(a, stream);
  return hipGetLastError();
}

hipError_t launch_combine_bwd(const CombineBwdArgs& a, hipStream_t stream) {
  const int64_t row = a.row_f32 ? 4 : 2, dy = a.dy_f32 ? 4 : 2;
  if (a.n > 0 && a.tokens * (2 * a.top_k * row + dy) > kCached / a.n)
    launch_combine_bwd_nt<true>(a, stream);
  else
    launch_combine_bwd_nt<false>(a, stream);
  return hipGetLastError();
}

}  // namespace fp8blk
