// Residual addition, root-mean-square norm and FP8 quantization of the
// normed rows (gfx950), and the norm's backward pass.
//
//   h = RN_bf16(x + r);  rstd = 1 / sqrt(mean h^2 + eps);  y = h rstd w
//   1x128: s = RN32(amax|y| / 448), code = e4m3(RN32(y / s))
//   1x32 : X from amax|y| by the E8M0 rule, code = e4m3(y 2^-X)
// y stays in fp32 between the norm and the FP8 rounding (rounding it to bf16
// first would round twice); h is rounded to bf16 because it is the residual
// stream that the next layer and the backward pass read.
//
// One workgroup per row.  Thread t holds the 8-element chunks t, t + T, ...
// of the row in registers between the sum of squares and the encode, so the
// row is read once; a 1x128 tile is 16 adjacent lanes, a 1x32 block 4.  Bound
// by HBM for many rows: 16384 x 7168 with residual, h and y, 9 bytes per
// element, in 180 us (5.9 TB/s).  A few rows are bound by latency: 3.9 us.
#include "device.h"
#include "launch.h"

namespace fp8blk {

namespace {

// Sum over the workgroup (its waves' sums added in wave order, so the
// result does not depend on timing); red holds 16 floats, which are free
// again after the workgroup's next barrier.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_add(v);
  const int waves = (int)(blockDim.x >> 6);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < waves; ++i) s += red[i];
  return s;
}

__device__ __forceinline__ void unpack8(const u32x4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf_lo(w[i]);
    f[2 * i + 1] = bf_hi(w[i]);
  }
}

__device__ __forceinline__ u32x4 pack8(const float* f) {
  return (u32x4){pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
}

template <bool NT>
__device__ __forceinline__ u32x4 load(const u32x4* p) {
  if constexpr (NT)
    return __builtin_nontemporal_load(p);
  else
    return *p;
}
template <bool NT, typename T>
__device__ __forceinline__ void store(T v, T* p) {
  if constexpr (NT)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}

// Weights of chunk c as fp32.
template <bool WF32>
__device__ __forceinline__ void load_weight8(const void* w, int c, float* f) {
  if constexpr (WF32) {
    const v4f* p = reinterpret_cast<const v4f*>(w) + 2 * c;
    const v4f a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = a[i];
      f[4 + i] = b[i];
    }
  } else {
    unpack8(reinterpret_cast<const u32x4*>(w)[c], f);
  }
}

struct NormParams {
  const u32x4* x;
  const u32x4* res;
  const void* w;
  int nch;          // chunks per row
  float cols;
  float eps;
  u32x2* q;
  void* scale;
  u32x4* h;
  u32x4* y;
  u32x4* ydq;
  float* rstd;
  int64_t rows;
};

// E8M0 code of a block from its fp32 amax: as e8m0_code, on the fp32 bits.
// CEIL: X is the smallest integer with amax <= 1.75 * 2^(8 + X), so one is
// added where the mantissa is above 1.75 (0x600000).
template <bool FLOOR>
__device__ __forceinline__ uint32_t e8m0_code_f32(uint32_t bits) {
  int c = (int)(bits >> 23) - 8;
  if (!FLOOR) c += (bits & 0x7FFFFFu) > 0x600000u ? 1 : 0;
  c = c < 0 ? 0 : c;
  return (uint32_t)(c > 254 ? 254 : c);
}

// BLK 32 or 128; CH chunks per thread.
template <int BLK, bool FLOOR, bool WF32, int CH, bool NT>
__global__ __launch_bounds__(1024) void rmsnorm_quant_kernel(NormParams p) {
  __shared__ float red[2][2][16];         // of this row and the one before, the sum and the rescaled one
  const int T = (int)blockDim.x, t = (int)threadIdx.x;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
  const int64_t base = row * p.nch;
  float f[CH][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + i * T;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (c < p.nch) {
      v = load<NT>(p.x + base + c);
      if (p.res) {
        float a[8], b[8];
        unpack8(v, a);
        unpack8(load<NT>(p.res + base + c), b);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] += b[j];
        v = pack8(a);
        store<NT>(v, p.h + base + c);
      }
    }
    unpack8(v, f[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(f[i][j], f[i][j], ss);
  }
  ss = block_sum(ss, red[turn][0]);
  const float mean = ss / p.cols + p.eps;
  float rstd = 1.0f / sqrtf(mean);
  if (!(mean < __builtin_inff())) {
    // squares (or their mean and eps) left the fp32 range: the same with h
    // 2^-96 (uniform branch).  The largest row, 32768 elements below 2^128,
    // sums up to less than 2^79 so, and a sum of squares of 2^128 to 2^-64.
    // eps takes the factor 2^-192 in two steps.
    float s2 = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = f[i][j] * 0x1p-96f;
        s2 = __builtin_fmaf(d, d, s2);
      }
    s2 = block_sum(s2, red[turn][1]);
    rstd = 0x1p-96f / sqrtf(s2 / p.cols + p.eps * 0x1p-96f * 0x1p-96f);
  }
  if (p.rstd && t == 0) p.rstd[row] = rstd;

#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + i * T;
    const bool in = c < p.nch;
    float w[8];
    load_weight8<WF32>(p.w, in ? c : 0, w);
    float am = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f[i][j] = f[i][j] * rstd * w[j];
      am = __builtin_fmaxf(am, __builtin_fabsf(f[i][j]));
    }
    // chunks past the row are whole tiles past it: their lanes take part in
    // the lane reductions with zeros and store nothing
    const uint32_t bits = group_max<BLK / 8>(in ? __float_as_uint(am) : 0u);
    float v[8], sval;
    uint32_t code = 0;
    if constexpr (BLK == 128) {
      const float amax = __uint_as_float(bits);
      sval = amax / kE4M3Max;
      // tiny tiles are scaled by 2^64 so that the reciprocal stays finite
      const float pre = amax < 0x1p-60f ? 0x1p64f : 1.0f;
      const float sp = sval * pre;
      const float r = sval > 0.f ? 1.0f / sp : 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float yp = f[i][j] * pre;
        const float q0 = yp * r;
        const float rn = __builtin_fmaf(q0, sp, -yp);
        v[j] = clamp448(__builtin_fmaf(rn, -r, q0));
      }
    } else {
      code = e8m0_code_f32<FLOOR>(bits);
      sval = e8m0_val(code);
      // 2^-X in two factors: X reaches 120 for y near the fp32 maximum
      const int X = (int)code - 127;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = clamp448(__builtin_ldexpf(f[i][j], -X));
    }
    if (in) {
      u32x2 cc;
      cc.x = cvt4_e4m3(v[0], v[1], v[2], v[3]);
      cc.y = cvt4_e4m3(v[4], v[5], v[6], v[7]);
      store<NT>(cc, p.q + base + c);
      if (p.y) store<NT>(pack8(f[i]), p.y + base + c);
      if (p.ydq) {
        float d[8];
        decode4_e4m3(cc.x, d);
        decode4_e4m3(cc.y, d + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] *= sval;
        store<NT>(pack8(d), p.ydq + base + c);
      }
      if ((t & (BLK / 8 - 1)) == 0) {
        if constexpr (BLK == 128)
          reinterpret_cast<float*>(p.scale)[(base + c) / 16] = sval;
        else
          reinterpret_cast<uint8_t*>(p.scale)[(base + c) / 4] = (uint8_t)code;
      }
    }
  }
  }
}

struct NormBwdParams {
  const u32x4* dy;
  const u32x4* h;
  const void* w;
  const float* rstd;
  const u32x4* dres;
  int64_t rows;
  int nch;
  float cols;
  u32x4* dx;
  float* part;      // [grid][cols] partial weight gradients
};

// Workgroup b takes the rows b, b + G, ...; the weight gradient of its rows
// stays in registers and goes to the workspace once.  Bound by reading dy, h
// and dres and writing dx: 8192 x 7168 in 90 us with the partials' sum (5.2
// TB/s).  A few thousand small rows are bound by the two dependent launches and
// the partials' way through memory (2352 x 512: 8.7 us, 2 for its bytes).  Rows
// wider than 16384 are read twice (the second time from the L2): kept in
// registers they spill, 2048 x 32768 in 233 us instead of 161.  Two rows at a
// time, rows kept packed across the barrier and dres loaded before it all took
// registers that cost a workgroup per CU, and 10 to 60% more time.
template <bool WF32, int CH, bool NT>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_kernel(NormBwdParams p) {
  constexpr bool KEEP = CH < 4;           // a row's chunks fit the registers
  __shared__ float red[2][16];            // of this row and the one before
  const int T = (int)blockDim.x, t = (int)threadIdx.x;
  int turn = 0;
  float acc[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    const int64_t base = row * p.nch;
    const float rstd = p.rstd[row];
    float xh[KEEP ? CH : 1][8], wd[KEEP ? CH : 1][8];
    float dot = 0.f;
    // chunk i's xh into x and dy into d
    auto read = [&](int i, float* x, float* d) {
      const int c = t + i * T;
      u32x4 a = {0u, 0u, 0u, 0u}, b = {0u, 0u, 0u, 0u};
      if (c < p.nch) {
        a = load<NT && KEEP>(p.h + base + c);
        b = load<NT && KEEP>(p.dy + base + c);
      }
      unpack8(a, x);
      unpack8(b, d);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= rstd;
    };
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + i * T, at = KEEP ? i : 0;
      read(i, xh[at], wd[at]);
      float w[8];
      load_weight8<WF32>(p.w, c < p.nch ? c : 0, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc[i][j] = __builtin_fmaf(wd[at][j], xh[at][j], acc[i][j]);
        wd[at][j] *= w[j];
        dot = __builtin_fmaf(wd[at][j], xh[at][j], dot);
      }
      if constexpr (!KEEP) __builtin_amdgcn_sched_barrier(0);     // one chunk in registers at a time
    }
    const float c1 = block_sum(dot, red[turn]) / p.cols;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + i * T, at = KEEP ? i : 0;
      if (c >= p.nch) continue;
      if constexpr (!KEEP) {
        read(i, xh[at], wd[at]);
        float w[8];
        load_weight8<WF32>(p.w, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) wd[at][j] *= w[j];
      }
      float d[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = rstd * __builtin_fmaf(-xh[at][j], c1, wd[at][j]);
      if (p.dres) {
        float r[8];
        unpack8(load<NT>(p.dres + base + c), r);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] += r[j];
      }
      store<NT>(pack8(d), p.dx + base + c);
    }
  }
  v4f* out = reinterpret_cast<v4f*>(p.part) + (int64_t)blockIdx.x * p.nch * 2;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + i * T;
    if (c >= p.nch) continue;
    out[2 * c] = (v4f){acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
    out[2 * c + 1] = (v4f){acc[i][4], acc[i][5], acc[i][6], acc[i][7]};
  }
}

// Sum of the partial weight gradients: 32 columns per workgroup (128 bytes of
// a partial), 64 threads to four of them (thread q takes the partials q, q +
// 64, ...), added in LDS as a tree.
template <bool WF32>
__global__ __launch_bounds__(512) void rmsnorm_dw_kernel(const v4f* __restrict__ part, int parts, int cols,
                                                         void* __restrict__ dw) {
  __shared__ v4f red[64][9];
  const int lane = (int)(threadIdx.x & 7), q = (int)(threadIdx.x >> 3);
  const int c4 = (int)blockIdx.x * 8 + lane;
  v4f s = {0.f, 0.f, 0.f, 0.f};
  if (c4 * 4 < cols)
#pragma unroll 8
    for (int i = q; i < parts; i += 64) s += part[(int64_t)i * (cols / 4) + c4];
  red[q][lane] = s;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  s = red[q][lane];
#pragma unroll
  for (int i = 8; i < 64; i += 8) s += red[q + i][lane];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  red[q][lane] = s;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (threadIdx.x >= 8 || c4 * 4 >= cols) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) s += red[i][lane];
  if constexpr (WF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<float*>(dw)[c4 * 4 + i] = s[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<uint16_t*>(dw)[c4 * 4 + i] = (uint16_t)pack_bf16x2(s[i], 0.f);
  }
}

// Chunks per thread and threads for a row of nch chunks: two chunks where
// there are rows enough to fill the card (7168 columns forward, 16384 rows: 180
// us against 184 with one, 2048: 23 against 28, 768: 11.5 against 12.7, from
// 384 to 512 the same), one for a few rows (2048 columns, one row: 3.2 us
// against 3.7, 511: 4.6 against 5.2, 1024: the same).
void row_shape(int nch, int64_t rows, int* ch, int* threads) {
  *ch = nch <= 1024 && (rows < 512 || nch <= 128) ? 1 : nch <= 2048 ? 2 : 4;
  *threads = ((nch + *ch - 1) / *ch + 63) / 64 * 64;
}

// Workgroups of the backward pass: 16 waves per CU, four workgroups at most,
// and two where one has more than eight waves, so that one's loads run beside
// the other's barrier (8192 x 7168: 90 us, 106 with one, 108 with four; 8192 x
// 512: 14 us with four, 29 with one, 19 with two, 14 with sixteen).  A
// workgroup takes two rows and, past 256 workgroups, four, so that the partial
// sums stay a small part of the traffic (500 x 7168: 12.7 us, 15.6 with one
// row each; 2352 x 512: 8.7 us, 9.0 with one).
int64_t bwd_parts(int64_t rows, int threads, int ch) {
  const int waves = threads / 64, least = ch == 1 ? 2 : 1;
  int per_cu = 16 / waves > least ? 16 / waves : least;
  per_cu = per_cu < 4 ? per_cu : 4;
  const int64_t most = 256 * (int64_t)per_cu;
  const int64_t want = rows <= 64 ? rows : rows <= 128 ? 64 : rows <= 512 ? rows / 2 : rows <= 1024 ? 256 : rows / 4;
  return want < most ? want : most;
}

}  // namespace

int64_t rmsnorm_bwd_parts(int64_t rows, int64_t cols) {
  int ch, threads;
  row_shape((int)(cols / 8), 0, &ch, &threads);
  return bwd_parts(rows, threads > 0 ? threads : 64, ch);
}

hipError_t launch_rmsnorm_quant(const RmsNorm& a, hipStream_t stream) {
  const int nch = (int)(a.cols / 8);
  int ch, threads;
  row_shape(nch, a.rows, &ch, &threads);
  NormParams p{reinterpret_cast<const u32x4*>(a.x), reinterpret_cast<const u32x4*>(a.residual), a.weight, nch,
               (float)a.cols, a.eps, reinterpret_cast<u32x2*>(a.q), a.scale, reinterpret_cast<u32x4*>(a.h),
               reinterpret_cast<u32x4*>(a.y), reinterpret_cast<u32x4*>(a.ydq), a.rstd, a.rows};
  const dim3 grid((unsigned)(a.rows < kMaxGrid ? a.rows : kMaxGrid)), block((unsigned)threads);
  const int64_t bytes = (a.residual ? 6 : 2) + 1 + (a.y ? 2 : 0) + (a.ydq ? 2 : 0);       // per element
  const bool nt = a.rows * a.cols * bytes > kCached;
#define FP8BLK_NORM(B, F, W, C)                                                                      \
  do {                                                                                               \
    if (nt) hipLaunchKernelGGL((rmsnorm_quant_kernel<B, F, W, C, true>), grid, block, 0, stream, p); \
    else hipLaunchKernelGGL((rmsnorm_quant_kernel<B, F, W, C, false>), grid, block, 0, stream, p);   \
  } while (0)
#define FP8BLK_NORM_CH(B, F, W)                     \
  do {                                              \
    if (ch == 1) FP8BLK_NORM(B, F, W, 1);           \
    else if (ch == 2) FP8BLK_NORM(B, F, W, 2);      \
    else FP8BLK_NORM(B, F, W, 4);                   \
  } while (0)
#define FP8BLK_NORM_W(B, F)                         \
  do {                                              \
    if (a.weight_f32) FP8BLK_NORM_CH(B, F, true);   \
    else FP8BLK_NORM_CH(B, F, false);               \
  } while (0)
  if (a.blk == 128) FP8BLK_NORM_W(128, false);
  else if (a.floor_rule) FP8BLK_NORM_W(32, true);
  else FP8BLK_NORM_W(32, false);
#undef FP8BLK_NORM_W
#undef FP8BLK_NORM_CH
#undef FP8BLK_NORM
  return hipGetLastError();
}

hipError_t launch_rmsnorm_bwd(const uint16_t* dy, const uint16_t* h, const void* w, bool w_f32, const float* rstd,
                              const uint16_t* dres, int64_t rows, int64_t cols, void* workspace, uint16_t* dx,
                              void* dw, hipStream_t stream) {
  const int nch = (int)(cols / 8);
  const int parts = (int)rmsnorm_bwd_parts(rows, cols);
  v4f* part = reinterpret_cast<v4f*>(workspace);
  if (rows > 0) {
    int ch, threads;
    row_shape(nch, 0, &ch, &threads);
    NormBwdParams p{reinterpret_cast<const u32x4*>(dy), reinterpret_cast<const u32x4*>(h), w, rstd,
                    reinterpret_cast<const u32x4*>(dres), rows, nch, (float)cols, reinterpret_cast<u32x4*>(dx),
                    reinterpret_cast<float*>(part)};
    const dim3 grid((unsigned)parts), block((unsigned)threads);
    const bool nt = rows * cols * (dres ? 8 : 6) > kCached;
#define FP8BLK_NB(W, C)                                                                      \
  do {                                                                                       \
    if (nt) hipLaunchKernelGGL((rmsnorm_bwd_kernel<W, C, true>), grid, block, 0, stream, p); \
    else hipLaunchKernelGGL((rmsnorm_bwd_kernel<W, C, false>), grid, block, 0, stream, p);   \
  } while (0)
    if (w_f32) {
      if (ch == 1) FP8BLK_NB(true, 1);
      else if (ch == 2) FP8BLK_NB(true, 2);
      else FP8BLK_NB(true, 4);
    } else {
      if (ch == 1) FP8BLK_NB(false, 1);
      else if (ch == 2) FP8BLK_NB(false, 2);
      else FP8BLK_NB(false, 4);
    }
#undef FP8BLK_NB
  }
  const dim3 grid((unsigned)((cols + 31) / 32));
  if (w_f32)
    hipLaunchKernelGGL(rmsnorm_dw_kernel<true>, grid, dim3(512), 0, stream, part, parts, (int)cols, dw);
  else
    hipLaunchKernelGGL(rmsnorm_dw_kernel<false>, grid, dim3(512), 0, stream, part, parts, (int)cols, dw);
  return hipGetLastError();
}

}  // namespace fp8blk
