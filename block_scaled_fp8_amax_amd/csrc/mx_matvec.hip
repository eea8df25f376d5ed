// Products of a few rows with MXFP4 matrices (gfx950), dense and grouped over
// routed experts: bf16 rows (the matvec calls), and MXFP8 or MXFP4 rows where
// the tiles of mx_gemm.hip would leave most of the GPU idle.
//   y[i][j] = sum_k x[i][k] e2m1(c[j][k]) 2^X[j][k / 32]
// Bound by reading the weights, 0.53 bytes each.
//
// A workgroup of KS waves makes 16 R columns of up to MX rows.  Wave w takes
// the stages w, w + KS, ... of 256 elements of K, all by itself: its loads go
// straight to its own ring of SLOTS stages in LDS (weights, rows and scales),
// its waits are its own, and the waves' sums are added in LDS at the end, in
// wave order.  With K cut KS ways most of a wave's share is on its way at
// once.
//
// bf16 rows take v_mfma_f32_16x16x32_bf16, one for 8 elements of each of four
// blocks: an E2M1 value times a power of two is exact in bf16, and
// v_cvt_scalef32_pk_bf16_fp4 makes two of them.  Quantized rows take the
// scaled product of mx_gemm.hip, where the cut of E4M3 sums is explained; it is
// kept here, so that it does not go by a call's size (two products: 13 rows of
// 4096 x 7168 as long, 64 rows 12.6 us, 10.7 with one).
// As there, lane l takes blocks 2 (l / 16) and 2 (l / 16) + 1 of a stage.
#include "groups.h"
#include "launch.h"
#include "mx.h"

namespace fp8blk {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// Eight codes of a dword times the block's scale, as an operand.
__device__ __forceinline__ v8bf decode8(uint32_t c, float s) {
  const u32x4 w = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3))};
  return __builtin_bit_cast(v8bf, w);
}

__device__ __forceinline__ float scale_of(uint32_t code) {
  return code == 255 ? __uint_as_float(0x7FC00000u) : e8m0_val(code);
}

enum { kBf16 = 0, kE4m3 = 1, kE4m3Split = 2, kE2m1 = 3 };

struct Rows {
  const uint8_t* x;
  const uint8_t* x_scale;     // quantized rows
  int64_t x_rows;
  const int32_t* row_index;   // null = the row itself
  const uint8_t* q;
  const uint8_t* scale;
  const int32_t* offsets;     // null = slices of all rows
  int groups;
  int64_t total_m, n, k, slice;
  void* y;
  bool out_f32;
};

template <int X, int R, int MX, int KS, int SLOTS>
struct Plan {
  static constexpr int kXRow = X == kBf16 ? 512 : X == kE2m1 ? 128 : 256;    // bytes of a row and stage
  static constexpr int kXLoads = (MX * kXRow + 1023) / 1024;
  static constexpr int kTiles = (MX + 15) / 16;                              // of 16 rows
  static constexpr int kW = R * 2048, kX = kXLoads * 1024;
  static constexpr int kWScale = R * 256, kXScale = X == kBf16 ? 0 : kTiles * 256;
  static constexpr int kStage = kW + kX + kWScale + kXScale;
  static constexpr int kLoads = 3 * R + kXLoads + (X == kBf16 ? 0 : kTiles);
  static constexpr int kSums = R * kTiles * 1024;                            // of a wave
  static constexpr int kWave = SLOTS * kStage > kSums ? SLOTS * kStage : kSums;
  static_assert((SLOTS - 1) * kLoads <= 63, "loads that vmcnt counts");
};

// Rows [lo, hi) of y by the 16 R columns from n0 of matrix grp, MX rows at a
// time; WAVE: bytes of LDS of each wave.
template <int X, int R, int MX, int KS, int SLOTS, int WAVE>
__device__ __forceinline__ void multiply_rows(const Rows& a, int grp, int lo, int hi, int64_t n0, uint8_t* smem) {
  using P = Plan<X, R, MX, KS, SLOTS>;
  constexpr int T = P::kTiles;
  static_assert(P::kWave <= WAVE, "LDS");
  const int t = (int)threadIdx.x, lane = t & 63, r16 = lane & 15, kg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const uint32_t K = (uint32_t)a.k;
  const int stages = (int)((K + 255) / 256), blocks = (int)(K / 32);
  const int cols = a.n - n0 < 16 * R ? (int)(a.n - n0) : 16 * R;
  const uint32_t q_row = K / 2, s_row = K / 32, x_row = X == kBf16 ? K * 2 : X == kE2m1 ? K / 2 : K;
  constexpr uint32_t kNowhere = 0xFFFFFFF0u;

  // weights: rows past the matrix's end lie past the buffer's, and are zeros
  const int64_t first = (int64_t)grp * a.n + n0;
  const u32x4 qb = buffer_of(a.q + first * q_row, (uint32_t)cols * q_row);
  // scales are read a dword at a time, 16 bytes of a row from the dword that
  // holds the stage's first
  const uint8_t* sc = a.scale + first * s_row;
  const uint32_t mis = (uint32_t)(reinterpret_cast<uintptr_t>(sc) & 3);
  const u32x4 sb = buffer_of(sc - mis, ((uint32_t)cols * s_row + mis + 3u) & ~3u);
  const u32x4 xb = buffer_of(a.x, (uint32_t)(a.x_rows * x_row));
  // (quantized rows: K is a multiple of 128 and x_scale 4-byte aligned, so each
  // row's scales begin a dword)
  const u32x4 xsb = buffer_of(a.x_scale, X == kBf16 ? 0u : (uint32_t)(a.x_rows * s_row));

  const uint32_t ring = lds_address(smem) + (uint32_t)(wave * WAVE);
  const uint8_t* mine = smem + wave * WAVE;
  // this lane's pieces of the loads
  const int wrow = lane / 8, wpiece = (lane % 8) ^ ((wrow >> 1) & 3);   // row 8 more turns the piece by 4
  constexpr int kXPer = P::kXRow / 16;
  const int srow = lane / 4;

  // unsigned: hi can lie within MX of 2^31
  for (uint32_t next = (uint32_t)lo; next < (uint32_t)hi; next += MX) {
    const int m0 = (int)next, mr = hi - m0 < MX ? hi - m0 : MX;
    auto row_of = [&](int m) -> uint32_t {
      m = m0 + (m < mr ? m : mr - 1);
      return (uint32_t)(a.row_index ? clamp_to(a.row_index[m], 0, (int)a.x_rows - 1) : m);
    };
    uint32_t xoff[P::kXLoads], xsoff[T];
    int xk[P::kXLoads];                // first element of the lane's piece in a stage
#pragma unroll
    for (int i = 0; i < P::kXLoads; ++i) {
      const int m = i * (1024 / P::kXRow) + lane / kXPer;
      const int piece = (lane % kXPer) ^ (kXPer >= 16 ? m & 15 : (m >> 1) & 7);
      xk[i] = piece * (256 / kXPer);
      xoff[i] = m < mr ? row_of(m) * x_row + (uint32_t)(piece * 16) : kNowhere;
    }
#pragma unroll
    for (int c = 0; c < T; ++c) xsoff[c] = X == kBf16 ? 0u : row_of(c * 16 + srow) * s_row;

    auto load = [&](int s, int slot) {
      const uint32_t at = ring + (uint32_t)(slot * P::kStage);
      const uint32_t k0 = (uint32_t)s * 256;
#pragma unroll
      for (int i = 0; i < 2 * R; ++i) {
        const int piece = wpiece ^ (i & 1 ? 4 : 0);
        const uint32_t off = (uint32_t)(i * 8 + wrow) * q_row + k0 / 2 + (uint32_t)(piece * 16);
        lds_load16(qb, k0 + (uint32_t)(piece * 32) < K ? off : kNowhere, at + (uint32_t)(i * 1024));
      }
#pragma unroll
      for (int i = 0; i < P::kXLoads; ++i) {
        const uint32_t off = xoff[i] + (X == kBf16 ? k0 * 2 : X == kE2m1 ? k0 / 2 : k0);
        lds_load16(xb, xoff[i] != kNowhere && k0 + (uint32_t)xk[i] < K ? off : kNowhere,
                   at + (uint32_t)(P::kW + i * 1024));
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const uint32_t off = (((uint32_t)(i * 16 + srow) * s_row + mis) & ~3u) + k0 / 32 + (uint32_t)(lane & 3) * 4;
        lds_load4(sb, off, at + (uint32_t)(P::kW + P::kX + i * 256));
      }
      if constexpr (X != kBf16) {
#pragma unroll
        for (int c = 0; c < T; ++c)
          lds_load4(xsb, xsoff[c] + k0 / 32 + (uint32_t)(lane & 3) * 4, at + (uint32_t)(P::kW + P::kX + P::kWScale + c * 256));
      }
    };

    v4f acc[R][T];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < T; ++c) acc[r][c] = (v4f){0.f, 0.f, 0.f, 0.f};

    const int mine_stages = stages > wave ? (stages - wave + KS - 1) / KS : 0;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
      if (i < mine_stages) load(wave + i * KS, i);
    int slot = 0;
    for (int i = 0; i < mine_stages; ++i) {
      if (i + SLOTS <= mine_stages)
        wait_loads<(SLOTS - 1) * P::kLoads>();
      else if (SLOTS > 2 && i + 2 <= mine_stages)
        wait_loads<P::kLoads>();
      else
        wait_loads<0>();
      const int s = wave + i * KS;
      const uint8_t* at = mine + slot * P::kStage;
      // operands of the whole stage into registers
      u32x4 w[R][2], x[T][X == kBf16 ? 8 : X == kE2m1 ? 2 : 4];
      uint32_t ws[R][2], xs[T][2];
      const int b0 = 8 * s + 2 * kg;       // this lane's blocks: b0, b0 + 1
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t m = ((uint32_t)(r * 16 + r16) * s_row + mis) & 3u;
        const uint8_t* sp = at + P::kW + P::kX + r * 256 + r16 * 16 + m + 2 * kg;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          w[r][j] = *reinterpret_cast<const u32x4*>(at + r * 2048 + r16 * 128 + (((2 * kg + j) ^ (r16 >> 1)) & 7) * 16);
          // past K: the codes are zeros, the byte is another row's
          ws[r][j] = b0 + j < blocks ? sp[j] : 127u;
        }
      }
#pragma unroll
      for (int c = 0; c < T; ++c) {
        const int m = c * 16 + r16;
        const uint8_t* xp = at + P::kW + m % MX * P::kXRow;       // (rows past MX are not stored: any row will do)
        const int turned = kXPer >= 16 ? (m % MX) & 15 : ((m % MX) >> 1) & 7;
        if constexpr (X == kBf16) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[c][e] = *reinterpret_cast<const u32x4*>(xp + ((8 * kg + e) ^ turned) * 16);
        } else if constexpr (X == kE2m1) {
#pragma unroll
          for (int j = 0; j < 2; ++j) x[c][j] = *reinterpret_cast<const u32x4*>(xp + ((2 * kg + j) ^ turned) * 16);
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int piece = 4 * (kg >> 1) + 2 * j + (kg & 1);
            x[c][2 * j] = *reinterpret_cast<const u32x4*>(xp + (piece ^ turned) * 16);
            x[c][2 * j + 1] = *reinterpret_cast<const u32x4*>(xp + ((piece + 8) ^ turned) * 16);
          }
        }
        if constexpr (X != kBf16) {
          const uint8_t* sp = at + P::kW + P::kX + P::kWScale + c * 256 + r16 * 16 + 2 * kg;
#pragma unroll
          for (int j = 0; j < 2; ++j) xs[c][j] = b0 + j < blocks ? sp[j] : 127u;
        }
      }
      wait_lds_reads();
      if (i + SLOTS < mine_stages) load(s + SLOTS * KS, slot);
      slot = slot + 1 == SLOTS ? 0 : slot + 1;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if constexpr (X == kBf16) {
            const float f = scale_of(ws[r][j]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const v8bf d = decode8(w[r][j][e], f);
#pragma unroll
              for (int c = 0; c < T; ++c)
                acc[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(d, __builtin_bit_cast(v8bf, x[c][4 * j + e]), acc[r][c],
                                                                    0, 0, 0);
            }
          } else {
#pragma unroll
            for (int c = 0; c < T; ++c) {
              if constexpr (X == kE2m1) {
                acc[r][c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(w[r][j]), frag(x[c][j]), acc[r][c],
                                                                             4, 4, 0, (int)ws[r][j], 0, (int)xs[c][j]);
              } else {
                v8i up = frag(x[c][2 * j], x[c][2 * j + 1]), low = up;
                if constexpr (X == kE4m3Split) {
                  up = large_codes(up);
                  low = low ^ up;
                }
                acc[r][c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(w[r][j]), up, acc[r][c], 4, 0, 0,
                                                                             (int)ws[r][j], 0, (int)xs[c][j]);
                if constexpr (X == kE4m3Split)
                  acc[r][c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(w[r][j]), low, acc[r][c], 4, 0, 0,
                                                                               (int)ws[r][j], 0, (int)xs[c][j]);
              }
            }
          }
        }
    }

    // lane l holds columns 4 (l / 16) .. + 3 of row l % 16 of each tile
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < T; ++c)
        *reinterpret_cast<v4f*>(red + ((wave * T + c) * R + r) * 256 + lane * 4) = acc[r][c];
    __syncthreads();
    for (int e = t; e < 16 * R * mr; e += 64 * KS) {
      const int m = e / (16 * R), j = e % (16 * R);
      if (j < cols) {
        const int at = (m >> 4) * (R * 256) + (j >> 4) * 256 + (((j >> 2) & 3) * 16 + (m & 15)) * 4 + (j & 3);
        float v = red[at];
#pragma unroll
        for (int w = 1; w < KS; ++w) v += red[w * (T * R * 256) + at];
        const int64_t to = (int64_t)(m0 + m) * a.n + n0 + j;
        if (a.out_f32)
          reinterpret_cast<float*>(a.y)[to] = v;
        else
          reinterpret_cast<uint16_t*>(a.y)[to] = (uint16_t)pack_bf16x2(v, 0.f);
      }
    }
    __syncthreads();
  }
}

// All rows of one matrix, in slices of `slice` of them.
template <int X, int R, int MX, int KS, int SLOTS>
__global__ __launch_bounds__(64 * KS) void mx_rows_kernel(Rows a) {
  constexpr int kWave = Plan<X, R, MX, KS, SLOTS>::kWave;
  static_assert(KS * kWave <= 160 * 1024, "LDS");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[KS * kWave];
  const int64_t lo = blockIdx.y * a.slice, hi = lo + a.slice < a.total_m ? lo + a.slice : a.total_m;
  multiply_rows<X, R, MX, KS, SLOTS, kWave>(a, 0, (int)lo, (int)hi, (int64_t)blockIdx.x * (16 * R), smem);
}

// The rows of the blockIdx.y-th group that has any: groups of up to four rows,
// most of them in decoding, with three stages on their way, others 16 rows at
// a time with two.
template <int X, int KS>
__global__ __launch_bounds__(64 * KS) void mx_groups_kernel(Rows a) {
  constexpr int R = 2, kFew = Plan<X, R, 4, KS, 3>::kWave, kMany = Plan<X, R, 16, KS, 2>::kWave;
  constexpr int kWave = kFew > kMany ? kFew : kMany;
  static_assert(KS * kWave <= 160 * 1024, "LDS");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[KS * kWave];
  int grp, lo, hi;
  if (!nth_group(a.offsets, a.groups, (int)a.total_m, (int)blockIdx.y, &grp, &lo, &hi)) return;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * R);
  if (hi - lo <= 4)
    multiply_rows<X, R, 4, KS, 3, kWave>(a, grp, lo, hi, n0, smem);
  else
    multiply_rows<X, R, 16, KS, 2, kWave>(a, grp, lo, hi, n0, smem);
}

template <int X, int R, int MX, int KS, int SLOTS>
void launch(const Rows& a, int64_t slices, hipStream_t stream) {
  const dim3 grid((unsigned)((a.n + 16 * R - 1) / (16 * R)), (unsigned)slices);
  hipLaunchKernelGGL((mx_rows_kernel<X, R, MX, KS, SLOTS>), grid, dim3(64 * KS), 0, stream, a);
}

template <int X>
void launch_groups(const Rows& a, hipStream_t stream) {
  const int64_t active = a.groups < a.total_m ? a.groups : a.total_m, tiles = (a.n + 31) / 32;
  const dim3 grid((unsigned)tiles, (unsigned)active);
  if (active * tiles <= 1024)
    hipLaunchKernelGGL((mx_groups_kernel<X, 4>), grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((mx_groups_kernel<X, 2>), grid, dim3(128), 0, stream, a);
}

// Slices of a dense call's rows: `want` rows each, fewer slices than a grid
// may have.
int64_t slice_rows(Rows* a, int64_t want) {
  const int64_t least = (a->total_m + 4095) / 4096;
  a->slice = want * ((least + want - 1) / want > 1 ? (least + want - 1) / want : 1);
  return (a->total_m + a->slice - 1) / a->slice;
}

}  // namespace

// Dense calls.  Up to 8 rows: as many rows as there are at a time, four waves
// to 16 columns, and stages as LDS allows.  More: slices of 16 rows (8 where
// columns are few), two tiles of columns to a workgroup once one would give
// every CU a workgroup, two waves instead of four once that does
// (us; 16 rows of 2048 x 7168: 6.2 in slices of 8, 7.0; of 8192 x 4096: 7.5 with
// two tiles, 9.5 with one; of 16384 x 4096: 12.2 with two waves, 13.1 with four;
// 32 rows of 4096 x 7168: 9.2 in slices of 16, 15.6 in one).
hipError_t launch_mx_rows(const MxRows& m, hipStream_t stream) {
  Rows a{reinterpret_cast<const uint8_t*>(m.x), nullptr, m.x_rows, m.row_index, m.q, m.scale, m.offsets, (int)m.groups,
         m.total_m, m.n, m.k, m.total_m, m.y, m.out_f32};
  const int64_t tiles = (a.n + 15) / 16;
  if (a.offsets) {
    launch_groups<kBf16>(a, stream);
  } else if (a.total_m <= 2) {
    launch<kBf16, 1, 2, 4, 4>(a, 1, stream);
  } else if (a.total_m <= 4) {
    launch<kBf16, 1, 4, 4, 4>(a, 1, stream);
  } else if (a.total_m <= 8) {
    launch<kBf16, 1, 8, 4, 2>(a, 1, stream);
  } else if (tiles * ((a.total_m + 7) / 8) <= 256) {
    launch<kBf16, 1, 8, 4, 2>(a, slice_rows(&a, 8), stream);
  } else {
    const int64_t slices = slice_rows(&a, 16);
    if (tiles * slices <= 256)
      launch<kBf16, 1, 16, 4, 2>(a, slices, stream);
    else if (tiles * slices <= 512)
      launch<kBf16, 2, 16, 4, 2>(a, slices, stream);
    else
      launch<kBf16, 2, 16, 2, 2>(a, slices, stream);
  }
  return hipGetLastError();
}

template <int X>
static void few(Rows* a, hipStream_t stream) {
  if (a->offsets)
    launch_groups<X>(*a, stream);
  else
    launch<X, 1, 16, 4, 2>(*a, slice_rows(a, 16), stream);
}

hipError_t launch_mx_few(const MxProduct& p, hipStream_t stream) {
  Rows a{p.a, p.a_scale, p.a_rows, p.row_index, p.b, p.b_scale, p.offsets, p.groups, p.m, p.n, p.k, p.m, p.y, p.out_f32};
  if (p.a_fp4)
    few<kE2m1>(&a, stream);
  else if (p.out_f32)
    few<kE4m3Split>(&a, stream);
  else
    few<kE4m3>(&a, stream);
  return hipGetLastError();
}

}  // namespace fp8blk
