// Products of a few bf16 rows with NVFP4 weights (gfx950), dense and
// grouped over routed experts:
//   y[i][j] = g[j] * sum_k x[i][k] e2m1(c[j][k]) e4m3(S[j][k / 16])
// An e2m1 value has 2 significant bits and an e4m3 scale 4, so their
// product is exact in bf16; sums are fp32 and the tensor scale multiplies
// them once.  Bound by reading the weights, 0.5625 bytes each.
//
// Two ways to multiply:
//   * matrix cores (mfma_rows): 16 weight rows by up to 16 x rows per
//     16x16x32 MFMA.  The operand layout wants 16 rows per load, four lanes
//     apart, which the address unit takes 64 pieces at a time (75% busy and
//     4.6 TB/s with such loads), so a wave loads rows along k, 128 bytes of
//     codes per 8 lanes, and turns them in its own piece of LDS.  Decoding
//     costs 2 vector instructions per weight whatever the x rows.
//   * dot products (dot_rows): for one or two x rows, 16 lanes to a weight
//     row, v_dot2_f32_bf16 on the unscaled values of a block and one fused
//     multiply by its scale: 1.7 instructions per weight at two rows, no
//     LDS.  Taken for groups of at most two rows on large grids: 64 rows on
//     52 experts of 4096 x 7168 in 150 us (5.7 TB/s), against 185 us on the
//     matrix cores; on grids of up to 256 tiles it was 7% slower at two rows.
#include "device.h"
#include "launch.h"

namespace fp8blk {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// Orders a wave's own LDS reads and writes across its lanes (the hardware
// keeps them in order; this keeps the compiler to it).
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Eight codes of a dword times the block scale, as an MFMA operand.
__device__ __forceinline__ v8bf decode8(uint32_t c, float s) {
  const v2f d0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
  const v2f d1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
  const v2f d2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
  const v2f d3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
  const u32x4 w = {pack_bf16x2(d0[0] * s, d0[1] * s), pack_bf16x2(d1[0] * s, d1[1] * s),
                   pack_bf16x2(d2[0] * s, d2[1] * s), pack_bf16x2(d3[0] * s, d3[1] * s)};
  return __builtin_bit_cast(v8bf, w);
}

// The ordinal-th non-empty group and its rows; false where there are fewer.
// Every wave finds it by itself, 256 groups at a time (their offsets loaded
// together: one at a time cost a memory latency each).
__device__ __forceinline__ bool nth_group(const MatvecArgs& a, int ordinal, int lane, int* grp, int* lo, int* hi) {
  int seen = 0;
  for (int b = 0; b < (int)a.groups; b += 256) {
    int l[4], h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = b + i * 64 + lane;
      const int at = e < (int)a.groups ? e : (int)a.groups - 1;
      l[i] = a.offsets[at];
      h[i] = a.offsets[at + 1];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      l[i] = clampi(l[i], 0, (int)a.total_m);
      h[i] = b + i * 64 + lane < (int)a.groups ? clampi(h[i], l[i], (int)a.total_m) : l[i];
      const unsigned long long full = __builtin_amdgcn_ballot_w64(h[i] > l[i]);
      const int here = __builtin_popcountll(full);
      if (ordinal < seen + here) {
        const bool mine = h[i] > l[i] && __builtin_popcountll(full & ((1ull << lane) - 1)) == ordinal - seen;
        const int src = __builtin_ctzll(__builtin_amdgcn_ballot_w64(mine));
        *grp = b + i * 64 + src;
        *lo = __builtin_amdgcn_readlane(l[i], src);
        *hi = __builtin_amdgcn_readlane(h[i], src);
        return true;
      }
      seen += here;
    }
  }
  return false;
}

// Loads through a buffer descriptor: 32-bit offsets from a base that the
// whole workgroup shares, and bytes at or past its length read as zeros, so
// lanes with nothing to load add kNoLoad, past any length, and need no branch.
typedef __amdgpu_buffer_rsrc_t Buffer;
constexpr uint32_t kNoLoad = 0x80000000u;   // lengths are below 2^31
__device__ __forceinline__ Buffer make_buffer(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, 0x00027000);
}
__device__ __forceinline__ u32x4 load16(Buffer b, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0);
}
// Codes of weights: NT, with the nontemporal bit (scales are read 32 bytes of
// a line at a time, and keep theirs).
template <bool NT>
__device__ __forceinline__ u32x4 load_codes(Buffer b, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, NT ? 2 : 0);
}

// One run of 32 weights: a lane's share of a step of dot_rows.
struct Run {
  u32x4 c;
  uint32_t s;
};

template <bool OUT_F32>
__device__ __forceinline__ void store_y(const MatvecArgs& a, int grp, int64_t row, int64_t j, float v) {
  v *= a.global_scale[((int64_t)grp * a.n + j) / a.rows_per_tensor];
  if constexpr (OUT_F32)
    reinterpret_cast<float*>(a.y)[row * a.n + j] = v;
  else
    reinterpret_cast<uint16_t*>(a.y)[row * a.n + j] = (uint16_t)pack_bf16x2(v, 0.f);
}

// Rows [lo, lo + rows) (one or two) of x by the 32 weight rows from n0, by
// one wave: lane l holds 32 consecutive k of weight row 4 q + l / 16 (a step
// is 512 k, 256 bytes of a row per 16 lanes), the next step's loads in
// flight during the products of this one.
//
// A block's sum is of unscaled products, which can leave the fp32 range where
// the scaled ones do not (|x| from 3.5e36 on; a scale of 0 then makes a NaN).
// That leaves an infinity or NaN in the row's sum whatever is added to it, so
// such sums are seen at the end: nothing is stored then, and the result is
// false.  Scaling the codes by their scale's power of two as they are
// converted avoids it too, for 2% more time (52 experts of 4096 x 7168: 154 us
// instead of 151).
constexpr int kDotQ = 8;
template <bool NT, bool OUT_F32>
__device__ __forceinline__ bool dot_rows(const MatvecArgs& a, int grp, int lo, int rows, int64_t n0, int lane) {
  constexpr int Q = kDotQ, M = 2;
  const int kl = lane & 15, sub = lane >> 4;
  const int K = (int)a.k;
  const int steps = (K + 511) / 512;
  const int64_t first = (int64_t)grp * a.n + n0;
  const int64_t nr = a.n - n0 < 4 * Q ? a.n - n0 : 4 * Q;
  const Buffer qb = make_buffer(a.q + first * (K / 2), (uint32_t)(nr * (K / 2)));
  const Buffer sb = make_buffer(a.block_scale + first * (K / 16), (uint32_t)(nr * (K / 16)));
  const Buffer xb = make_buffer(a.x, (uint32_t)(a.x_rows * K * 2));
  const uint32_t q0 = (uint32_t)(sub * (K / 2) + kl * 16), s0 = (uint32_t)(sub * (K / 16) + kl * 2);
  uint32_t x0[M];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    int r = lo + (m < rows ? m : 0);
    if (a.row_index) r = clampi(a.row_index[r], 0, (int)a.x_rows - 1);
    x0[m] = (uint32_t)r * (uint32_t)(K * 2) + kl * 64;
  }
  float acc[Q][M];
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int m = 0; m < M; ++m) acc[q][m] = 0.f;
  Run c0[Q], c1[Q];
  u32x4 xa[M][4], xc[M][4];
  auto load = [&](int s, Run* c, u32x4 (*x)[4]) {
    const uint32_t skip = s * 512 + kl * 32 < K ? 0u : kNoLoad;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[m][i] = load16(xb, ((x0[m] + (uint32_t)s * 1024) | skip) + 16 * i);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      c[q].c = load_codes<NT>(qb, (q0 + (uint32_t)(q * 2 * K + s * 256)) | skip);
      c[q].s = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(sb, (s0 + (uint32_t)(q * (K / 4) + s * 32)) | skip, 0, 0);
    }
  };
  auto multiply = [&](const Run* c, const u32x4 (*x)[4]) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const v2f sc = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[q].s, false);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        v2bf w[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t d = c[q].c[2 * b + h];
          w[4 * h + 0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 0);
          w[4 * h + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 1);
          w[4 * h + 2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 2);
          w[4 * h + 3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 3);
        }
#pragma unroll
        for (int m = 0; m < M; ++m) {
          float s = 0.f;
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            const uint32_t xw = x[m][2 * b + p / 4][p & 3];
            s = __builtin_amdgcn_fdot2_f32_bf16(w[p], __builtin_bit_cast(v2bf, xw), s, false);
          }
          acc[q][m] = __builtin_fmaf(s, sc[b], acc[q][m]);
        }
      }
    }
  };
  load(0, c0, xa);
  for (int s = 0; s < steps; s += 2) {
    load(s + 1, c1, xc);
    __builtin_amdgcn_sched_barrier(0);   // the loads go out before the products they do not feed
    multiply(c0, xa);
    __builtin_amdgcn_sched_barrier(0);
    load(s + 2, c0, xa);
    __builtin_amdgcn_sched_barrier(0);
    multiply(c1, xc);
    __builtin_amdgcn_sched_barrier(0);
  }
  bool finite = true;
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int m = 0; m < M; ++m) {
      float v = acc[q][m];
      v = dpp_add<kQuadSwap1>(v);
      v = dpp_add<kQuadSwap2>(v);
      v = dpp_add<kRowHalfMirror>(v);
      acc[q][m] = dpp_add<kRowMirror>(v);
      finite = finite && __builtin_fabsf(acc[q][m]) < __builtin_inff();
    }
  if (__builtin_amdgcn_ballot_w64(!finite) != 0) return false;
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int64_t j = n0 + q * 4 + sub;
      if (kl == 0 && m < rows && j < a.n) store_y<OUT_F32>(a, grp, lo + m, j, acc[q][m]);
    }
  return true;
}

// LDS of one step of a wave in mfma_rows.
template <int R, int MX>
struct Stage {
  // codes [16 R][128 bytes] with the 16-byte chunk c of row r at c ^ (r & 7),
  // scales [16 R][16], x [MX][528 bytes] (512 and a pad), so that both the
  // row-wise writes and the reads of 16 rows at one k spread over the banks
  static constexpr int kCodes = R * 2048, kScales = R * 256, kXRow = 528;
  static constexpr int kStep = kCodes + kScales + MX * kXRow;
  // reused for the wave's sums
  static constexpr int kSums = R * ((MX + 15) / 16) * 1024;
  static constexpr int kBytes = kStep > kSums ? kStep : kSums;
};

// Rows [lo, hi) of x, MX at a time, by the 16 R weight rows from n0, by a
// workgroup of KS waves: wave w takes the steps w, w + KS, ... of 256 k, and
// the waves' sums are added in LDS in wave order.  In a step lane l holds 64
// consecutive k of weight row l % 16 of each tile and of x row l % 16, at
// 64 (l / 16): the order of k within a step is the lanes' own, the same on
// both sides.  The next step's loads are in flight (in registers) while this
// one is multiplied from LDS.  AL: k % 64 == 0 and buffers aligned so that a
// lane's codes are 16 aligned bytes and its scales a dword.
template <bool AL, int R, int MX, int KS, bool NT, bool OUT_F32>
__device__ __forceinline__ void mfma_rows(const MatvecArgs& a, int grp, int lo, int hi, int64_t n0, uint8_t* smem,
                                          int t, int wave) {
  using S = Stage<R, MX>;
  constexpr int XI = (MX + 1) / 2;        // 16-byte x loads per lane and step
  constexpr int CT = (MX + 15) / 16;      // tiles of 16 x rows
  const int lane = t & 63, col = lane & 15, g = lane >> 4;
  const int K = (int)a.k;
  const int steps = (K + 255) / 256;
  const int64_t first = (int64_t)grp * a.n + n0;
  const int64_t rows = a.n - n0 < 16 * R ? a.n - n0 : 16 * R;
  const Buffer qb = make_buffer(a.q + first * (K / 2), (uint32_t)(rows * (K / 2)));
  // scales are read a dword at a time: from the dword that holds the first
  const uint8_t* sbase = a.block_scale + first * (K / 16);
  const uint32_t smis = AL ? 0u : (uint32_t)(reinterpret_cast<uintptr_t>(sbase) & 3);
  const Buffer sb = make_buffer(sbase - smis, ((uint32_t)(rows * (K / 16)) + smis + 3u) & ~3u);
  const Buffer xb = make_buffer(a.x, (uint32_t)(a.x_rows * K * 2));
  uint8_t* lds = smem + wave * S::kBytes;

  // unsigned: hi can lie within MX of 2^31
  for (uint32_t next = (uint32_t)lo; next < (uint32_t)hi; next += MX) {
    const int m0 = (int)next;
    const int mr = hi - m0 < MX ? hi - m0 : MX;
    uint32_t x0[XI];
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int m = 2 * i + (lane >> 5);
      int r = m0 + (m < mr ? m : 0);
      if (a.row_index) r = clampi(a.row_index[r], 0, (int)a.x_rows - 1);
      x0[i] = ((uint32_t)r * (uint32_t)(K * 2) + (lane & 31) * 16) | (m < mr ? 0u : kNoLoad);
    }
    v4f acc[R][CT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[r][c] = (v4f){0.f, 0.f, 0.f, 0.f};
    u32x4 cq[R][2], cx[XI];
    uint32_t cs[R];

    auto load = [&](int s) {
      const int kc = s * 256 + (lane & 7) * 32;      // this lane's codes
      const int ks = s * 256 + (lane & 3) * 64;      // its four scales
      const int kx = s * 256 + (lane & 31) * 8;      // its x
      const uint32_t qo = (uint32_t)((lane >> 3) * (K / 2) + kc / 2);
      const uint32_t so = (uint32_t)((lane >> 2) * (K / 16) + ks / 16);
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t o = qo + (uint32_t)((16 * r + 8 * h) * (K / 2));
          if constexpr (AL) {
            cq[r][h] = load_codes<NT>(qb, o | (kc < K ? 0u : kNoLoad));
          } else {
            const u32x2 u = __builtin_amdgcn_raw_buffer_load_b64(qb, o | (kc < K ? 0u : kNoLoad), 0, 0);
            const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(qb, (o + 8) | (kc + 16 < K ? 0u : kNoLoad), 0, 0);
            cq[r][h] = (u32x4){u.x, u.y, v.x, v.y};
          }
        }
        const uint32_t o = so + (uint32_t)(16 * r * (K / 16));
        if constexpr (AL) {
          cs[r] = __builtin_amdgcn_raw_buffer_load_b32(sb, o | (ks < K ? 0u : kNoLoad), 0, 0);
        } else {
          // four bytes at any address: two dwords, shifted; bytes past the
          // row belong to the next one and are cleared
          const uint32_t at = o + smis, skip = ks < K ? 0u : kNoLoad;
          const uint32_t u = __builtin_amdgcn_raw_buffer_load_b32(sb, (at & ~3u) | skip, 0, 0);
          const uint32_t v = __builtin_amdgcn_raw_buffer_load_b32(sb, ((at & ~3u) + 4u) | skip, 0, 0);
          const uint32_t w = (uint32_t)((((uint64_t)v << 32) | u) >> ((at & 3) * 8));
          const int left = (K - ks) / 16;
          cs[r] = left >= 4 ? w : (left > 0 ? w & ((1u << (8 * left)) - 1u) : 0u);
        }
      }
#pragma unroll
      for (int i = 0; i < XI; ++i) cx[i] = load16(xb, (x0[i] + (uint32_t)s * 512) | (kx < K ? 0u : kNoLoad));
    };
    load(wave);
    for (int s = wave; s < steps; s += KS) {
      // this step into LDS; one wave's LDS operations keep their order
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<u32x4*>(lds + r * 2048 + (8 * h + (lane >> 3)) * 128 +
                                    (((lane & 7) ^ (lane >> 3)) & 7) * 16) = cq[r][h];
        *reinterpret_cast<uint32_t*>(lds + S::kCodes + r * 256 + lane * 4) = cs[r];
      }
#pragma unroll
      for (int i = 0; i < XI; ++i)
        *reinterpret_cast<u32x4*>(lds + S::kCodes + S::kScales + (2 * i + (lane >> 5)) * S::kXRow + (lane & 31) * 16) =
            cx[i];
      // With 32 rows of x (16 loads a step) the step past the last one is not
      // loaded: 8192 x 7168 in 15.2 us, 16.4 with it.  With fewer rows, or the
      // loads of AL false, the branch cost more than those loads (4096 x 16384
      // at 16 rows: 12.9 us, 12.2 without).
      if (!(AL && MX == 32) || s + KS < steps) load(s + KS);
      __builtin_amdgcn_sched_barrier(0);
      wave_fence();
      u32x4 xf[CT][8];
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const int m = 16 * c + col;      // columns past the rows are not stored: any row will do
        const uint8_t* xl = lds + S::kCodes + S::kScales + (m < mr ? m : 0) * S::kXRow + g * 128;
#pragma unroll
        for (int i = 0; i < 8; ++i) xf[c][i] = *reinterpret_cast<const u32x4*>(xl + 16 * i);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint8_t* row = lds + r * 2048 + col * 128;
        const u32x4 q0 = *reinterpret_cast<const u32x4*>(row + (((2 * g) ^ col) & 7) * 16);
        const u32x4 q1 = *reinterpret_cast<const u32x4*>(row + (((2 * g + 1) ^ col) & 7) * 16);
        float f[4];
        decode4_e4m3(*reinterpret_cast<const uint32_t*>(lds + S::kCodes + r * 256 + col * 16 + g * 4), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const v8bf w = decode8(i < 4 ? q0[i] : q1[i - 4], f[i / 2]);
#pragma unroll
          for (int c = 0; c < CT; ++c)
            acc[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(v8bf, xf[c][i]), acc[r][c], 0, 0,
                                                                0);
        }
      }
      wave_fence();
    }

    // lane l holds rows 4 (l / 16) + v of column l % 16
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < CT; ++c)
        *reinterpret_cast<v4f*>(red + ((wave * CT + c) * R + r) * 256 + lane * 4) = acc[r][c];
    __syncthreads();
    for (int e = t; e < 16 * R * mr; e += 64 * KS) {
      const int m = e / (16 * R), j = e % (16 * R);
      if (n0 + j < a.n) {
        const int at = (m >> 4) * (R * 256) + (j >> 4) * 256 + (((j >> 2) & 3) * 16 + (m & 15)) * 4 + (j & 3);
        float v = red[at];
#pragma unroll
        for (int w = 1; w < KS; ++w) v += red[w * (CT * R * 256) + at];
        store_y<OUT_F32>(a, grp, m0 + m, n0 + j, v);
      }
    }
    __syncthreads();
  }
}

template <bool AL, int R, int MX, int KS, bool NT, bool OUT_F32>
__global__ __launch_bounds__(64 * KS) void matvec_kernel(MatvecArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[KS * Stage<R, MX>::kBytes];
  const int t = (int)threadIdx.x;
  int grp = 0, lo = 0, hi = 0;
  if (a.offsets) {
    if (!nth_group(a, (int)blockIdx.y, t & 63, &grp, &lo, &hi)) return;
  } else {
    lo = (int)(blockIdx.y * a.slice);
    hi = lo + (int)a.slice < (int)a.total_m ? lo + (int)a.slice : (int)a.total_m;
  }
  mfma_rows<AL, R, MX, KS, NT, OUT_F32>(a, grp, lo, hi, (int64_t)blockIdx.x * (16 * R), smem, t,
                                    __builtin_amdgcn_readfirstlane(t >> 6));
}

// One wave per 32 weight rows; the matrix cores for groups of more than two
// rows, which a skewed routing has among its small ones, and for sums that
// left the fp32 range (the cores take scaled weights).
template <bool NT, bool OUT_F32>
__global__ __launch_bounds__(64) void matvec_stream_kernel(MatvecArgs a) {
  static_assert(4 * kDotQ == 16 * 2, "both ways take 32 weight rows");
  __shared__ __attribute__((aligned(16))) uint8_t smem[Stage<2, 16>::kBytes];
  const int t = (int)threadIdx.x;
  int grp = 0, lo = 0, hi = (int)a.total_m;
  if (a.offsets && !nth_group(a, (int)blockIdx.y, t, &grp, &lo, &hi)) return;
  const int64_t n0 = (int64_t)blockIdx.x * 32;
  if (hi - lo > 2 || !dot_rows<NT, OUT_F32>(a, grp, lo, hi - lo, n0, t))
    mfma_rows<true, 2, 16, 1, NT, OUT_F32>(a, grp, lo, hi, n0, smem, t, 0);
}

template <bool AL, int R, int MX, int KS, bool NT = false>
void launch_tiles(const MatvecArgs& a, int64_t slices, hipStream_t stream) {
  const dim3 grid((unsigned)((a.n + 16 * R - 1) / (16 * R)), (unsigned)slices);
  if (a.out_f32)
    hipLaunchKernelGGL((matvec_kernel<AL, R, MX, KS, NT, true>), grid, dim3(64 * KS), 0, stream, a);
  else
    hipLaunchKernelGGL((matvec_kernel<AL, R, MX, KS, NT, false>), grid, dim3(64 * KS), 0, stream, a);
}

template <bool NT>
void launch_stream(const MatvecArgs& a, int64_t active, hipStream_t stream) {
  const dim3 grid((unsigned)((a.n + 31) / 32), (unsigned)active);
  if (a.out_f32)
    hipLaunchKernelGGL((matvec_stream_kernel<NT, true>), grid, dim3(64), 0, stream, a);
  else
    hipLaunchKernelGGL((matvec_stream_kernel<NT, false>), grid, dim3(64), 0, stream, a);
}

// Rows of x per pass, tiles per workgroup and waves that share k.  tiles:
// 16-row tiles of all groups.  Up to 256 (one per CU) the most waves per
// tile win (4096 x 7168: 7.8 us at 16 rows with 8 waves to a tile, 9.0 with
// 4, 11.0 with 4 to two tiles); past that two tiles share a wave's x (7168 x
// 2048: 5.8 us, against 7.3 with 8 waves to a tile), and four on large grids
// (64 groups of 16 rows, 7168 x 2048: 155 us, 171 with two).  With one or
// two rows there is little x to share (8192 x 4096: 6.4 us with 4 waves to a
// tile, 7.1 with two tiles).  One tile per workgroup spends as much of the
// address unit on x as on weights, so it loads no more rows than it needs
// (4096 x 7168: 6.4 us for up to 4 rows, 6.7 for up to 8, 7.4 for up to 16),
// except for groups, of which one may have many more rows than the others;
// two steps in flight, or half a tile per workgroup, gained nothing.
template <bool AL>
void launch_rows(const MatvecArgs& a, int64_t slices, int64_t tiles, int64_t rows, bool nt, hipStream_t stream) {
  if (rows <= 2 && !a.offsets) {
    if (tiles <= 256)
      launch_tiles<AL, 1, 2, 8>(a, slices, stream);
    else
      launch_tiles<AL, 1, 2, 4>(a, slices, stream);
  } else if (rows <= 16) {
    if (tiles <= 256 && rows <= 4 && !a.offsets)
      launch_tiles<AL, 1, 4, 8>(a, slices, stream);
    else if (tiles <= 256 && rows <= 8 && !a.offsets)
      launch_tiles<AL, 1, 8, 8>(a, slices, stream);
    else if (tiles <= 256)
      launch_tiles<AL, 1, 16, 8>(a, slices, stream);
    else if (tiles <= 1024)
      launch_tiles<AL, 2, 16, 4>(a, slices, stream);
    else if (AL && nt)
      launch_tiles<AL, 4, 16, 4, AL>(a, slices, stream);
    else
      launch_tiles<AL, 4, 16, 4>(a, slices, stream);
  } else {
    if (tiles <= 256)
      launch_tiles<AL, 1, 32, 8>(a, slices, stream);
    else if (tiles <= 1024)
      launch_tiles<AL, 2, 32, 4>(a, slices, stream);
    else if (AL && nt)
      launch_tiles<AL, 4, 32, 2, AL>(a, slices, stream);
    else
      launch_tiles<AL, 4, 32, 2>(a, slices, stream);
  }
}

}  // namespace

hipError_t launch_matvec(const MatvecArgs& args, hipStream_t stream) {
  MatvecArgs a = args;
  // non-empty groups at most, and rows per group at least, if they are even
  const int64_t active = a.offsets ? (a.groups < a.total_m ? a.groups : a.total_m) : 1;
  int64_t rows = (a.total_m + active - 1) / active;
  const int64_t tiles = (a.n + 15) / 16 * active;
  const bool al = a.k % 64 == 0 && ((reinterpret_cast<uintptr_t>(a.q) & 15) == 0) &&
                  ((reinterpret_cast<uintptr_t>(a.block_scale) & 3) == 0);
  // Where tiles leave CUs idle, more than eight rows are shared out among
  // workgroups (1000 x 7184: 16 rows in 7.3 us, in one slice 8.0; 32 rows in
  // 8.4 and 11.4; slices of four took 7.9 and 8.3, and 8 rows of 2000 x 7184
  // 7.6 in two slices, 7.1 in one).
  int64_t slices = active;
  a.slice = a.total_m;
  if (!a.offsets && tiles <= 128 && rows > 8) {
    const int64_t most = 256 / tiles < (rows + 7) / 8 ? 256 / tiles : (rows + 7) / 8;
    a.slice = rows = (a.total_m + most - 1) / most;
    slices = (a.total_m + rows - 1) / rows;
  }
  const bool nt = al && tiles > 1024 && active * a.n * (a.k / 2) > kCached;
  if (al && rows <= 2 && tiles > 1024) {
    if (nt)
      launch_stream<true>(a, active, stream);
    else
      launch_stream<false>(a, active, stream);
  } else if (al) {
    launch_rows<true>(a, slices, tiles, rows, nt, stream);
  } else {
    launch_rows<false>(a, slices, tiles, rows, nt, stream);
  }
  return hipGetLastError();
}

}  // namespace fp8blk
