// Products of MXFP8 or MXFP4 rows with MXFP4 matrices (gfx950), dense and
// grouped over routed experts:
//   y[i][j] = sum over blocks b of 2^(Xa + Xb) sum over the block of a w
// by v_mfma_scale_f32_16x16x128_f8f6f4, which takes the E8M0 scales.
//
// Operand layout of a 16x16x128 (checked with random operands): lane l holds
// row l % 16; of E2M1 rows the 16 bytes (32 elements) at 16 (l / 16), of
// E4M3 rows the bytes at 16 (l / 16) and at 64 + 16 (l / 16).  Its scale is
// that of block l / 16 of the row.  The weights are the first operand, so
// that a lane's four results are four consecutive columns of one row of y.
//
// E4M3 products are added, in runs of 8 elements, 13 bits below the sum of
// the largest two exponents (probed; runs and blocks are added in fp32).  With
// |a| < 2 apart from |a| >= 2 no bit of any product lies that low, so float
// results take two products with the codes of either kind.
#include <type_traits>

#include "groups.h"
#include "launch.h"

namespace fp8blk {

namespace {

__device__ __forceinline__ v8i frag(u32x4 lo) { return (v8i){(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, 0, 0, 0, 0}; }
__device__ __forceinline__ v8i frag(u32x4 lo, u32x4 hi) {
  return (v8i){(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

__device__ __forceinline__ v8i frag(v8i f) { return f; }

// f(0), ..., f(N - 1) with compile-time arguments.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    each<N, I + 1>(f);
  }
}

// The codes with |a| >= 2 (bit 6 of a byte).
__device__ __forceinline__ v8i large_codes(v8i c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t m = ((uint32_t)c[i] >> 6) & 0x01010101u;
    c[i] &= (int)((m << 8) - m);
  }
  return c;
}

// Tiles.  A workgroup of WM x WN waves makes BM x BN outputs, a wave MI x NI
// tiles of 16 x 16.  K advances 256 elements (8 blocks) a stage through a ring
// of SLOTS stages in LDS that loads fill straight from memory; a row is 128
// bytes (E2M1) or 256 (E4M3) of a stage.  16-byte piece c of row r lies at
// c ^ turn(r), so that the 16 rows of an operand read spread over all banks
// (other turns took twice the time).
//
// A stage is two steps of 128 elements.  Which blocks a step takes is free as
// long as both operands agree: lane l takes block 2 (l / 16) in the first and
// the block after it in the second, so that the scales of both are two
// consecutive bytes of a row, read at once, of which the instruction picks the
// step's.
//
// While a step's matrix products run, the operands of the next step are read,
// each row's into the registers that its products have just left.  In the
// middle of stage s, then, every wave has all of stage s in registers or
// behind it and waits for its own part of stage s + 1; behind the one barrier
// there, stage s + SLOTS is loaded into the place of stage s.
//
// Scales come for two stages at a time, 16 bytes of a row: a load covers 16
// rows by four pieces of 4 bytes.
template <bool FP4>
__device__ __forceinline__ int turn(int r) {
  return FP4 ? (r >> 1) & 7 : r & 15;
}

template <bool A_FP4, int MI, int NI, int WM, int WN, int SLOTS>
struct Plan {
  static constexpr int kWaves = WM * WN, BM = 16 * MI * WM, BN = 16 * NI * WN;
  static constexpr int kARow = A_FP4 ? 128 : 256;
  static constexpr int kA = BM * kARow, kStage = kA + BN * 128;
  static constexpr int kALoads = kA / 1024 / kWaves, kLoads = kStage / 1024 / kWaves;   // of a wave and stage
  static constexpr int kChunk = (BM + BN) * 16;
  static constexpr int kScaleLoads = (kChunk / 256 + kWaves - 1) / kWaves;              // of a wave and chunk, at most
  static constexpr int kScales = SLOTS * kStage, kBytes = kScales + 2 * kChunk;
  static_assert(kA % (1024 * kWaves) == 0 && kStage % (1024 * kWaves) == 0, "shares of the loads");
  static_assert(kBytes + kMaxGroups * 4 <= 160 * 1024, "LDS");
};

template <bool A_FP4, bool SPLIT, int MI, int NI, int WM, int WN, int SLOTS>
__global__ __launch_bounds__(64 * WM * WN) void mx_gemm_kernel(MxProduct p, TileGrid grid) {
  using P = Plan<A_FP4, MI, NI, WM, WN, SLOTS>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[P::kBytes];
  __shared__ int upto[kMaxGroups];
  const int t = (int)threadIdx.x, lane = t & 63, r16 = lane & 15, kg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6), wm = wave % WM, wn = wave / WM;
  const uint32_t K = (uint32_t)p.k;
  const int stages = (int)((K + 255) / 256), pieces = (int)(K / 128);
  const uint32_t a_row = A_FP4 ? K / 2 : K, b_row = K / 2, s_row = K / 32;
  const uint32_t lds0 = lds_address(smem);
  const int tiles = count_tiles<P::BM, 64 * P::kWaves>(grid, upto);
  // where a lane's operands lie in a stage (rows of 16 tiles keep their turn),
  // and its scales in a chunk
  const uint32_t xa0 = A_FP4 ? (uint32_t)((wm * MI * 16 + r16) * 128 + ((2 * kg) ^ turn<true>(r16)) * 16)
                             : (uint32_t)((wm * MI * 16 + r16) * 256 + ((4 * (kg >> 1) + (kg & 1)) ^ turn<false>(r16)) * 16);
  const uint32_t xa1 = xa0 ^ (A_FP4 ? 16u : 32u);
  const uint32_t wb0 = (uint32_t)(P::kA + (wn * NI * 16 + r16) * 128 + ((2 * kg) ^ turn<true>(r16)) * 16);
  const uint32_t wb1 = wb0 ^ 16u;
  const uint32_t xs = (uint32_t)(P::kScales + (wm * MI * 16 + r16) * 16 + 2 * kg);
  const uint32_t ws = (uint32_t)(P::kScales + (P::BM + wn * NI * 16 + r16) * 16 + 2 * kg);
  // Pieces past K (of a last half stage) are read as zeros, at this offset.
  // Whether a lane's piece is in the upper half is the same for all its loads:
  // their rows are a multiple of 16 apart.
  constexpr uint32_t kNowhere = 0xFFFFFFF0u;
  constexpr int kAPer = P::kARow / 16;
  const uint32_t a_past = ((lane % kAPer) ^ turn<A_FP4>(wave * (64 / kAPer) + lane / kAPer)) & (kAPer / 2) ? kNowhere : 0u;
  const uint32_t b_past = ((lane % 8) ^ turn<true>(wave * 8 + lane / 8)) & 4 ? kNowhere : 0u;
  static_assert(P::kWaves * (64 / kAPer) % 16 == 0 && P::kWaves * 8 % 16 == 0, "rows of a lane's loads");

  for (int it = 0;; ++it) {
    const int id = tile_of_turn(it, tiles);
    if (id >= tiles) break;
    const Tile tile = tile_at<P::BM>(grid, upto, id);
    const int64_t m0 = tile.row0, n0 = (int64_t)tile.col * P::BN;
    const int cols = p.n - n0 < P::BN ? (int)(p.n - n0) : P::BN;
    // rows past the tile's end read its last one again; nothing of them is
    // stored
    auto row_of = [&](int r) -> uint32_t {
      r = r < tile.rows ? r : tile.rows - 1;
      return p.row_index ? (uint32_t)clamp_to(p.row_index[m0 + r], 0, (int)p.a_rows - 1) : (uint32_t)r;
    };
    const u32x4 a = buffer_of(p.a + (p.row_index ? 0 : m0 * a_row), kNowhere);
    const u32x4 b = buffer_of(p.b + (tile.group * p.n + n0) * b_row, kNowhere);
    const uint8_t* as = p.a_scale + (p.row_index ? 0 : m0 * s_row);
    const uint8_t* bs = p.b_scale + (tile.group * p.n + n0) * s_row;
    // this wave's loads of a stage: blocks wave, wave + kWaves, ... of 1 KiB
    uint32_t off[P::kLoads], soff[P::kScaleLoads];
#pragma unroll
    for (int j = 0; j < P::kLoads; ++j) {
      const int blk = j * P::kWaves + wave;
      if (j < P::kALoads) {
        const int r = blk * (64 / kAPer) + lane / kAPer;
        off[j] = row_of(r) * a_row + (uint32_t)(((lane % kAPer) ^ turn<A_FP4>(r)) * 16);
      } else {
        const int r = (blk - P::kA / 1024) * 8 + lane / 8, rr = r < cols ? r : cols - 1;
        off[j] = (uint32_t)rr * b_row + (uint32_t)(((lane % 8) ^ turn<true>(r)) * 16);
      }
    }
#pragma unroll
    for (int j = 0; j < P::kScaleLoads; ++j) {
      const int r = (j * P::kWaves + wave) * 16 + lane / 4;
      if (r < P::BM) {
        soff[j] = row_of(r) * s_row;
      } else {
        soff[j] = (uint32_t)(r - P::BM < cols ? r - P::BM : cols - 1) * s_row;
      }
    }
    // Scales past K are those of the row's last piece: of zeros, which only a
    // NaN among them changes, and that one has made the row's results NaN.
    auto load_scales = [&](int chunk) {
      int s = 4 * chunk + (lane & 3);
      s = s < pieces ? s : pieces - 1;
#pragma unroll
      for (int j = 0; j < P::kScaleLoads; ++j) {
        const int blk = j * P::kWaves + wave;
        if (blk * 256 < P::kChunk)
          lds_load4(blk * 16 < P::BM ? as : bs, soff[j] + (uint32_t)s * 4,
                    lds0 + P::kScales + (uint32_t)((chunk & 1) * P::kChunk + blk * 256));
      }
    };
    auto load_stage = [&](int s, uint32_t slot) {
      const bool half = 2 * s + 1 == pieces;
      const uint32_t ap = half ? a_past : 0u, bp = half ? b_past : 0u;
#pragma unroll
      for (int j = 0; j < P::kLoads; ++j) {
        const uint32_t to = lds0 + slot + (uint32_t)(j * P::kWaves + wave) * 1024;
        if (j < P::kALoads)
          lds_load16(a, (off[j] + (uint32_t)s * P::kARow) | ap, to);
        else
          lds_load16(b, (off[j] + (uint32_t)s * 128) | bp, to);
      }
    };

    v4f acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
    typename std::conditional<A_FP4, u32x4, v8i>::type xf[MI];
    u32x4 w0[NI], w1[NI];
    int sx[MI], sw[NI], swnext[NI];
    auto read_x = [&](uint32_t at, int i) {
      const u32x4 lo = *reinterpret_cast<const u32x4*>(smem + at + (uint32_t)(i * 16 * P::kARow));
      if constexpr (A_FP4)
        xf[i] = lo;
      else
        xf[i] = frag(lo, *reinterpret_cast<const u32x4*>(smem + (at ^ 128u) + (uint32_t)(i * 16 * P::kARow)));
    };
    auto read_w = [&](u32x4& w, uint32_t at, int i) {
      w = *reinterpret_cast<const u32x4*>(smem + at + (uint32_t)(i * 2048));
    };
    auto read_scale = [&](uint32_t at, int i) -> int {
      return (int)*reinterpret_cast<const uint16_t*>(smem + at + (uint32_t)(i * 256));
    };
    // row i of the products of step STEP of a stage
    auto multiply = [&](auto step, int i, const u32x4* w) {
      constexpr int STEP = decltype(step)::value;
      v8i hi = frag(xf[i]), lo = hi;
      if constexpr (SPLIT) {
        hi = large_codes(hi);
        lo = lo ^ hi;
      }
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(w[j]), hi, acc[i][j], 4, A_FP4 ? 4 : 0, STEP,
                                                                     sw[j], STEP, sx[i]);
        if constexpr (SPLIT)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(w[j]), lo, acc[i][j], 4, 0, STEP, sw[j],
                                                                       STEP, sx[i]);
      }
    };

    // the first stages and scales
    load_scales(0);
    load_scales(1);
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
      if (i < stages) load_stage(i, (uint32_t)(i * P::kStage));
    if (stages >= SLOTS) wait_loads<(SLOTS - 1) * P::kLoads>(); else wait_loads<0>();
    barrier();
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      read_x(xa0, i);
      sx[i] = read_scale(xs, i);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      read_w(w0[i], wb0, i);
      sw[i] = read_scale(ws, i);
    }

    uint32_t slot = 0;
    for (int s = 0; s < stages; ++s) {
      constexpr int kMult = SPLIT ? 2 * NI : NI, kXReads = A_FP4 ? 1 : 2;
      each<MI>([&](auto ic) {
        constexpr int i = decltype(ic)::value, first = i * NI / MI, last = (i + 1) * NI / MI;
        multiply(std::integral_constant<int, 0>{}, i, w0);
        read_x(slot + xa1, i);
#pragma unroll
        for (int j = first; j < last; ++j) read_w(w1[j], slot + wb1, j);
        __builtin_amdgcn_sched_group_barrier(0x008, kMult, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, kXReads + (last - first), 0);
      });
      // (the compiler would move products past the barrier and the branches)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) asm volatile("" : "+v"(acc[i][j]));
      wait_lds_reads();
      if (s + SLOTS - 1 < stages) wait_loads<(SLOTS - 2) * P::kLoads>(); else wait_loads<0>();
      barrier();
      if (s + SLOTS < stages) load_stage(s + SLOTS, slot);
      if (s & 1) load_scales((s + 1) / 2 + 1);
      slot = slot + P::kStage == SLOTS * P::kStage ? 0u : slot + P::kStage;
      const uint32_t at = (uint32_t)(((s + 1) >> 1 & 1) * P::kChunk + ((s + 1) & 1) * 8);
      each<MI>([&](auto ic) {
        constexpr int i = decltype(ic)::value, first = i * NI / MI, last = (i + 1) * NI / MI;
        multiply(std::integral_constant<int, 1>{}, i, w1);
        read_x(slot + xa0, i);
        sx[i] = read_scale(at + xs, i);
#pragma unroll
        for (int j = first; j < last; ++j) {
          read_w(w0[j], slot + wb0, j);
          swnext[j] = read_scale(at + ws, j);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, kMult, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, kXReads + 1 + 2 * (last - first), 0);
      });
#pragma unroll
      for (int j = 0; j < NI; ++j) sw[j] = swnext[j];
    }

    // lane l holds row l % 16 and columns 4 (l / 16) .. + 3 of each 16 x 16
    const bool whole = (p.n & 3) == 0;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int r = (wm * MI + i) * 16 + r16;
      if (r >= tile.rows) continue;
      const int64_t at = (m0 + r) * p.n + n0;
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int c = (wn * NI + j) * 16 + kg * 4;
        const v4f v = acc[i][j];
        if (whole) {
          if (c >= cols) continue;
          if (p.out_f32)
            *reinterpret_cast<v4f*>(reinterpret_cast<float*>(p.y) + at + c) = v;
          else
            *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(p.y) + at + c) =
                (u32x2){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (c + e >= cols) continue;
            if (p.out_f32)
              reinterpret_cast<float*>(p.y)[at + c + e] = v[e];
            else
              reinterpret_cast<uint16_t*>(p.y)[at + c + e] = (uint16_t)pack_bf16x2(v[e], 0.f);
          }
        }
      }
    }
    wait_loads<0>();
    wait_lds_reads();
    barrier();   // the next tile's loads reuse the stages
  }
}

template <bool A_FP4, bool SPLIT, int MI, int NI, int WM, int WN, int SLOTS>
void launch_tiles(const MxProduct& p, int64_t tiles, int num_cu, hipStream_t stream) {
  using P = Plan<A_FP4, MI, NI, WM, WN, SLOTS>;
  TileGrid g{p.offsets, p.groups, (int)p.m, (int)((p.n + P::BN - 1) / P::BN), 8};
  const int64_t per_cu = 160 * 1024 / (P::kBytes + kMaxGroups * 4);
  const int64_t most = (num_cu >= 8 ? num_cu / 8 * 8 : 8) * per_cu;
  const int64_t wgs = tiles < most ? (tiles + 7) / 8 * 8 : most;
  hipLaunchKernelGGL((mx_gemm_kernel<A_FP4, SPLIT, MI, NI, WM, WN, SLOTS>), dim3((unsigned)wgs), dim3(64 * WM * WN), 0,
                     stream, p, g);
}

// The tile of a call, from the rows of a group if they are spread evenly over
// as many groups as there can be, and the tiles that makes.  Large tiles read
// less; small ones fill the CUs.  Measured (us, bf16 results; E4M3 / E2M1 rows):
//   256 x 256, E2M1 only: 16384 rows on 64 experts of 4096 x 4096: 259, 128 x
//     256: 270;
//   128 x 256, from three quarters of the CUs on: 1500 x 4096 x 2048: 19.9 /
//     16.7, 128 x 128: 23.3 / 17.4; at half (2048 x 2048 x 4096) 30.8 / 24.0 and
//     21.5 / 18.2;
//   64 x 256 for up to 64 rows, 32 x 128 for up to 32: 2048 rows on 64 experts
//     of 4096 x 4096: 149 / 145 and 151 / 136, 64 x 64: 176 / 154; 1024 rows on
//     32: 73 / 69, 67 / 65 and 95 / 84;
//   64 x 64 by eight waves: 256 x 2048 x 7168: 15.3 / 13.8, by four 18.0 / 15.4.
// Float results of E4M3 rows, whose operands take twice the registers and
// products: 64 x 256 (2048 x 2048 x 4096: 34.5, 128 x 128: 40.5, 128 x 256:
// 55.9) or 32 x 128 (1009 x 2002 x 5120: 29.5, 64 x 64: 31.4).
template <bool A_FP4, bool SPLIT>
void launch_rule(const MxProduct& p, int num_cu, hipStream_t stream) {
  const int64_t active = p.offsets ? (p.groups < p.m ? p.groups : p.m) : 1;
  const int64_t rows = (p.m + active - 1) / active;
  auto most = [&](int64_t bm, int64_t bn) {     // tiles at most
    return (p.offsets ? p.m / bm + active : (p.m + bm - 1) / bm) * ((p.n + bn - 1) / bn);
  };
  auto fills = [&](int64_t bm, int64_t bn) {
    return 4 * active * ((rows + bm - 1) / bm) * ((p.n + bn - 1) / bn) >= 3 * num_cu;
  };
  if constexpr (SPLIT) {
    if (rows > 32 && fills(64, 256))
      launch_tiles<A_FP4, SPLIT, 2, 4, 2, 4, 2>(p, most(64, 256), num_cu, stream);
    else
      launch_tiles<A_FP4, SPLIT, 1, 4, 2, 2, 2>(p, most(32, 128), num_cu, stream);
  } else {
    if constexpr (A_FP4) {
      if (rows > 128 && fills(256, 256))
        return launch_tiles<A_FP4, SPLIT, 8, 4, 2, 4, 2>(p, most(256, 256), num_cu, stream);
    }
    if (rows > 64 && fills(128, 256))
      launch_tiles<A_FP4, SPLIT, 4, 4, 2, 4, A_FP4 ? 3 : 2>(p, most(128, 256), num_cu, stream);
    else if (rows > 64 && fills(128, 128))
      launch_tiles<A_FP4, SPLIT, 4, 2, 2, 4, A_FP4 ? 4 : 2>(p, most(128, 128), num_cu, stream);
    else if (rows > 32 && rows <= 64 && fills(64, 256))
      launch_tiles<A_FP4, SPLIT, 2, 4, 2, 4, 3>(p, most(64, 256), num_cu, stream);
    else if (rows <= 32 && fills(32, 128))
      launch_tiles<A_FP4, SPLIT, 1, 4, 2, 2, 2>(p, most(32, 128), num_cu, stream);
    else
      launch_tiles<A_FP4, SPLIT, 2, 1, 2, 4, 3>(p, most(64, 64), num_cu, stream);
  }
}

}  // namespace

// Few rows: the kernel that cuts K instead (us, E4M3 / E2M1; dense 64 x 4096 x
// 7168: 11.2 / 9.1, tiles 15.6 / 13.9, 128 rows: 18.5 / 14.7 and 15.6 / 13.9;
// 512 rows on 60 of 64 experts of 4096 x 4096: 131 / 125, tiles 137 / 126, 1024
// rows on 32: 122 / 120, tiles 67 / 65).
hipError_t launch_mx_product(const MxProduct& p, int num_cu, hipStream_t stream) {
  const int64_t active = p.offsets ? (p.groups < p.m ? p.groups : p.m) : 1;
  if (p.offsets ? p.m <= 8 * active : ((p.m + 15) / 16) * ((p.n + 15) / 16) <= 4 * num_cu) return launch_mx_few(p, stream);
  if (p.a_fp4)
    launch_rule<true, false>(p, num_cu, stream);
  else if (p.out_f32)
    launch_rule<false, true>(p, num_cu, stream);
  else
    launch_rule<false, false>(p, num_cu, stream);
  return hipGetLastError();
}

}  // namespace fp8blk
