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
// tiles of 16 x 16.  K advances 128 elements a step through a ring of SLOTS
// stages in LDS that loads fill straight from memory; a row is 64 bytes (E2M1)
// or 128 (E4M3) of a stage.  16-byte piece c of row r lies at c ^ turn(r), so
// that the operand reads of 16 rows spread over all banks, whether eight or
// sixteen lanes are served at once.
//
// One barrier a step: at the top of step s every wave has its operands of
// step s in registers (so stage s may be overwritten) and has waited for its
// own part of stage s + 1, so behind the barrier stage s + SLOTS is loaded
// into the place of stage s, and the matrix products of step s run while the
// operands of step s + 1 are read, each row's into the registers that its
// products have just left.
//
// Scales come in chunks of four steps, 16 bytes of a row: a load covers 16
// rows by four steps of 4 bytes.  A lane reads the byte of its row and block
// with the operand.
template <bool FP4>
__device__ __forceinline__ int turn(int r) {
  return FP4 ? ((r >> 2) & 3) ^ (r & 2) : (r >> 1) & 7;
}

template <bool A_FP4, int MI, int NI, int WM, int WN, int SLOTS>
struct Plan {
  static constexpr int kWaves = WM * WN, BM = 16 * MI * WM, BN = 16 * NI * WN;
  static constexpr int kARow = A_FP4 ? 64 : 128;
  static constexpr int kA = BM * kARow, kStage = kA + BN * 64;
  static constexpr int kLoads = kStage / 1024 / kWaves;          // of a wave and stage
  static constexpr int kChunk = (BM + BN) * 16;
  static constexpr int kScaleLoads = kChunk / 256 / kWaves;      // of a wave and chunk
  static constexpr int kScales = SLOTS * kStage, kBytes = kScales + 2 * kChunk;
  static_assert(kStage % (1024 * kWaves) == 0 && kChunk % (256 * kWaves) == 0 && kScaleLoads <= 4, "shares of the loads");
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
  const int steps = (int)(K / 128);
  const uint32_t a_row = A_FP4 ? K / 2 : K, b_row = K / 2, s_row = K / 32;
  const uint32_t lds0 = lds_address(smem);
  const int tiles = count_tiles<P::BM, 64 * P::kWaves>(grid, upto);
  // where a lane's operands lie in a stage, and its scales in a chunk
  const uint32_t xa = (uint32_t)((wm * MI * 16 + r16) * P::kARow + (kg ^ turn<A_FP4>(r16)) * 16);
  const uint32_t wb = (uint32_t)(P::kA + (wn * NI * 16 + r16) * 64 + (kg ^ turn<true>(r16)) * 16);
  const uint32_t xs = (uint32_t)(P::kScales + (wm * MI * 16 + r16) * 16 + kg);
  const uint32_t ws = (uint32_t)(P::kScales + (P::BM + wn * NI * 16 + r16) * 16 + kg);

  for (int it = 0;; ++it) {
    const int id = tile_of_turn(it, 2);
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
    const uint8_t* a = p.a + (p.row_index ? 0 : m0 * a_row);
    const uint8_t* as = p.a_scale + (p.row_index ? 0 : m0 * s_row);
    const uint8_t* b = p.b + (tile.group * p.n + n0) * b_row;
    const uint8_t* bs = p.b_scale + (tile.group * p.n + n0) * s_row;
    // this wave's loads of a stage: blocks wave, wave + kWaves, ... of 1 KiB
    uint32_t off[P::kLoads], soff[P::kScaleLoads];
#pragma unroll
    for (int j = 0; j < P::kLoads; ++j) {
      const int blk = j * P::kWaves + wave;
      if (blk * 1024 < P::kA) {
        constexpr int per = P::kARow / 16;
        const int r = blk * (64 / per) + lane / per;
        off[j] = row_of(r) * a_row + (uint32_t)(((lane % per) ^ turn<A_FP4>(r)) * 16);
      } else {
        const int r = (blk - P::kA / 1024) * 16 + lane / 4, rr = r < cols ? r : cols - 1;
        off[j] = (uint32_t)rr * b_row + (uint32_t)(((lane % 4) ^ turn<true>(r)) * 16);
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
    auto load_scales = [&](int chunk) {
      int s = 4 * chunk + (lane & 3);
      s = s < steps ? s : steps - 1;
#pragma unroll
      for (int j = 0; j < P::kScaleLoads; ++j) {
        const int blk = j * P::kWaves + wave;
        lds_load4(blk * 16 < P::BM ? as : bs, soff[j] + (uint32_t)s * 4,
                  lds0 + P::kScales + (uint32_t)((chunk & 1) * P::kChunk + blk * 256));
      }
    };
    auto load_stage = [&](int s, uint32_t slot) {
#pragma unroll
      for (int j = 0; j < P::kLoads; ++j) {
        const int blk = j * P::kWaves + wave;
        const bool is_a = blk * 1024 < P::kA;
        lds_load16(is_a ? a : b, off[j] + (uint32_t)s * (is_a ? P::kARow : 64), lds0 + slot + (uint32_t)blk * 1024);
      }
    };

    v4f acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
    typename std::conditional<A_FP4, u32x4, v8i>::type xf[MI];
    u32x4 wf[NI], wnext[NI];
    int sx[MI], sw[NI], swnext[NI];
    auto read_x = [&](uint32_t slot, uint32_t scale, int i) {
      sx[i] = smem[scale + xs + (uint32_t)(i * 256)];
      const uint8_t* at = smem + (slot + xa + (uint32_t)(i * 16 * P::kARow));
      if constexpr (A_FP4) {
        xf[i] = *reinterpret_cast<const u32x4*>(at);
      } else {
        const uint8_t* up = smem + ((slot + xa + (uint32_t)(i * 16 * P::kARow)) ^ 64u);
        xf[i] = frag(*reinterpret_cast<const u32x4*>(at), *reinterpret_cast<const u32x4*>(up));
      }
    };
    auto read_w = [&](uint32_t slot, uint32_t scale, int i) {
      swnext[i] = smem[scale + ws + (uint32_t)(i * 256)];
      wnext[i] = *reinterpret_cast<const u32x4*>(smem + (slot + wb + (uint32_t)(i * 1024)));
    };
    // the first stages and scales
    load_scales(0);
    load_scales(1);
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
      if (i < steps) load_stage(i, (uint32_t)(i * P::kStage));
    wait_loads<0>();
    barrier();
#pragma unroll
    for (int i = 0; i < MI; ++i) read_x(0, 0, i);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      read_w(0, 0, i);
      wf[i] = wnext[i];
      sw[i] = swnext[i];
    }

    uint32_t slot = 0;
    for (int s = 0; s < steps; ++s) {
      wait_lds_reads();
      if (s + SLOTS - 1 < steps) wait_loads<(SLOTS - 2) * P::kLoads>(); else wait_loads<0>();
      barrier();
      if (s + SLOTS < steps) load_stage(s + SLOTS, slot);
      if ((s & 3) == 3) load_scales(s / 4 + 2);
      slot = slot + P::kStage == SLOTS * P::kStage ? 0u : slot + P::kStage;
      const uint32_t at = (uint32_t)(((s + 1) >> 2 & 1) * P::kChunk + ((s + 1) & 3) * 4);
      each<MI>([&](auto ic) {
        constexpr int i = decltype(ic)::value, w0 = i * NI / MI, w1 = (i + 1) * NI / MI;
        v8i hi = frag(xf[i]), lo = hi;
        if constexpr (SPLIT) {
          hi = large_codes(hi);
          lo = lo ^ hi;
        }
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(wf[j]), hi, acc[i][j], 4, A_FP4 ? 4 : 0, 0,
                                                                       sw[j], 0, sx[i]);
          if constexpr (SPLIT)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(wf[j]), lo, acc[i][j], 4, 0, 0, sw[j], 0,
                                                                         sx[i]);
        }
        read_x(slot, at, i);
#pragma unroll
        for (int j = w0; j < w1; ++j) read_w(slot, at, j);
        __builtin_amdgcn_sched_group_barrier(0x008, SPLIT ? 2 * NI : NI, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, (A_FP4 ? 2 : 3) + 2 * (w1 - w0), 0);
      });
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        wf[i] = wnext[i];
        sw[i] = swnext[i];
      }
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

template <bool A_FP4, bool SPLIT>
void launch_rule(const MxProduct& p, int num_cu, hipStream_t stream) {
  // tiles if the rows are spread evenly over as many groups as there can be
  const int64_t active = p.offsets ? (p.groups < p.m ? p.groups : p.m) : 1;
  const int64_t rows = (p.m + active - 1) / active;
  auto tiles = [&](int64_t bm, int64_t bn) {
    return (p.offsets ? p.m / bm + p.groups : (p.m + bm - 1) / bm) * ((p.n + bn - 1) / bn);
  };
  auto even = [&](int64_t bm, int64_t bn) { return active * ((rows + bm - 1) / bm) * ((p.n + bn - 1) / bn); };
  if constexpr (A_FP4) {
    if (rows > 128 && even(256, 256) >= num_cu)
      return launch_tiles<A_FP4, SPLIT, 8, 4, 2, 4, 4>(p, tiles(256, 256), num_cu, stream);
  }
  if (rows > 64 && even(128, 256) >= num_cu)
    launch_tiles<A_FP4, SPLIT, 4, 4, 2, 4, 4>(p, tiles(128, 256), num_cu, stream);
  else if (rows > 64 && even(128, 128) >= num_cu)
    launch_tiles<A_FP4, SPLIT, 4, 2, 2, 4, 4>(p, tiles(128, 128), num_cu, stream);
  else
    launch_tiles<A_FP4, SPLIT, 2, 2, 2, 2, 4>(p, tiles(64, 64), num_cu, stream);
}

}  // namespace

hipError_t launch_mx_product(const MxProduct& p, int num_cu, hipStream_t stream) {
  if (p.a_fp4)
    launch_rule<true, false>(p, num_cu, stream);
  else if (p.out_f32)
    launch_rule<false, true>(p, num_cu, stream);
  else
    launch_rule<false, false>(p, num_cu, stream);
  return hipGetLastError();
}

}  // namespace fp8blk
