// Gradients of the experts' products in bf16 (gfx950), grouped:
//   dgrad: dx[t][j] = sum_n dy[t][n] W[g][n][j]   (rows t of group g)
//   wgrad: dw[g][i][j] = sum_t dy[t][i] x[row(t)][j]
// by v_mfma_f32_16x16x32_bf16: lane l holds row (column) l % 16 of an operand
// and the 8 summed places at 8 (l / 16).
//
// Of the operands only dgrad's dy has its summed places side by side in
// memory.  The others lie in LDS as they do in memory, summed places apart,
// and are read by ds_read_b64_tr_b16, which turns 4 places by 16 columns of
// 16 lanes: lane i of the 16 gives the address of 4 columns 4 (i % 4) of place
// i / 4 and gets the 4 places of column i.
//
// Tiles.  A workgroup of WM x WN waves makes BM x BN outputs, a wave MI x NI
// tiles of 16 x 16.  The sum advances 64 places a stage (two steps of 32)
// through two stages in LDS that loads fill straight from memory.
// A row of dgrad's dy is 128 bytes of a stage, its 16-byte piece c at c ^
// turn(r); a place of the other operands is a row of 2 BM or 2 BN bytes, its
// 32-byte piece c at c ^ spread(place), so that reads of 4 places by two lane
// groups fall on all banks (3.4 cycles a read; 16 without).
//
// The loop is that of the MXFP4 products: while a step's matrix products run,
// the operands of the next step are read (by eight waves, which have registers
// for one set of rows, each row's into those that its products have just left),
// in the middle of a stage one barrier frees it, and stages go on from tile to
// tile of a workgroup.  (Wgrad reads the offsets of a new tile's group from
// memory there, dgrad those of the group it has found in LDS; either waits for
// what is on its way.)
//
// The first operand of a product is the one whose columns are those of the
// result, so that a lane's four results are consecutive in memory.
//
// Places past the sum's end are zeros on both sides: loads past a buffer's
// length give zeros, and the lengths end where the group (or n) does.
#include "groups.h"
#include "launch.h"

namespace fp8blk {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));

constexpr int kPlaces = 64;   // of a stage
constexpr int kSlots = 2;     // stages in LDS
constexpr uint32_t kNowhere = 0xFFFFFFF0u;

template <int MI, int NI, int WM, int WN>
struct Plan {
  static constexpr int kWaves = WM * WN, BM = 16 * MI * WM, BN = 16 * NI * WN;
  static constexpr int kR = BM * kPlaces * 2, kStage = kR + BN * kPlaces * 2;
  static constexpr int kRLoads = kR / 1024 / kWaves, kLoads = kStage / 1024 / kWaves;   // of a wave and stage
  static constexpr int kCLoads = kLoads - kRLoads;
  static constexpr int kIndex = kSlots * kStage, kBytes = kIndex + 2 * kPlaces * 4;
  static constexpr int kStores = MI * NI / 2;       // of a wave and whole tile, bf16 (floats: twice that, half of them waited for)
  static constexpr bool kTwice = kWaves <= 4;       // registers for two sets of rows
  static constexpr bool kInAcc = kTwice;            // results in accumulation registers
  static_assert(kR % (1024 * kWaves) == 0 && kStage % (1024 * kWaves) == 0, "shares of the loads");
  static_assert(BM >= 128 && BN >= 128 && kWaves * 8 % 16 == 0, "pieces of a place, rows of a lane's loads");
  static_assert(kLoads + kStores < 64, "vmcnt");
  static_assert(kBytes + kMaxGroups * 4 <= 160 * 1024, "LDS");
};

__device__ __forceinline__ int turn(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int spread(int place) { return (place & 3) | ((place >> 1) & 4); }

__device__ __forceinline__ u32x2 read_turned(uint32_t lds) {
  typedef __attribute__((address_space(3))) v4s lds_v4s;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(uintptr_t)lds));
}

__device__ __forceinline__ u32x4 uniform(u32x4 v) {
  return (u32x4){(uint32_t)__builtin_amdgcn_readfirstlane((int)v.x), (uint32_t)__builtin_amdgcn_readfirstlane((int)v.y),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)v.z), (uint32_t)__builtin_amdgcn_readfirstlane((int)v.w)};
}

// A tile of the result: its first row and column, the rows and columns that are
// there, the places of its sum and (wgrad) the first of them.
struct Work {
  int group, rows, cols, places;
  int64_t row0, col0, first;
};

template <bool WGRAD, bool GATHER, bool F32, int MI, int NI, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void expert_grad_kernel(GroupedGrad a, TileGrid grid) {
  using P = Plan<MI, NI, WM, WN>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[P::kBytes];
  __shared__ int upto[WGRAD ? 1 : kMaxGroups];
  const int t = (int)threadIdx.x, lane = t & 63, r16 = lane & 15, kg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6), wm = wave / WN, wn = wave % WN;
  const int64_t N = a.n, K = a.k;
  const uint32_t lds0 = lds_address(smem);
  int tiles = grid.groups * grid.tiles_n * grid.band;
  if constexpr (!WGRAD) tiles = __builtin_amdgcn_readfirstlane(count_tiles<P::BM, 64 * P::kWaves>(grid, upto));
  // Where a lane's operands lie in a stage.  Turned ones: piece c of place p
  // at p * row + ((c ^ spread(p)) * 32), of which a lane takes 8 bytes; c's bits
  // above the wave's first piece are added by exclusive or.
  const int place = 8 * kg + (r16 >> 2);
  const uint32_t turned = (uint32_t)(spread(place) * 32 + (r16 & 3) * 8);
  const uint32_t cb = lds0 + (uint32_t)(P::kR + place * (P::BN * 2)) + (turned ^ (uint32_t)(wn * NI * 32));
  const uint32_t rb = WGRAD ? lds0 + (uint32_t)(place * (P::BM * 2)) + (turned ^ (uint32_t)(wm * MI * 32))
                            : (uint32_t)((wm * MI * 16 + r16) * 128 + (kg ^ turn(r16)) * 16);
  auto work_of = [&](int id) {
    Work w;
    if constexpr (WGRAD) {
      // band row tiles of a group by tiles_n column tiles, in bands of 8 row tiles
      const int per = grid.band * grid.tiles_n, q = id / per, r = id - q * per;
      int lo, hi;
      rows_of_group(a.offsets, q, (int)a.total_m, &lo, &hi);
      lo = __builtin_amdgcn_readfirstlane(lo);
      hi = __builtin_amdgcn_readfirstlane(hi);
      const int band = grid.band < 8 ? grid.band : 8;
      const int b = r / (band * grid.tiles_n), rr = r - b * (band * grid.tiles_n);
      const int here = grid.band - b * band < band ? grid.band - b * band : band;
      w.group = __builtin_amdgcn_readfirstlane(q);
      w.row0 = (int64_t)__builtin_amdgcn_readfirstlane(b * band + rr % here) * P::BM;
      w.col0 = (int64_t)__builtin_amdgcn_readfirstlane(rr / here) * P::BN;
      w.rows = N - w.row0 < P::BM ? (int)(N - w.row0) : P::BM;
      w.first = lo;
      w.places = hi - lo;
    } else {
      const Tile tile = tile_at<P::BM>(grid, upto, id);
      w.group = tile.group;
      w.row0 = tile.row0;
      w.rows = tile.rows;
      w.col0 = (int64_t)tile.col * P::BN;
      w.first = 0;
      w.places = (int)N;
    }
    w.cols = K - w.col0 < P::BN ? (int)(K - w.col0) : P::BN;
    return w;
  };
  auto stages_of = [&](const Work& w) { return stages_in(w.places, kPlaces); };

  // The stages to load, from tile to tile; behind the last they are of nothing.
  constexpr int kCRow = P::BN / 8, kRRow = P::BM / 8;     // 16-byte pieces of a place
  int d_it = -1, d_stage = 0, d_stages = 0, d_left = 0;
  bool d_over = false;
  Work d;
  u32x4 r_from = buffer_of(a.dy, 0), c_from = r_from;
  uint32_t past = 0;
  uint32_t off[P::kLoads];
  int index[P::kCLoads];
  auto place_of = [&](int j) { return (j * P::kWaves + wave) * (64 / kCRow) + lane / kCRow; };   // of load j of c
  auto next_stage = [&]() {
    if (d_over) return;
    if (++d_stage >= d_stages) {
      d_stage = 0;
      for (d_stages = 0; d_stages == 0;) {
        const int id = tile_of_turn(++d_it);
        if (id >= tiles) break;
        d = work_of(id);
        d_stages = stages_of(d);
      }
      if (d_stages == 0) {
        d_over = true;
        d_left = 0;
        r_from.z = c_from.z = 0;
        return;
      }
      // This wave's loads: blocks wave, wave + kWaves, ... of 1 KiB.  Offsets of
      // turned operands are from the stage's first place (gathered x: from x
      // itself, without the row).
#pragma unroll
      for (int j = 0; j < P::kLoads; ++j) {
        if (j < P::kRLoads && !WGRAD) {
          const int r = (j * P::kWaves + wave) * 8 + lane / 8;
          off[j] = (uint32_t)r * (uint32_t)(N * 2) + (uint32_t)(((lane % 8) ^ turn(r)) * 16);
        } else if (j < P::kRLoads) {
          const int p = (j * P::kWaves + wave) * (64 / kRRow) + lane / kRRow;
          off[j] = (uint32_t)p * (uint32_t)(N * 2) + (uint32_t)(d.row0 * 2) +
                   (uint32_t)(((lane % kRRow) ^ (spread(p) * 2)) * 16);
        } else {
          const int p = place_of(j - P::kRLoads);
          off[j] = (GATHER ? 0u : (uint32_t)p * (uint32_t)(K * 2)) + (uint32_t)(d.col0 * 2) +
                   (uint32_t)(((lane % kCRow) ^ (spread(p) * 2)) * 16);
        }
      }
      if (!WGRAD) r_from = buffer_of(a.dy + d.row0 * N, (uint32_t)d.rows * (uint32_t)(N * 2));
      if (GATHER) c_from = buffer_of(a.x, (uint32_t)(a.x_rows * K * 2));
    }
    d_left = d.places - d_stage * kPlaces;
    const uint32_t here = (uint32_t)(d_left < kPlaces ? d_left : kPlaces);
    const int64_t p0 = d.first + (int64_t)d_stage * kPlaces;
    if (WGRAD) r_from = buffer_of(a.dy + p0 * N, here * (uint32_t)(N * 2));
    if (!GATHER) c_from = buffer_of(WGRAD ? a.x + p0 * K : a.w + ((int64_t)d.group * N + p0) * K, here * (uint32_t)(K * 2));
    // (dgrad's dy: a lane's piece is the same in all loads)
    past = !WGRAD && ((lane % 8) ^ turn(wave * 8 + lane / 8)) * 8 >= d_left ? kNowhere : 0u;
  };
  auto load = [&](uint32_t slot, int from, int end) {
    // (uniform, but the compiler does not see it)
    const u32x4 rs = uniform(r_from), cs = uniform(c_from);
#pragma unroll
    for (int j = from; j < end; ++j) {
      const uint32_t to = lds0 + slot + (uint32_t)(j * P::kWaves + wave) * 1024;
      if (j < P::kRLoads) {
        lds_load16(rs, (WGRAD ? off[j] : off[j] + (uint32_t)d_stage * 128) | past, to);
      } else if constexpr (GATHER) {
        const int at = clamp_to(index[j - P::kRLoads], 0, (int)a.x_rows - 1);
        lds_load16(cs, place_of(j - P::kRLoads) < d_left ? (uint32_t)at * (uint32_t)(K * 2) + off[j] : kNowhere, to);
      } else {
        lds_load16(cs, off[j], to);
      }
    }
  };
  // The indices of gathered x go ahead by a stage, into two places in turn.
  int i_it = -1, i_stage = 0, i_stages = 0;
  bool i_over = false;
  Work x;
  auto load_index = [&](uint32_t to) {
    if constexpr (GATHER) {
      if (i_over) return;
      if (++i_stage >= i_stages) {
        i_stage = 0;
        for (i_stages = 0; i_stages == 0;) {
          const int id = tile_of_turn(++i_it);
          if (id >= tiles) break;
          x = work_of(id);
          i_stages = stages_of(x);
        }
        if (i_stages == 0) {
          i_over = true;
          return;
        }
      }
      const int left = x.places - i_stage * kPlaces;
      if (wave != 0) return;
      const u32x4 from = buffer_of(a.row_index + x.first + (int64_t)i_stage * kPlaces,
                                   (uint32_t)(left < kPlaces ? left : kPlaces) * 4);
      lds_load4(from, (uint32_t)lane * 4, lds0 + P::kIndex + to);
    }
  };
  auto read_index = [&](uint32_t at, int from, int end) {      // for loads from .. end - 1
#pragma unroll
    for (int j = from; GATHER && j < end; ++j)
      if (j >= P::kRLoads && j < P::kLoads)
        index[j - P::kRLoads] = *reinterpret_cast<const int*>(smem + P::kIndex + at + place_of(j - P::kRLoads) * 4);
  };

  int it = 0, id = tile_of_turn(0);
  if (id >= tiles) return;
  constexpr uint32_t kTurn = kPlaces * 4;       // between the places of indices
  uint32_t index_at = 0;                        // of the next stage to load
  load_index(0);
  load_index(kTurn);
  if constexpr (GATHER) {
    wait_loads<0>();
    barrier();
  }
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    next_stage();
    read_index((uint32_t)i * kTurn, 0, P::kLoads);
    load((uint32_t)(i * P::kStage), 0, P::kLoads);
  }
  if constexpr (GATHER) {
    wait_lds_reads();
    barrier();
    load_index(0);
  }

  v4f acc[MI][NI];
  u32x4 r0[MI], r1[P::kTwice ? MI : 1], c0[NI], c1[NI];
  auto read_r = [&](u32x4& r, uint32_t slot, int step, int i) {
    if constexpr (WGRAD) {
      const uint32_t at = (rb ^ (uint32_t)(i * 32)) + slot + (uint32_t)(step * 32 * P::BM * 2);
      const u32x2 u = read_turned(at), v = read_turned(at + 4 * P::BM * 2);
      r = (u32x4){u.x, u.y, v.x, v.y};
    } else {
      r = *reinterpret_cast<const u32x4*>(smem + (rb ^ (uint32_t)(step * 64)) + slot + i * 2048);
    }
  };
  auto read_c = [&](u32x4& c, uint32_t slot, int step, int j) {
    const uint32_t at = (cb ^ (uint32_t)(j * 32)) + slot + (uint32_t)(step * 32 * P::BN * 2);
    const u32x2 u = read_turned(at), v = read_turned(at + 4 * P::BN * 2);
    c = (u32x4){u.x, u.y, v.x, v.y};
  };
  // (the compiler would move products past the barriers and the branches)
  auto pin_row = [&](int i) {
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      if constexpr (P::kInAcc) asm volatile("" : "+a"(acc[i][j])); else asm volatile("" : "+v"(acc[i][j]));
    }
  };
  auto pin = [&]() {
#pragma unroll
    for (int i = 0; i < MI; ++i) pin_row(i);
  };
  // The products of a step, with the next one's reads beside the first of them
  // and (LOAD) the loads of a stage beside all.
  constexpr int kProducts = MI * NI, kSpan = MI > 1 ? kProducts - NI : kProducts;
  auto part = [](int q, int span, int all) { return q < span ? q * all / span : all; };
  auto step = [&](auto load_too, u32x4* r, const u32x4* c, u32x4* rnext, u32x4* cnext, uint32_t slot, int next,
                  uint32_t freed, uint32_t indices) {
    each<kProducts>([&](auto qc) {
      constexpr int q = decltype(qc)::value, i = q / NI, j = q % NI;
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, c[j]), __builtin_bit_cast(v8bf, r[i]),
                                                          acc[i][j], 0, 0, 0);
      if constexpr (P::kTwice) {
        constexpr int kReads = MI + NI;       // row 0, all columns, the other rows
#pragma unroll
        for (int e = part(q, kSpan, kReads); e < part(q + 1, kSpan, kReads); ++e) {
          if (e == 0 || e > NI)
            read_r(rnext[e ? e - NI : 0], slot, next, e ? e - NI : 0);
          else
            read_c(cnext[e - 1], slot, next, e - 1);
        }
      } else {
#pragma unroll
        for (int e = part(q, kSpan, NI); e < part(q + 1, kSpan, NI); ++e) read_c(cnext[e], slot, next, e);
        if (j == NI - 1) read_r(r[i], slot, next, i);
      }
      if constexpr (decltype(load_too)::value) {
        constexpr int from = part(q, kProducts, P::kLoads), end = part(q + 1, kProducts, P::kLoads);
        read_index(indices, q ? from + 2 : 0, end + 2);       // ahead by two loads
        load(freed, from, end);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    pin();
  };

  wait_loads<0>();
  barrier();
#pragma unroll
  for (int i = 0; i < MI; ++i) read_r(r0[i], 0, 0, i);
#pragma unroll
  for (int j = 0; j < NI; ++j) read_c(c0[j], 0, 0, j);

  uint32_t slot = 0;
  bool stored = false;       // kStores stores or more are behind the last loads
  for (;;) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
    pin();
    // Waves whose rows or columns are all behind the tile's last only load.
    // (Of eight, waves 0 to 3, on a SIMD each, have the first rows.)
    const Work here = d_it == it ? d : work_of(id);
    const bool busy = wm * MI * 16 < here.rows && wn * NI * 16 < here.cols;
    const int stages = stages_of(here);
    for (int s = 0; s < stages; ++s) {
      u32x4* const rs = P::kTwice ? r1 : r0;
      if (busy) step(std::false_type{}, r0, c0, rs, c1, slot, 1, 0u, 0u);
      wait_lds_reads();
      if (stored) wait_loads<P::kStores>(); else wait_loads<0>();
      stored = false;
      barrier();
      const uint32_t freed = slot;
      slot ^= (uint32_t)P::kStage;
      next_stage();
      const uint32_t indices = index_at;
      index_at ^= kTurn;
      load_index(index_at);
      // (the next stage may be of another tile)
      if (busy || s + 1 == stages) {
        step(std::true_type{}, rs, c1, r0, c0, slot, 0, freed, indices);
      } else {
        read_index(indices, 0, P::kLoads);
        load(freed, 0, P::kLoads);
      }
    }

    // Lane l holds row l % 16 and columns 4 (l / 16) .. + 3 of each 16 x 16.  For
    // bf16, lane groups 0 and 1, 2 and 3 exchange results of two tiles: eight
    // consecutive columns for each, 64 bytes of a row for the four.
    const int row = wm * MI * 16, col = wn * NI * 16;
    const int64_t first = (WGRAD ? (int64_t)here.group * N + here.row0 : here.row0) * K + here.col0 + row * K + col;
    const int lane_col = F32 ? kg * 4 : (kg & 1) * 16 + (kg >> 1) * 8;
    const int rows = here.rows - row - r16, cols = here.cols - col - lane_col;     // from the lane's first on
    const uint32_t lane_at = ((uint32_t)r16 * (uint32_t)K + (uint32_t)lane_col) * (F32 ? 4u : 2u);
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        pin_row(i);
        uint8_t* const out = reinterpret_cast<uint8_t*>(a.out) + (first + (int64_t)i * 16 * K) * 4;
#pragma unroll
        for (int j = 0; j < NI; ++j)
          if (i * 16 < rows && j * 16 < cols) *reinterpret_cast<v4f*>(out + j * 64 + lane_at) = acc[i][j];
      }
    } else {
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        pin_row(i);
        uint8_t* const out = reinterpret_cast<uint8_t*>(a.out) + (first + (int64_t)i * 16 * K) * 2;
#pragma unroll
        for (int j = 0; j < NI; j += 2) {
          const v4f u = acc[i][j], v = acc[i][j + 1];
          const auto lo = __builtin_amdgcn_permlane16_swap(pack_bf16x2(u[0], u[1]), pack_bf16x2(v[0], v[1]), false, false);
          const auto hi = __builtin_amdgcn_permlane16_swap(pack_bf16x2(u[2], u[3]), pack_bf16x2(v[2], v[3]), false, false);
          if (i * 16 < rows && j * 16 < cols)
            *reinterpret_cast<u32x4*>(out + j * 32 + lane_at) = (u32x4){lo[0], hi[0], lo[1], hi[1]};
        }
      }
    }
    stored = stored || (here.rows == P::BM && here.cols == P::BN);
    id = tile_of_turn(++it);
    if (id >= tiles) break;
  }
  wait_loads<0>();   // (of nothing)
}

template <bool WGRAD, bool GATHER, int MI, int NI, int WM, int WN>
void launch_tiles(const GroupedGrad& a, int64_t row_tiles, int num_cu, hipStream_t stream) {
  using P = Plan<MI, NI, WM, WN>;
  const int64_t tiles_n = (a.k + P::BN - 1) / P::BN;
  TileGrid g{WGRAD ? nullptr : a.offsets, a.groups, (int)a.total_m, (int)tiles_n,
             WGRAD ? (int)((a.n + P::BM - 1) / P::BM) : 8};
  const int64_t tiles = WGRAD ? (int64_t)a.groups * g.band * tiles_n : row_tiles * tiles_n;
  const int64_t per_cu = 160 * 1024 / (P::kBytes + (WGRAD ? 4 : kMaxGroups * 4));
  const int64_t most = (num_cu >= 8 ? num_cu / 8 * 8 : 8) * per_cu;
  const int64_t wgs = tiles < most ? (tiles + 7) / 8 * 8 : most;
  // (a kernel for either type: one for both has fewer registers to spare, 1250
  // us for 1150 of gathered bf16 gradients of weights)
  if (a.out_f32)
    hipLaunchKernelGGL((expert_grad_kernel<WGRAD, GATHER, true, MI, NI, WM, WN>), dim3((unsigned)wgs),
                       dim3(64 * WM * WN), 0, stream, a, g);
  else
    hipLaunchKernelGGL((expert_grad_kernel<WGRAD, GATHER, false, MI, NI, WM, WN>), dim3((unsigned)wgs),
                       dim3(64 * WM * WN), 0, stream, a, g);
}

}  // namespace

// Tiles of 256 x 256 by eight waves from one to a CU on, for more than 128 rows
// a group, else of 128 x 128 by four (us: 16384 rows on 32 experts of 4096 x
// 7168, bf16, 1017 and 1178; 4096 rows on 32 of 2048 x 4096, float, 171 and 148).
hipError_t launch_grouped_dgrad(const GroupedGrad& a, int num_cu, hipStream_t stream) {
  const int64_t active = a.groups < a.total_m ? a.groups : a.total_m;
  const int64_t rows = (a.total_m + active - 1) / active;
  const int64_t even = active * ((rows + 255) / 256) * ((a.k + 255) / 256);
  if (rows > 128 && even >= num_cu)
    launch_tiles<false, false, 8, 4, 2, 4>(a, a.total_m / 256 + a.groups, num_cu, stream);
  else
    launch_tiles<false, false, 4, 4, 2, 2>(a, a.total_m / 128 + a.groups, num_cu, stream);
  return hipGetLastError();
}

// The same tiles, the large ones where they fill three quarters of the CUs'
// turns (us, gathered, bf16: 16384 rows on 32 experts of 4096 x 7168: 1130 and
// 1490; 921 rows on 8 of 1000 x 1416, 192 tiles: 16 and 17; on 11, 264 tiles: 20
// and 17).
hipError_t launch_grouped_wgrad(const GroupedGrad& a, int num_cu, hipStream_t stream) {
  const int64_t large = a.groups * ((a.n + 255) / 256) * ((a.k + 255) / 256), turns = (large + num_cu - 1) / num_cu;
  const bool big = 4 * large >= 3 * turns * num_cu;
  if (a.row_index) {
    if (big) launch_tiles<true, true, 8, 4, 2, 4>(a, 0, num_cu, stream);
    else launch_tiles<true, true, 4, 4, 2, 2>(a, 0, num_cu, stream);
  } else {
    if (big) launch_tiles<true, false, 8, 4, 2, 4>(a, 0, num_cu, stream);
    else launch_tiles<true, false, 4, 4, 2, 2>(a, 0, num_cu, stream);
  }
  return hipGetLastError();
}

}  // namespace fp8blk
