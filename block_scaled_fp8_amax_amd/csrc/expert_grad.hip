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
// through a ring of SLOTS stages in LDS that loads fill straight from memory.
// A row of dgrad's dy is 128 bytes of a stage, its 16-byte piece c at c ^
// turn(r); a place of the other operands is a row of 2 BM or 2 BN bytes, its
// 32-byte piece c at c ^ spread(place), so that reads of 4 places by two lane
// groups fall on all banks (3.4 cycles a read; 16 without).
//
// The loop is that of the MXFP4 products: while a step's matrix products run,
// the operands of the next step are read, each into the registers that its
// products have just left; in the middle of a stage one barrier frees it.
//
// The first operand of a product is the one whose columns are those of the
// result, so that a lane's four results are consecutive in memory.
//
// Places past the sum's end are zeros on both sides: loads past a buffer's
// length give zeros, and the lengths end where the group (or n) does.
#include <type_traits>

#include "groups.h"
#include "launch.h"

namespace fp8blk {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));

// f(0), ..., f(N - 1) with compile-time arguments.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    each<N, I + 1>(f);
  }
}

constexpr int kPlaces = 64;   // of a stage

template <int MI, int NI, int WM, int WN, int SLOTS>
struct Plan {
  static constexpr int kWaves = WM * WN, BM = 16 * MI * WM, BN = 16 * NI * WN;
  static constexpr int kR = BM * kPlaces * 2, kStage = kR + BN * kPlaces * 2;
  static constexpr int kRLoads = kR / 1024 / kWaves, kLoads = kStage / 1024 / kWaves;   // of a wave and stage
  static constexpr int kIndex = SLOTS * kStage, kBytes = kIndex + 2 * kPlaces * 4;
  static_assert(kR % (1024 * kWaves) == 0 && kStage % (1024 * kWaves) == 0, "shares of the loads");
  static_assert(BM >= 128 && BN >= 128, "pieces of a place");
  static_assert(kBytes + kMaxGroups * 4 <= 160 * 1024, "LDS");
};

__device__ __forceinline__ int turn(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int spread(int place) { return (place & 3) | ((place >> 1) & 4); }

__device__ __forceinline__ u32x2 read_turned(uint32_t lds) {
  typedef __attribute__((address_space(3))) v4s lds_v4s;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(uintptr_t)lds));
}

template <bool WGRAD, bool GATHER, int MI, int NI, int WM, int WN, int SLOTS>
__global__ __launch_bounds__(64 * WM * WN) void expert_grad_kernel(GroupedGrad a, TileGrid grid) {
  using P = Plan<MI, NI, WM, WN, SLOTS>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[P::kBytes];
  __shared__ int upto[WGRAD ? 1 : kMaxGroups];
  const int t = (int)threadIdx.x, lane = t & 63, r16 = lane & 15, kg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6), wm = wave % WM, wn = wave / WM;
  const int64_t N = a.n, K = a.k;
  const uint32_t lds0 = lds_address(smem);
  const int tiles = WGRAD ? grid.groups * grid.tiles_n * grid.band : count_tiles<P::BM, 64 * P::kWaves>(grid, upto);
  // Where a lane's operands lie in a stage.  Turned ones: piece c of place p
  // at p * row + ((c ^ spread(p)) * 32), of which a lane takes 8 bytes; c's bits
  // above the wave's first piece are added by exclusive or.
  const int place = 8 * kg + (r16 >> 2);
  const uint32_t turned = (uint32_t)(spread(place) * 32 + (r16 & 3) * 8);
  const uint32_t cb = lds0 + (uint32_t)(P::kR + place * (P::BN * 2)) + (turned ^ (uint32_t)(wn * NI * 32));
  const uint32_t rb = WGRAD ? lds0 + (uint32_t)(place * (P::BM * 2)) + (turned ^ (uint32_t)(wm * MI * 32))
                            : (uint32_t)((wm * MI * 16 + r16) * 128 + (kg ^ turn(r16)) * 16);

  for (int it = 0;; ++it) {
    const int id = tile_of_turn(it, tiles);
    if (id >= tiles) break;
    int group, places, cols, rows;     // of the tile: columns and rows of the result that are there
    int64_t row0, col0, first;         // first: the group's first row
    if constexpr (WGRAD) {
      // band row tiles of a group by tiles_n column tiles, in bands of 8 row tiles
      const int per = grid.band * grid.tiles_n, q = id / per, r = id - q * per;
      group = group_at(q, grid.groups);
      int lo, hi;
      rows_of_group(a.offsets, group, (int)a.total_m, &lo, &hi);
      group = __builtin_amdgcn_readfirstlane(group);
      lo = __builtin_amdgcn_readfirstlane(lo);
      hi = __builtin_amdgcn_readfirstlane(hi);
      const int band = grid.band < 8 ? grid.band : 8;
      const int b = r / (band * grid.tiles_n), rr = r - b * (band * grid.tiles_n);
      const int here = grid.band - b * band < band ? grid.band - b * band : band;
      row0 = (int64_t)(b * band + rr % here) * P::BM;
      col0 = (int64_t)(rr / here) * P::BN;
      rows = N - row0 < P::BM ? (int)(N - row0) : P::BM;
      first = lo;
      places = hi - lo;
    } else {
      const Tile tile = tile_at<P::BM>(grid, upto, id);
      group = tile.group;
      row0 = tile.row0;
      rows = tile.rows;
      col0 = (int64_t)tile.col * P::BN;
      first = 0;
      places = (int)N;
    }
    cols = K - col0 < P::BN ? (int)(K - col0) : P::BN;
    const int stages = (places + kPlaces - 1) / kPlaces;

    // This wave's loads of a stage: blocks wave, wave + kWaves, ... of 1 KiB.
    // Offsets of turned operands are from the stage's first place (gathered x:
    // from x itself, without the row).
    constexpr int kCRow = P::BN / 8, kRRow = P::BM / 8;     // 16-byte pieces of a place
    uint32_t off[P::kLoads];
    int cplace[P::kLoads - P::kRLoads];
#pragma unroll
    for (int j = 0; j < P::kLoads; ++j) {
      const int blk = (j < P::kRLoads ? j : j - P::kRLoads) * P::kWaves + wave;
      if (j < P::kRLoads && !WGRAD) {
        const int r = blk * 8 + lane / 8;
        off[j] = (uint32_t)(r < rows ? r : rows - 1) * (uint32_t)(N * 2) + (uint32_t)(((lane % 8) ^ turn(r)) * 16);
      } else if (j < P::kRLoads) {
        const int p = blk * (64 / kRRow) + lane / kRRow;
        off[j] = (uint32_t)p * (uint32_t)(N * 2) + (uint32_t)(row0 * 2) + (uint32_t)(((lane % kRRow) ^ (spread(p) * 2)) * 16);
      } else {
        const int p = blk * (64 / kCRow) + lane / kCRow;
        cplace[j - P::kRLoads] = p;
        off[j] = (GATHER ? 0u : (uint32_t)p * (uint32_t)(K * 2)) + (uint32_t)(col0 * 2) +
                 (uint32_t)(((lane % kCRow) ^ (spread(p) * 2)) * 16);
      }
    }
    // Pieces and places past the end are read at this offset, as zeros.
    constexpr uint32_t kNowhere = 0xFFFFFFF0u;
    const int piece = (lane % 8) ^ turn(wave * 8 + lane / 8);      // of dgrad's dy, the same in all loads
    static_assert(P::kWaves * 8 % 16 == 0, "rows of a lane's loads");
    const u32x4 dy_rows = buffer_of(a.dy + row0 * N, kNowhere);
    const u32x4 x_all = buffer_of(a.x, GATHER ? (uint32_t)(a.x_rows * K * 2) : 0u);
    auto load_index = [&](int s) {
      if (!GATHER || wave != 0) return;
      const int64_t at = first + (int64_t)s * kPlaces + lane;
      const uint32_t last = (uint32_t)(a.total_m - 1);
      lds_load4(a.row_index, (at < a.total_m ? (uint32_t)at : last) * 4, lds0 + P::kIndex + (uint32_t)(s & 1) * (kPlaces * 4));
    };
    int index[P::kLoads - P::kRLoads];
    auto read_index = [&](int s) {
      if constexpr (GATHER) {
#pragma unroll
        for (int j = 0; j < P::kLoads - P::kRLoads; ++j)
          index[j] = *reinterpret_cast<const int*>(smem + P::kIndex + (s & 1) * (kPlaces * 4) + cplace[j] * 4);
      }
    };
    auto load_stage = [&](int s, uint32_t slot) {
      const int left = places - s * kPlaces;
      const uint32_t here = (uint32_t)(left < kPlaces ? left : kPlaces);
      const int64_t p0 = first + (int64_t)s * kPlaces;
      const u32x4 r = WGRAD ? buffer_of(a.dy + p0 * N, here * (uint32_t)(N * 2)) : dy_rows;
      const u32x4 c = GATHER ? x_all
                             : buffer_of(WGRAD ? a.x + p0 * K : a.w + ((int64_t)group * N + p0) * K, here * (uint32_t)(K * 2));
      const uint32_t past = !WGRAD && piece * 8 >= left ? kNowhere : 0u;
#pragma unroll
      for (int j = 0; j < P::kLoads; ++j) {
        const uint32_t to = lds0 + slot + (uint32_t)(j * P::kWaves + wave) * 1024;
        if (j < P::kRLoads) {
          lds_load16(r, (WGRAD ? off[j] : off[j] + (uint32_t)s * 128) | past, to);
        } else if constexpr (GATHER) {
          const int at = clamp_to(index[j - P::kRLoads], 0, (int)a.x_rows - 1);
          const uint32_t from = (uint32_t)at * (uint32_t)(K * 2) + off[j];
          lds_load16(c, cplace[j - P::kRLoads] < left ? from : kNowhere, to);
        } else {
          lds_load16(c, off[j], to);
        }
      }
    };

    v4f acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
    u32x4 rf[MI], c0[NI], c1[NI];
    auto read_r = [&](uint32_t slot, int step, int i) {
      if constexpr (WGRAD) {
        const uint32_t at = (rb ^ (uint32_t)(i * 32)) + slot + (uint32_t)(step * 32 * P::BM * 2);
        const u32x2 u = read_turned(at), v = read_turned(at + 4 * P::BM * 2);
        rf[i] = (u32x4){u.x, u.y, v.x, v.y};
      } else {
        rf[i] = *reinterpret_cast<const u32x4*>(smem + (rb ^ (uint32_t)(step * 64)) + slot + i * 2048);
      }
    };
    auto read_c = [&](u32x4& c, uint32_t slot, int step, int j) {
      const uint32_t at = (cb ^ (uint32_t)(j * 32)) + slot + (uint32_t)(step * 32 * P::BN * 2);
      const u32x2 u = read_turned(at), v = read_turned(at + 4 * P::BN * 2);
      c = (u32x4){u.x, u.y, v.x, v.y};
    };
    auto multiply = [&](int i, const u32x4* c) {
#pragma unroll
      for (int j = 0; j < NI; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, c[j]), __builtin_bit_cast(v8bf, rf[i]),
                                                            acc[i][j], 0, 0, 0);
    };

    if (stages > 0) {
      // the first stages, and the indices of the two after them
      if constexpr (GATHER) {
#pragma unroll
        for (int i = 0; i < SLOTS; i += 2) {
          load_index(i);
          load_index(i + 1);
          wait_loads<0>();
          barrier();
#pragma unroll
          for (int h = i; h < SLOTS && h < i + 2; ++h) {
            read_index(h);
            if (h < stages) load_stage(h, (uint32_t)(h * P::kStage));
          }
          wait_lds_reads();
          barrier();
        }
        load_index(SLOTS);
        load_index(SLOTS + 1);
        wait_loads<0>();
      } else {
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
          if (i < stages) load_stage(i, (uint32_t)(i * P::kStage));
        if (stages >= SLOTS) wait_loads<(SLOTS - 1) * P::kLoads>(); else wait_loads<0>();
      }
      barrier();
#pragma unroll
      for (int i = 0; i < MI; ++i) read_r(0, 0, i);
#pragma unroll
      for (int j = 0; j < NI; ++j) read_c(c0[j], 0, 0, j);
    }
    uint32_t slot = 0;
    for (int s = 0; s < stages; ++s) {
      constexpr int kRReads = WGRAD ? 2 : 1;
      read_index(s + SLOTS);
      each<MI>([&](auto ic) {
        constexpr int i = decltype(ic)::value, from = i * NI / MI, to = (i + 1) * NI / MI;
        multiply(i, c0);
        read_r(slot, 1, i);
#pragma unroll
        for (int j = from; j < to; ++j) read_c(c1[j], slot, 1, j);
        __builtin_amdgcn_sched_group_barrier(0x008, NI, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, kRReads + 2 * (to - from), 0);
      });
      // (the compiler would move products past the barrier and the branches)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) asm volatile("" : "+v"(acc[i][j]));
      wait_lds_reads();
      if (s + SLOTS - 1 < stages) wait_loads<(SLOTS - 2) * P::kLoads>(); else wait_loads<0>();
      barrier();
      load_index(s + SLOTS + 2);
      if (s + SLOTS < stages) load_stage(s + SLOTS, slot);
      slot = slot + P::kStage == SLOTS * P::kStage ? 0u : slot + P::kStage;
      each<MI>([&](auto ic) {
        constexpr int i = decltype(ic)::value, from = i * NI / MI, to = (i + 1) * NI / MI;
        multiply(i, c1);
        read_r(slot, 0, i);
#pragma unroll
        for (int j = from; j < to; ++j) read_c(c0[j], slot, 0, j);
        __builtin_amdgcn_sched_group_barrier(0x008, NI, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, kRReads + 2 * (to - from), 0);
      });
    }

    // lane l holds row l % 16 and columns 4 (l / 16) .. + 3 of each 16 x 16
    const int64_t out0 = WGRAD ? ((int64_t)group * N + row0) * K + col0 : row0 * K + col0;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int r = (wm * MI + i) * 16 + r16;
      if (r >= rows) continue;
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int c = (wn * NI + j) * 16 + kg * 4;
        if (c >= cols) continue;
        const int64_t at = out0 + r * K + c;
        const v4f v = acc[i][j];
        if (a.out_f32)
          *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.out) + at) = v;
        else
          *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(a.out) + at) =
              (u32x2){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      }
    }
    wait_loads<0>();
    wait_lds_reads();
    barrier();   // the next tile's loads reuse the stages
  }
}

template <bool WGRAD, bool GATHER, int MI, int NI, int WM, int WN, int SLOTS>
void launch_tiles(const GroupedGrad& a, int64_t row_tiles, int num_cu, hipStream_t stream) {
  using P = Plan<MI, NI, WM, WN, SLOTS>;
  const int64_t tiles_n = (a.k + P::BN - 1) / P::BN;
  TileGrid g{WGRAD ? nullptr : a.offsets, a.groups, (int)a.total_m, (int)tiles_n,
             WGRAD ? (int)((a.n + P::BM - 1) / P::BM) : 8};
  const int64_t tiles = WGRAD ? (int64_t)a.groups * g.band * tiles_n : row_tiles * tiles_n;
  const int64_t per_cu = 160 * 1024 / (P::kBytes + (WGRAD ? 4 : kMaxGroups * 4));
  const int64_t most = (num_cu >= 8 ? num_cu / 8 * 8 : 8) * per_cu;
  const int64_t wgs = tiles < most ? (tiles + 7) / 8 * 8 : most;
  hipLaunchKernelGGL((expert_grad_kernel<WGRAD, GATHER, MI, NI, WM, WN, SLOTS>), dim3((unsigned)wgs),
                     dim3(64 * WM * WN), 0, stream, a, g);
}

}  // namespace

hipError_t launch_grouped_dgrad(const GroupedGrad& a, int num_cu, hipStream_t stream) {
  const int64_t active = a.groups < a.total_m ? a.groups : a.total_m;
  const int64_t rows = (a.total_m + active - 1) / active;
  const int64_t even = active * ((rows + 255) / 256) * ((a.k + 255) / 256);
  if (rows > 128 && even >= num_cu)
    launch_tiles<false, false, 8, 4, 2, 4, 2>(a, a.total_m / 256 + a.groups, num_cu, stream);
  else
    launch_tiles<false, false, 4, 4, 2, 2, 2>(a, a.total_m / 128 + a.groups, num_cu, stream);
  return hipGetLastError();
}

hipError_t launch_grouped_wgrad(const GroupedGrad& a, int num_cu, hipStream_t stream) {
  const int64_t big = a.groups * ((a.n + 255) / 256) * ((a.k + 255) / 256);
  if (a.row_index) {
    if (big >= num_cu) launch_tiles<true, true, 8, 4, 2, 4, 2>(a, 0, num_cu, stream);
    else launch_tiles<true, true, 4, 4, 2, 2, 2>(a, 0, num_cu, stream);
  } else {
    if (big >= num_cu) launch_tiles<true, false, 8, 4, 2, 4, 2>(a, 0, num_cu, stream);
    else launch_tiles<true, false, 4, 4, 2, 2, 2>(a, 0, num_cu, stream);
  }
  return hipGetLastError();
}

}  // namespace fp8blk
