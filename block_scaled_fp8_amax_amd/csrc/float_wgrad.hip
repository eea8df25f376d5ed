// Float gradients of the experts' weights (gfx950), grouped:
//   dw[g][i][j] = sum_t dy[t][i] x[row(t)][j]
// the tiles, layouts and products of the other gradients, but a tile at a time:
// its results, four bytes for each, are twice what all operands are, and pass
// memory faster alone than among the next tile's loads (16384 rows on 32 experts
// of 4096 x 7168, 3.8 GB of results: 1.62 ms, 594 TFLOP/s; 1.84 the other way).
//
// While a step's matrix products run, the operands of the next step are read,
// each into the registers that its products have just left; in the middle of a
// stage one barrier frees it, and the stage after next is loaded in its place.
#include "launch.h"
#include "turned.h"

namespace fp8blk {

namespace {

template <int MI, int NI, int WM, int WN, int SLOTS>
struct Plan {
  static constexpr int kWaves = WM * WN, BM = 16 * MI * WM, BN = 16 * NI * WN;
  static constexpr int kR = BM * kPlaces * 2, kStage = kR + BN * kPlaces * 2;
  static constexpr int kRLoads = kR / 1024 / kWaves, kLoads = kStage / 1024 / kWaves;   // of a wave and stage
  static constexpr int kIndex = SLOTS * kStage, kBytes = kIndex + 2 * kPlaces * 4;
  static_assert(kR % (1024 * kWaves) == 0 && kStage % (1024 * kWaves) == 0, "shares of the loads");
  static_assert(BM >= 128 && BN >= 128, "pieces of a place");
  static_assert(kBytes <= 160 * 1024, "LDS");
};

template <bool GATHER, int MI, int NI, int WM, int WN, int SLOTS>
__global__ __launch_bounds__(64 * WM * WN) void float_wgrad_kernel(GroupedGrad a, TileGrid grid) {
  using P = Plan<MI, NI, WM, WN, SLOTS>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[P::kBytes];
  const int t = (int)threadIdx.x, lane = t & 63, r16 = lane & 15, kg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6), wm = wave % WM, wn = wave / WM;
  const int64_t N = a.n, K = a.k;
  const uint32_t lds0 = lds_address(smem);
  const int tiles = grid.groups * grid.tiles_n * grid.band;
  // Where a lane's operands lie in a stage.  Turned ones: piece c of place p
  // at p * row + ((c ^ spread(p)) * 32), of which a lane takes 8 bytes; c's bits
  // above the wave's first piece are added by exclusive or.
  const int place = 8 * kg + (r16 >> 2);
  const uint32_t turned = (uint32_t)(spread(place) * 32 + (r16 & 3) * 8);
  const uint32_t cb = lds0 + (uint32_t)(P::kR + place * (P::BN * 2)) + (turned ^ (uint32_t)(wn * NI * 32));
  const uint32_t rb = lds0 + (uint32_t)(place * (P::BM * 2)) + (turned ^ (uint32_t)(wm * MI * 32));

  for (int it = 0;; ++it) {
    const int id = tile_of_turn(it, tiles);
    if (id >= tiles) break;
    // band row tiles of a group by tiles_n column tiles, in bands of 8 row tiles
    const int per = grid.band * grid.tiles_n, q = id / per, r = id - q * per;
    const int band = grid.band < 8 ? grid.band : 8;
    const int b = r / (band * grid.tiles_n), rr = r - b * (band * grid.tiles_n);
    const int in_band = grid.band - b * band < band ? grid.band - b * band : band;
    int group = group_at(q, grid.groups), lo, hi;
    rows_of_group(a.offsets, group, (int)a.total_m, &lo, &hi);
    group = __builtin_amdgcn_readfirstlane(group);
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
    const int64_t row0 = (int64_t)(b * band + rr % in_band) * P::BM, col0 = (int64_t)(rr / in_band) * P::BN;
    const int rows = N - row0 < P::BM ? (int)(N - row0) : P::BM, cols = K - col0 < P::BN ? (int)(K - col0) : P::BN;
    const int64_t first = lo;                 // the group's first row
    const int places = hi - lo;
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
      if (j < P::kRLoads) {
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
    const u32x4 x_all = buffer_of(a.x, GATHER ? (uint32_t)(a.x_rows * K * 2) : 0u);
    auto load_index = [&](int s) {
      if (!GATHER || wave != 0) return;
      const int left = places - s * kPlaces;
      if (left <= 0) return;
      const u32x4 from =
          buffer_of(a.row_index + first + (int64_t)s * kPlaces, (uint32_t)(left < kPlaces ? left : kPlaces) * 4);
      lds_load4(from, (uint32_t)lane * 4, lds0 + P::kIndex + (uint32_t)(s & 1) * (kPlaces * 4));
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
      const u32x4 r = buffer_of(a.dy + p0 * N, here * (uint32_t)(N * 2));
      const u32x4 c = GATHER ? x_all : buffer_of(a.x + p0 * K, here * (uint32_t)(K * 2));
#pragma unroll
      for (int j = 0; j < P::kLoads; ++j) {
        const uint32_t to = lds0 + slot + (uint32_t)(j * P::kWaves + wave) * 1024;
        if (j < P::kRLoads) {
          lds_load16(r, off[j], to);
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
      const uint32_t at = (rb ^ (uint32_t)(i * 32)) + slot + (uint32_t)(step * 32 * P::BM * 2);
      const u32x2 u = read_turned(at), v = read_turned(at + 4 * P::BM * 2);
      rf[i] = (u32x4){u.x, u.y, v.x, v.y};
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
      constexpr int kRReads = 2;
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
    float* const out = reinterpret_cast<float*>(a.out) + ((int64_t)group * N + row0) * K + col0;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int r = (wm * MI + i) * 16 + r16;
      if (r >= rows) continue;
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int c = (wn * NI + j) * 16 + kg * 4;
        if (c >= cols) continue;
        *reinterpret_cast<v4f*>(out + r * K + c) = acc[i][j];
      }
    }
    wait_loads<0>();
    wait_lds_reads();
    barrier();   // the next tile's loads reuse the stages
  }
}

template <bool GATHER, int MI, int NI, int WM, int WN, int SLOTS>
void launch_tiles(const GroupedGrad& a, int num_cu, hipStream_t stream) {
  using P = Plan<MI, NI, WM, WN, SLOTS>;
  TileGrid g{nullptr, a.groups, (int)a.total_m, (int)((a.k + P::BN - 1) / P::BN), (int)((a.n + P::BM - 1) / P::BM)};
  const int64_t tiles = (int64_t)a.groups * g.band * g.tiles_n;
  const int64_t per_cu = 160 * 1024 / P::kBytes;
  const int64_t most = (num_cu >= 8 ? num_cu / 8 * 8 : 8) * per_cu;
  const int64_t wgs = tiles < most ? (tiles + 7) / 8 * 8 : most;
  hipLaunchKernelGGL((float_wgrad_kernel<GATHER, MI, NI, WM, WN, SLOTS>), dim3((unsigned)wgs), dim3(64 * WM * WN), 0,
                     stream, a, g);
}

}  // namespace

// Tiles of 256 x 256 by eight waves where they fill three quarters of the CUs'
// turns, else of 128 x 128 by four (us, gathered: 16384 rows on 32 experts of
// 4096 x 7168: 1619 and 2146; 921 rows on 8 of 1000 x 1416, 192 tiles: 18 and 22;
// on 11, 264 tiles: 28 and 23).
hipError_t launch_float_wgrad(const GroupedGrad& a, int num_cu, hipStream_t stream) {
  const bool big = fills_turns(a.groups * ((a.n + 255) / 256) * ((a.k + 255) / 256), num_cu);
  if (a.row_index) {
    if (big) launch_tiles<true, 8, 4, 2, 4, 2>(a, num_cu, stream);
    else launch_tiles<true, 4, 4, 2, 2, 2>(a, num_cu, stream);
  } else {
    if (big) launch_tiles<false, 8, 4, 2, 4, 2>(a, num_cu, stream);
    else launch_tiles<false, 4, 4, 2, 2, 2>(a, num_cu, stream);
  }
  return hipGetLastError();
}

}  // namespace fp8blk
