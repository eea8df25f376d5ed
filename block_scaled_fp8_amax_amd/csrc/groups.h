// Rows of routed experts and the tiles over them, as the kernels of the MXFP4
// experts find them, and the loads that fill LDS with those tiles.
#pragma once

#include <type_traits>

#include "device.h"

namespace fp8blk {

// f(0), ..., f(N - 1) with compile-time arguments.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    each<N, I + 1>(f);
  }
}

__device__ __forceinline__ int clamp_to(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// Stages of `each` places (or rows) that hold `places` of them, up to 2^31 - 1.
__host__ __device__ __forceinline__ int stages_in(int places, int each) {
  return (int)(((uint32_t)places + (uint32_t)each - 1u) / (uint32_t)each);
}

// The offsets are not checked on the host: group g's rows are [lo, hi) with
// lo = off[g] and hi = off[g + 1] clamped into [0, total_m] and hi >= lo.
__device__ __forceinline__ void rows_of_group(const int32_t* offsets, int g, int total_m, int* lo, int* hi) {
  *lo = clamp_to(offsets[g], 0, total_m);
  *hi = clamp_to(offsets[g + 1], *lo, total_m);
}

// The ordinal-th group with rows, and these; false where there are fewer.  For
// one wave, which looks at 256 groups at a time.
__device__ __forceinline__ bool nth_group(const int32_t* offsets, int groups, int total_m, int ordinal, int* g, int* lo,
                                          int* hi) {
  const int lane = (int)threadIdx.x & 63;
  int seen = 0;
  for (int b = 0; b < groups; b += 256) {
    int l[4], h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = b + i * 64 + lane, at = e < groups ? e : groups - 1;
      l[i] = offsets[at];
      h[i] = offsets[at + 1];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      l[i] = clamp_to(l[i], 0, total_m);
      h[i] = b + i * 64 + lane < groups ? clamp_to(h[i], l[i], total_m) : l[i];
      const unsigned long long full = __builtin_amdgcn_ballot_w64(h[i] > l[i]);
      const int here = __builtin_popcountll(full);
      if (ordinal < seen + here) {
        const bool mine = h[i] > l[i] && __builtin_popcountll(full & ((1ull << lane) - 1)) == ordinal - seen;
        const int src = __builtin_ctzll(__builtin_amdgcn_ballot_w64(mine));
        *g = b + i * 64 + src;
        *lo = __builtin_amdgcn_readlane(l[i], src);
        *hi = __builtin_amdgcn_readlane(h[i], src);
        return true;
      }
      seen += here;
    }
  }
  return false;
}

// Most groups of a call: one int of LDS each.
constexpr int kMaxGroups = 1024;

// Most tiles that are counted.  Results that fit the GPU's memory have fewer;
// offsets that fall and rise again, which may name each row many times, would
// have more than an int counts, and tiles outside the rows with it.
constexpr int kMostTiles = 1 << 30;
__host__ __device__ __forceinline__ int add_tiles(int a, int b) { return a < kMostTiles - b ? a + b : kMostTiles; }
__host__ __device__ __forceinline__ int times_tiles(int a, int b) {
  const int64_t all = (int64_t)a * b;
  return all < kMostTiles ? (int)all : kMostTiles;
}

// The tiles of a call: every group's rows cut into row tiles of BM, times
// `tiles_n` column tiles.  Tiles are numbered group by group;
// inside a group in bands of `band` row tiles, column by column, so
// that consecutive numbers share operands.
struct TileGrid {
  const int32_t* offsets;   // null: one group of all rows
  int groups, total_m, tiles_n, band;
};

// Row tiles of the groups up to each place, in `upto` (LDS, `groups` ints);
// returns the number of tiles.  For a workgroup of THREADS threads, all of
// which have to call it.
template <int BM, int THREADS>
__device__ __forceinline__ int count_tiles(const TileGrid& t, int* upto) {
  if (!t.offsets) return times_tiles(stages_in(t.total_m, BM), t.tiles_n);
  constexpr int PER = kMaxGroups / THREADS;
  const int i = (int)threadIdx.x;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int q = i + j * THREADS;
    if (q >= t.groups) break;
    int lo, hi;
    rows_of_group(t.offsets, q, t.total_m, &lo, &hi);
    upto[q] = stages_in(hi - lo, BM);
  }
  __syncthreads();
  for (int d = 1; d < t.groups; d <<= 1) {
    int v[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int q = i + j * THREADS;
      v[j] = q < t.groups && q >= d ? upto[q - d] : 0;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int q = i + j * THREADS;
      if (q < t.groups) upto[q] = add_tiles(upto[q], v[j]);
    }
    __syncthreads();
  }
  return times_tiles(upto[t.groups - 1], t.tiles_n);
}

struct Tile {
  int group, row0, rows, col;   // rows: of the tile; col: column tile
};

// Tile number `id` (below count_tiles' result).  Wave-uniform.
template <int BM>
__device__ __forceinline__ Tile tile_at(const TileGrid& t, const int* upto, int id) {
  int g = 0, before = 0, here, lo = 0, hi = t.total_m;
  if (t.offsets) {
    const int slot = id / t.tiles_n;
    int a = 0, b = t.groups - 1;      // place q with upto[q - 1] <= slot < upto[q]
    while (a < b) {
      const int mid = (a + b + 1) >> 1;
      if (upto[mid - 1] <= slot) a = mid; else b = mid - 1;
    }
    before = a > 0 ? upto[a - 1] : 0;
    here = upto[a] - before;
    g = a;
    rows_of_group(t.offsets, g, t.total_m, &lo, &hi);
  } else {
    here = stages_in(hi, BM);
  }
  const int r = id - before * t.tiles_n;
  const int band = t.band < here ? t.band : here;
  const int b = r / (band * t.tiles_n), rr = r - b * (band * t.tiles_n);
  const int rows_here = here - b * band < band ? here - b * band : band;
  Tile out;
  out.group = __builtin_amdgcn_readfirstlane(g);
  out.row0 = __builtin_amdgcn_readfirstlane(lo + (b * band + rr % rows_here) * BM);
  out.rows = __builtin_amdgcn_readfirstlane(hi - out.row0 < BM ? hi - out.row0 : BM);
  out.col = __builtin_amdgcn_readfirstlane(rr / rows_here);
  return out;
}

// The `it`-th tile of this workgroup.  Workgroup b runs on XCD b % 8, and the
// XCDs have L2 caches of their own: each takes runs of consecutive tiles in
// turn, one for each of its workgroups.  (Runs of two for each leave more idle
// in the last turn: both gradients of 16384 rows on 32 experts of 4096 x 7168
// 2639 us, 2507 so; products of 131072 rows on 256 of them 3625, 3492 so.)
__device__ __forceinline__ int tile_of_turn(int it) {
  const int w = (int)(gridDim.x >> 3);
  return (it * 8 + (int)(blockIdx.x & 7)) * w + (int)(blockIdx.x >> 3);
}

// ------------------------------------------------- loads into LDS, and waits

// A buffer's descriptor, and 16 or 4 bytes per lane from voff on in it straight
// to LDS at lds + 16 (4) * lane; `lds` is wave-uniform.  Lanes whose bytes reach
// past the buffer's length write zeros.  Counted by vmcnt, in order.
__device__ __forceinline__ u32x4 buffer_of(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return (u32x4){(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)), bytes, 0x00027000u};
}
__device__ __forceinline__ void lds_load4(u32x4 buffer, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds" ::"v"(voff), "s"(buffer), "s"(lds)
               : "memory");
}
__device__ __forceinline__ void lds_load16(u32x4 buffer, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(voff), "s"(buffer), "s"(lds)
               : "memory");
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

__device__ __forceinline__ void barrier() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
}

// Address of a __shared__ object in LDS.
__device__ __forceinline__ uint32_t lds_address(const void* p) { return (uint32_t)(uintptr_t)p; }

}  // namespace fp8blk
