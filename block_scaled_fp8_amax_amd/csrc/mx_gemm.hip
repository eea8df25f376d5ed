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
// The products of an aligned run of 8 elements are added without what lies below
// 2^(e - 13), toward zero, e the largest exponent(a) + exponent(b) of the run's
// products (probed with products that cancel; subnormal operands count as the
// least normal one; runs and blocks are added in fp32).  E2M1 products have no
// bit that low.  E4M3 rows lose at most 7 * 2^-12 of a run's largest product so,
// and bf16 results of them keep it: their operands are known to 2^-4, and one
// product in place of two is twice the rate (8192 x 8192 x 7168: 354 us, 660;
// 131072 rows on 256 experts of 4096 x 7168: 3440, 6600).  Float results take
// two, with the codes of |a| >= 2 and with the others: bits down to 2^-3 under
// e <= 8 + 2, down to 2^-10 under e <= 0 + 2, so that nothing is lost.
#include "groups.h"
#include "launch.h"
#include "mx.h"

namespace fp8blk {

namespace {

// N consecutive results, at any address that their type may have.
template <int N>
__device__ __forceinline__ void store_run(float* y, const float (&v)[N]) {
  typedef float run __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
  for (int e = 0; e < N; e += 4) *reinterpret_cast<run*>(y + e) = (run){v[e], v[e + 1], v[e + 2], v[e + 3]};
}
template <int N>
__device__ __forceinline__ void store_run(uint16_t* y, const float (&v)[N]) {
  typedef uint32_t run __attribute__((ext_vector_type(N / 2), aligned(2)));
  run w;
#pragma unroll
  for (int e = 0; e < N; e += 2) w[e / 2] = pack_bf16x2(v[e], v[e + 1]);
  *reinterpret_cast<run*>(y) = w;
}
// One at byte `at` of a buffer, or nowhere if that lies behind its end.
__device__ __forceinline__ void store_one(__amdgpu_buffer_rsrc_t y, float, uint32_t at, float v) {
  __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), y, (int)at, 0, 0);
}
__device__ __forceinline__ void store_one(__amdgpu_buffer_rsrc_t y, uint16_t, uint32_t at, float v) {
  __builtin_amdgcn_raw_buffer_store_b16((uint16_t)pack_bf16x2(v, 0.f), y, (int)at, 0, 0);
}

// Tiles.  A workgroup of WM x WN waves makes BM x BN outputs, a wave MI x NI
// tiles of 16 x 16.  K advances 256 elements (8 blocks) a stage through a ring
// of SLOTS stages in LDS that loads fill straight from memory; a row is 128
// bytes (E2M1) or 256 (E4M3) of a stage, whole cache lines.  16-byte piece c of
// row r lies at c ^ turn(r), so that the 16 rows of an operand read spread over
// all banks (other turns took twice the time).
//
// A stage is two steps of 128 elements.  Which blocks a step takes is free as
// long as both operands agree: lane l takes block 2 (l / 16) in the first and
// the block after it in the second, so that the scales of both are two
// consecutive bytes of a row, read at once, of which the instruction picks the
// step's.
//
// Operands are held twice: while a step's matrix products run, those of the
// next step are read, early enough to be there when it begins.  In the middle
// of stage s, then, every wave has all of stage s in registers and waits for
// its own part of stage s + 1; behind the one barrier there, stage s + SLOTS is
// loaded into the place of stage s.
//
// Stages go on from tile to tile of a workgroup: while one tile ends, loads are
// for the next.  Behind the last tile they find an empty buffer, which costs
// nothing and keeps their number the same.  A new tile's group, and the indices
// of gathered rows, are read where its first loads are formed, and each of those
// reads waits for all that is on its way (131072 E4M3 rows on 256 experts of
// 4096 x 7168: 3510 us gathered, 3457 without an index).
//
// Scales come for CHUNK stages at a time, 8 CHUNK bytes of a row, into two
// places in turn.  (Each row touched takes a cache line's time, so that CHUNK
// is as large as LDS allows: 2 instead of 4 cost 100 ns a stage of 128 x 256.)
template <bool FP4>
__device__ __forceinline__ int turn(int r) {
  return FP4 ? (r >> 1) & 7 : r & 15;
}

// The column of y (row of the weights) that row r of the tile's weights in LDS
// is: a lane's results of two tiles are eight consecutive columns, and those of
// a group of four lanes a whole 64 bytes of bf16.
template <int NI>
__device__ __forceinline__ int column(int r) {
  return NI % 2 ? r : (r & ~31) | (r & 12) << 1 | (r & 16) >> 2 | (r & 3);
}

template <bool A_FP4, int MI, int NI, int WM, int WN, int SLOTS>
struct Plan {
  static constexpr int kWaves = WM * WN, BM = 16 * MI * WM, BN = 16 * NI * WN;
  static constexpr int kARow = A_FP4 ? 128 : 256, kAPer = kARow / 16;                   // 16-byte pieces of a row
  static constexpr int kA = BM * kARow, kStage = kA + BN * 128;
  static constexpr int kALoads = kA / 1024 / kWaves, kLoads = kStage / 1024 / kWaves;   // of a wave and stage
  static constexpr int kRing = SLOTS * kStage;
  static constexpr int kLds = 160 * 1024 - kMaxGroups * 4;
  static constexpr int CHUNK = kRing + (BM + BN) * 64 <= kLds ? 4 : 2;
  static constexpr int kSRow = 8 * CHUNK, kChunk = (BM + BN) * kSRow, kSRows = 256 / kSRow;   // rows of a load
  static constexpr int kSA = BM / kSRows / kWaves, kSLoads = (BM + BN) / kSRows / kWaves;     // of a wave and chunk
  static constexpr int kScales = kRing, kBytes = kScales + 2 * kChunk;
  // loads of a wave that may be on their way when the first stage, and a later
  // one, is waited for; the least stores of a wave and whole tile
  static constexpr int kFirst = (SLOTS - 1) * kLoads, kLater = (SLOTS - 2) * kLoads, kStores = NI % 2 ? MI * NI : MI * NI / 2;
  // The products beside which a stage's loads go out, from the middle of a
  // stage on; until which stage the stores of the tile before may be on their
  // way when a stage is waited for.
  static constexpr int kSpan = SLOTS > 2 ? 2 * MI * NI : MI * NI, kPast = SLOTS > 2 ? SLOTS - 2 : 1;
  static_assert(kA % (1024 * kWaves) == 0 && kStage % (1024 * kWaves) == 0, "shares of the loads");
  static_assert(BM % (kSRows * kWaves) == 0 && BN % (kSRows * kWaves) == 0, "shares of the scales' loads");
  static_assert(kWaves * 8 % 32 == 0 && kWaves * (64 / kAPer) % 16 == 0 && kSRows * kWaves % 32 == 0, "a lane's rows");
  static_assert(SLOTS >= 2 && SLOTS <= 3, "a chunk of scales is waited for with the stage after the one it is sent for with");
  static_assert(kFirst + kStores < 64, "vmcnt");
  static_assert(kBytes <= kLds, "LDS");
};

template <bool A_FP4, bool SPLIT, int MI, int NI, int WM, int WN, int SLOTS>
__global__ __launch_bounds__(64 * WM * WN) void mx_gemm_kernel(MxProduct p, TileGrid grid) {
  using P = Plan<A_FP4, MI, NI, WM, WN, SLOTS>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[P::kBytes];
  __shared__ int upto[kMaxGroups];
  const int t = (int)threadIdx.x, lane = t & 63, r16 = lane & 15, kg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6), wm = wave / WN, wn = wave % WN;
  const uint32_t K = (uint32_t)p.k;
  const int stages = (int)((K + 255) / 256), chunks = (stages + P::CHUNK - 1) / P::CHUNK;
  const uint32_t a_row = A_FP4 ? K / 2 : K, b_row = K / 2, s_row = K / 32;
  const uint32_t lds0 = lds_address(smem);
  const int tiles = __builtin_amdgcn_readfirstlane(count_tiles<P::BM, 64 * P::kWaves>(grid, upto));
  // where a lane's operands lie in a stage (rows of 16 tiles keep their turn),
  // and its scales in a chunk
  const uint32_t xa0 = A_FP4 ? (uint32_t)((wm * MI * 16 + r16) * 128 + ((2 * kg) ^ turn<true>(r16)) * 16)
                             : (uint32_t)((wm * MI * 16 + r16) * 256 + ((4 * (kg >> 1) + (kg & 1)) ^ turn<false>(r16)) * 16);
  const uint32_t xa1 = xa0 ^ (A_FP4 ? 16u : 32u);
  const uint32_t wb0 = (uint32_t)(P::kA + (wn * NI * 16 + r16) * 128 + ((2 * kg) ^ turn<true>(r16)) * 16);
  const uint32_t wb1 = wb0 ^ 16u;
  const uint32_t xs = (uint32_t)(P::kScales + (wm * MI * 16 + r16) * P::kSRow);
  const uint32_t ws = (uint32_t)(P::kScales + (P::BM + wn * NI * 16 + r16) * P::kSRow);
  auto columns = [&](const Tile& of) {
    const int64_t rest = p.n - (int64_t)of.col * P::BN;
    return rest < P::BN ? (int)rest : P::BN;
  };
  // Rows behind the tile's last, and columns behind y's, lie behind the end of
  // their buffers and are read as zeros (or, where that is past 32 bits, as
  // the first row); nothing of them is stored.
  auto row_of = [&](const Tile& of, int r) -> uint32_t {
    if (!p.row_index) return (uint32_t)r;
    return r < of.rows ? (uint32_t)clamp_to(p.row_index[(int64_t)of.row0 + r], 0, (int)p.a_rows - 1) : (uint32_t)p.a_rows;
  };

  // What lies past K (in a last half stage) is read as zeros, at this offset.
  // Whether a lane's pieces are in the upper half is the same for all its
  // loads: their rows are a multiple of 16 apart.
  constexpr uint32_t kNowhere = 0xFFFFFFF0u;
  const int a_piece = (lane % P::kAPer) ^ turn<A_FP4>(wave * (64 / P::kAPer) + lane / P::kAPer);
  const uint32_t a_past = a_piece & (P::kAPer / 2) ? kNowhere : 0u;
  const uint32_t b_past = ((lane % 8) ^ turn<true>(wave * 8 + lane / 8)) & 4 ? kNowhere : 0u;

  // The stages to load, and the scales (below), from tile to tile: tiles as
  // tile_at finds them, unless one of these has it already.
  int s_it = -1, s_chunk = chunks;
  Tile s_tile;
  int d_it = -1, d_stage = stages;
  Tile d_tile;
  u32x4 a, b;
  uint32_t aoff[P::kALoads], boff = 0;
  auto next_stage = [&]() {
    if (++d_stage < stages) return;
    d_stage = 0;
    const int id = tile_of_turn(++d_it);
    if (id >= tiles) {
      a.z = b.z = 0;
      return;
    }
    const Tile of = d_it == s_it ? s_tile : tile_at<P::BM>(grid, upto, id);
    d_tile = of;
    const int64_t n0 = (int64_t)of.col * P::BN;
    a = p.row_index ? buffer_of(p.a, (uint32_t)p.a_rows * a_row)
                    : buffer_of(p.a + of.row0 * (int64_t)a_row, (uint32_t)of.rows * a_row);
    b = buffer_of(p.b + (of.group * p.n + n0) * b_row, (uint32_t)columns(of) * b_row);
    // this wave's loads: blocks wave, wave + kWaves, ... of 1 KiB
#pragma unroll
    for (int j = 0; j < P::kALoads; ++j) {
      const int r = (j * P::kWaves + wave) * (64 / P::kAPer) + lane / P::kAPer;
      aoff[j] = row_of(of, r) * a_row + (uint32_t)(((lane % P::kAPer) ^ turn<A_FP4>(r)) * 16);
    }
    const int r = wave * 8 + lane / 8;
    boff = (uint32_t)column<NI>(r) * b_row + (uint32_t)(((lane % 8) ^ turn<true>(r)) * 16);
  };
  auto load = [&](uint32_t slot, int from, int end) {
    const bool half = (uint32_t)d_stage * 256 + 128 == K;
    const uint32_t an = half ? a_past : 0u, bn = half ? b_past : 0u;
#pragma unroll
    for (int j = from; j < end; ++j) {
      const uint32_t to = lds0 + slot + (uint32_t)(j * P::kWaves + wave) * 1024;
      if (j < P::kALoads)
        lds_load16(a, (aoff[j] + (uint32_t)d_stage * P::kARow) | an, to);
      else
        lds_load16(b, (boff + (uint32_t)(j - P::kALoads) * (P::kWaves * 8 * b_row) + (uint32_t)d_stage * 128) | bn, to);
    }
  };
  u32x4 as, bs;
  uint32_t asoff[P::kSA], bsoff = 0;
  // A stage's 8 bytes of row r lie at their place ^ bit 3 of r, so that 16 rows
  // spread over all banks.
  constexpr int kSPer = P::kSRow / 4;
  const uint32_t piece = (uint32_t)((lane % kSPer) ^ (((wave * P::kSRows + lane / kSPer) >> 3 & 1) * 2)) * 4;
  const uint32_t stage_turn = (uint32_t)(r16 >> 3) * 8, pick = 0x0C0C0100u + 0x0202u * (uint32_t)kg;   // bytes 2 kg, 2 kg + 1
  auto next_scales = [&](int place) {
    if (++s_chunk >= chunks) {
      s_chunk = 0;
      const int id = tile_of_turn(++s_it);
      if (id >= tiles) {
        as.z = bs.z = 0;
      } else {
        const Tile of = s_tile = tile_at<P::BM>(grid, upto, id);
        const int64_t n0 = (int64_t)of.col * P::BN;
        as = p.row_index ? buffer_of(p.a_scale, (uint32_t)p.a_rows * s_row)
                         : buffer_of(p.a_scale + of.row0 * (int64_t)s_row, (uint32_t)of.rows * s_row);
        bs = buffer_of(p.b_scale + (of.group * p.n + n0) * s_row, (uint32_t)columns(of) * s_row);
#pragma unroll
        for (int j = 0; j < P::kSA; ++j) {
          asoff[j] = row_of(of, (j * P::kWaves + wave) * P::kSRows + lane / kSPer) * s_row + piece;
        }
        bsoff = (uint32_t)column<NI>(wave * P::kSRows + lane / kSPer) * s_row + piece;
      }
    }
    const uint32_t along = (uint32_t)(s_chunk * P::kSRow), none = along + piece < s_row ? 0u : kNowhere;
#pragma unroll
    for (int j = 0; j < P::kSLoads; ++j) {
      const uint32_t to = lds0 + (uint32_t)(P::kScales + place * P::kChunk + (j * P::kWaves + wave) * 256);
      if (j < P::kSA)
        lds_load4(as, (asoff[j] + along) | none, to);
      else
        lds_load4(bs, (bsoff + (uint32_t)(j - P::kSA) * (P::kWaves * P::kSRows * s_row) + along) | none, to);
    }
  };

  int it = 0, id = tile_of_turn(0);
  if (id >= tiles) return;
  next_scales(0);
  next_scales(1);
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    next_stage();
    load((uint32_t)(i * P::kStage), 0, P::kLoads);
  }

  typedef typename std::conditional<A_FP4, u32x4, v8i>::type XFrag;
  v4f acc[MI][NI];
  XFrag x0[MI], x1[MI];
  u32x4 w0[NI], w1[NI];
  int sx[MI], sw[NI];
  u32x2 sxnext[MI], swnext[NI];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
  };
  auto read_x = [&](XFrag& x, uint32_t at, int i) {
    const u32x4 lo = *reinterpret_cast<const u32x4*>(smem + at + (uint32_t)(i * 16 * P::kARow));
    if constexpr (A_FP4)
      x = lo;
    else
      x = frag(lo, *reinterpret_cast<const u32x4*>(smem + (at ^ 128u) + (uint32_t)(i * 16 * P::kARow)));
  };
  auto read_w = [&](u32x4& w, uint32_t at, int i) {
    w = *reinterpret_cast<const u32x4*>(smem + at + (uint32_t)(i * 2048));
  };
  auto read_scale = [&](uint32_t at, int i) {
    return *reinterpret_cast<const u32x2*>(smem + at + (uint32_t)(i * 16 * P::kSRow));
  };
  auto own = [&](u32x2 scales) { return (int)__builtin_amdgcn_perm(scales.y, scales.x, pick); };
  // product j of row i of step STEP of a stage
  v8i hi, lo;
  auto multiply = [&](auto step, int i, int j, const XFrag* x, const u32x4* w) {
    constexpr int STEP = decltype(step)::value;
    if (j == 0) {
      hi = frag(x[i]);
      if constexpr (SPLIT) {
        lo = hi;
        hi = large_codes(hi);
        lo = lo ^ hi;
      }
    }
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(w[j]), hi, acc[i][j], 4, A_FP4 ? 4 : 0, STEP, sw[j],
                                                                 STEP, sx[i]);
    if constexpr (SPLIT)
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(w[j]), lo, acc[i][j], 4, 0, STEP, sw[j], STEP,
                                                                   sx[i]);
  };
  // (the compiler would move products past the barriers and the branches)
  auto pin_row = [&](int i) {
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      if constexpr (MI * NI >= 32) asm volatile("" : "+a"(acc[i][j])); else asm volatile("" : "+v"(acc[i][j]));
    }
  };
  auto pin = [&]() {
#pragma unroll
    for (int i = 0; i < MI; ++i) pin_row(i);
  };
  // The reads of a step (x 0, all w, the other x) go out beside its first
  // products, the loads of a stage beside those of P::kSpan from its middle on.
  constexpr int kProducts = MI * NI, kReads = MI + NI, kReadSpan = MI > 1 ? kProducts - NI : kProducts;
  auto part = [](int q, int span, int all) { return q < span ? q * all / span : all; };

  wait_loads<P::kFirst>();
  barrier();
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    read_x(x0[i], xa0, i);
    sx[i] = own(read_scale(xs + stage_turn, i));
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    read_w(w0[i], wb0, i);
    sw[i] = own(read_scale(ws + stage_turn, i));
  }

  // of the stage being multiplied: its place in the ring, that of its scales;
  // and the place behind it, that loads fill
  uint32_t slot = 0, place = 0, freed = P::kRing - P::kStage;
  int in_chunk = 0;
  bool stored = false;                 // kStores stores of the tile before, or more, are behind the last loads
  for (;;) {
    // Waves whose rows are all behind the tile's last only load.  (Waves 0 to 3,
    // on a SIMD each, have the first rows.)
    const Tile here = d_it == it ? d_tile : tile_at<P::BM>(grid, upto, id);
    const bool busy = wm * MI * 16 < here.rows;
    clear();
    pin();
    for (int s = 0; s < stages; ++s) {
      if (busy) {
        each<kProducts>([&](auto qc) {
          constexpr int q = decltype(qc)::value;
          multiply(std::integral_constant<int, 0>{}, q / NI, q % NI, x0, w0);
#pragma unroll
          for (int r = part(q, kReadSpan, kReads); r < part(q + 1, kReadSpan, kReads); ++r) {
            if (r == 0 || r > NI)
              read_x(x1[r ? r - NI : 0], slot + xa1, r ? r - NI : 0);
            else
              read_w(w1[r - 1], slot + wb1, r - 1);
          }
          load(freed, part(kProducts + q, P::kSpan, P::kLoads), part(kProducts + q + 1, P::kSpan, P::kLoads));
          __builtin_amdgcn_sched_barrier(0);
        });
        pin();
        wait_lds_reads();
      } else {
        load(freed, part(kProducts, P::kSpan, P::kLoads), P::kLoads);
      }
      if (stored && s < P::kPast) wait_loads<P::kLater + P::kStores>(); else wait_loads<P::kLater>();
      barrier();
      freed = slot;
      slot = slot + P::kStage == (uint32_t)P::kRing ? 0u : slot + P::kStage;
      if (++in_chunk == P::CHUNK || s + 1 == stages) {
        next_scales((int)place);
        place ^= 1;
        in_chunk = 0;
      }
      next_stage();
      const uint32_t at = place * P::kChunk + ((uint32_t)in_chunk * 8 ^ stage_turn);
      // The next stage may be of another tile.
      if (busy || s + 1 == stages) {
        each<kProducts>([&](auto qc) {
          constexpr int q = decltype(qc)::value;
          multiply(std::integral_constant<int, 1>{}, q / NI, q % NI, x1, w1);
#pragma unroll
          for (int r = part(q, kReadSpan, kReads); r < part(q + 1, kReadSpan, kReads); ++r) {
            if (r == 0 || r > NI) {
              const int i = r ? r - NI : 0;
              read_x(x0[i], slot + xa0, i);
              sxnext[i] = read_scale(at + xs, i);
            } else {
              read_w(w0[r - 1], slot + wb0, r - 1);
              swnext[r - 1] = read_scale(at + ws, r - 1);
            }
          }
          load(freed, part(q, P::kSpan, P::kLoads), part(q + 1, P::kSpan, P::kLoads));
          __builtin_amdgcn_sched_barrier(0);
        });
        pin();
#pragma unroll
        for (int i = 0; i < MI; ++i) sx[i] = own(sxnext[i]);
#pragma unroll
        for (int j = 0; j < NI; ++j) sw[j] = own(swnext[j]);
      } else {
        load(freed, 0, part(kProducts, P::kSpan, P::kLoads));
      }
    }

    // Lane l holds of each 16 x 16 row l % 16 and four columns.  Runs that the
    // last column cuts are stored one by one, what is outside into nothing: a
    // branch for each would make most of the kernel's code.
    constexpr int kRun = NI % 2 ? 4 : 8;
    const int64_t n0 = (int64_t)here.col * P::BN;
    const int cols = columns(here);
    stored = here.rows == P::BM && cols == P::BN;
    auto store = [&](auto* y) {
      typedef typename std::remove_pointer<decltype(y)>::type T;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        pin_row(i);                               // (few results at a time in registers)
        const int row = (wm * MI + i) * 16;       // the first
        T* const first = y + ((int64_t)here.row0 + row) * p.n + n0;
        const bool there = row + r16 < here.rows;
#pragma unroll
        for (int j = 0; j < NI; j += kRun / 4) {
          const int col = wn * NI * 16 + j * 16, c = col + kg * kRun;
          float v[kRun];
#pragma unroll
          for (int e = 0; e < kRun; ++e) v[e] = acc[i][j + e / 4][e % 4];
          if (col + 4 * kRun <= cols) {
            if (there) store_run<kRun>(first + r16 * p.n + c, v);
          } else if (col < cols) {
            const __amdgpu_buffer_rsrc_t to =
                __builtin_amdgcn_make_buffer_rsrc(first, 0, (int)(16 * p.n * sizeof(T)), 0x00027000);
#pragma unroll
            for (int e = 0; e < kRun; ++e)
              store_one(to, T(), there && c + e < cols ? (uint32_t)((r16 * p.n + c + e) * sizeof(T)) : kNowhere, v[e]);
          }
        }
      }
    };
    // (E4M3 rows: floats exactly where products are split)
    if (A_FP4 ? p.out_f32 : SPLIT) store(reinterpret_cast<float*>(p.y)); else store(reinterpret_cast<uint16_t*>(p.y));
    id = tile_of_turn(++it);
    if (id >= tiles) break;
  }
  wait_loads<0>();   // (of the empty buffers)
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
//   256 x 256 by four waves, E2M1 only, from 1024 rows on: 8192 x 8192 x 7168:
//     247, 128 x 256: 266; 512 rows on each of 64 experts of 4096 x 7168: 692
//     and 669.  (It keeps 87 registers in memory, what it reads back between a
//     tile's rows of results waits for their stores; 8192 x 8190 x 7168, whose
//     last columns are cut: 281);
//   128 x 256, from three quarters of the CUs on: 1500 x 4096 x 2048: 16.9 /
//     14.9, 128 x 128: 21.7 / 17.1; at half (2048 x 2048 x 4096) 25.5 / 20.2 and
//     21.3 / 15.8;
//   64 x 256 for up to 64 rows, 32 x 128 for up to 32: 2048 rows on 64 experts
//     of 4096 x 4096: 163 / 132 and 155 / 133, 64 x 64: 203 / 155; 1024 rows on
//     32: 81 / 66, 68 / 57 and 112 / 68;
//   64 x 64 by four waves, from two to a CU on: 512 x 4096 x 4096: 17.2 / 13.6,
//     by eight 19.7 / 15.5; 256 rows: 13.2 / 11.5 and 11.5 / 10.5.
// Float results of E4M3 rows, whose operands take twice the registers (128 x 256
// keeps 13 in memory, read back for cut columns) and products: 128 x 256 from four to a CU on (8192 x 4096 x 4096: 206, 64 x 256:
// 230; 2048 x 2048 x 4096: 52 and 33), 64 x 256 (that: 33, 32 x 128: 42), or 32
// x 128 (1009 x 2002 x 5120: 27.7, 64 x 64: 31.2, 64 x 256: 37).
template <bool A_FP4, bool SPLIT>
void launch_rule(const MxProduct& p, int num_cu, hipStream_t stream) {
  const int64_t active = p.offsets ? (p.groups < p.m ? p.groups : p.m) : 1;
  const int64_t rows = (p.m + active - 1) / active;
  auto most = [&](int64_t bm, int64_t bn) {     // tiles at most
    return (p.offsets ? p.m / bm + active : (p.m + bm - 1) / bm) * ((p.n + bn - 1) / bn);
  };
  auto fills = [&](int64_t bm, int64_t bn, int quarters = 3) {   // of the CUs
    return 4 * active * ((rows + bm - 1) / bm) * ((p.n + bn - 1) / bn) >= quarters * num_cu;
  };
  if constexpr (SPLIT) {
    if (rows > 64 && fills(128, 256, 16))
      launch_tiles<A_FP4, SPLIT, 4, 4, 2, 4, 2>(p, most(128, 256), num_cu, stream);
    else if (rows > 32 && fills(64, 256))
      launch_tiles<A_FP4, SPLIT, 2, 4, 2, 4, 2>(p, most(64, 256), num_cu, stream);
    else
      launch_tiles<A_FP4, SPLIT, 1, 4, 2, 2, 2>(p, most(32, 128), num_cu, stream);
  } else {
    if constexpr (A_FP4) {
      if (rows >= 1024 && fills(256, 256))
        return launch_tiles<A_FP4, SPLIT, 8, 8, 2, 2, 2>(p, most(256, 256), num_cu, stream);
    }
    if (rows > 64 && fills(128, 256))
      launch_tiles<A_FP4, SPLIT, 4, 4, 2, 4, A_FP4 ? 3 : 2>(p, most(128, 256), num_cu, stream);
    else if (rows > 64 && fills(128, 128))
      launch_tiles<A_FP4, SPLIT, 4, 2, 2, 4, A_FP4 ? 3 : 2>(p, most(128, 128), num_cu, stream);
    else if (rows > 32 && rows <= 64 && fills(64, 256))
      launch_tiles<A_FP4, SPLIT, 2, 4, 2, 4, A_FP4 ? 3 : 2>(p, most(64, 256), num_cu, stream);
    else if (rows <= 32 && fills(32, 128))
      launch_tiles<A_FP4, SPLIT, 1, 4, 2, 2, A_FP4 ? 3 : 2>(p, most(32, 128), num_cu, stream);
    else if (fills(64, 64, 8))
      launch_tiles<A_FP4, SPLIT, 2, 2, 2, 2, 2>(p, most(64, 64), num_cu, stream);
    else
      launch_tiles<A_FP4, SPLIT, 2, 1, 2, 4, 3>(p, most(64, 64), num_cu, stream);
  }
}

}  // namespace

// Few rows: the kernel that cuts K instead, up to 8 a group (us, E4M3 / E2M1;
// dense 64 x 4096 x 7168: 10.7 / 7.6, tiles 16.6 / 14.8, 128 rows: 17.3 / 13.0
// and 16.6 / 14.8; gathered, 64 rows on 52 of 256 experts of 4096 x 7168: 139 /
// 138, tiles 166 / 154; 512 on 60 of 64 of 4096 x 4096: 106 / 97, tiles 106 / 98;
// 1024 on 64: 133 / 120 and 110 / 104).  The host does not know which groups
// have rows: few rows for 256 groups that 32 of them get go the slower way
// (2048 rows of 4096 x 7168: 356 / 321, tiles 118 / 101).  The kernel finds all
// rows of A with 32-bit byte offsets.
hipError_t launch_mx_product(const MxProduct& p, int num_cu, hipStream_t stream) {
  const int64_t active = p.offsets ? (p.groups < p.m ? p.groups : p.m) : 1;
  const bool few = p.offsets ? p.m <= 8 * active : ((p.m + 15) / 16) * ((p.n + 15) / 16) <= 4 * num_cu;
  if (few && p.a_rows * (p.a_fp4 ? p.k / 2 : p.k) < (int64_t(1) << 32)) return launch_mx_few(p, stream);
  if (p.a_fp4)
    launch_rule<true, false>(p, num_cu, stream);
  else if (p.out_f32)
    launch_rule<false, true>(p, num_cu, stream);
  else
    launch_rule<false, false>(p, num_cu, stream);
  return hipGetLastError();
}

}  // namespace fp8blk
