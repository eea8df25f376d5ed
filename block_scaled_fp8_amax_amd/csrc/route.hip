// Routing to experts (gfx950): scores, group-limited top-k, weights; their
// gradient; and the plan that sorts (token, choice) pairs by expert.
//
//   s = softmax(l) or sigmoid(l);  key = s + bias
//   ids = top-k of key over the best groups, ties to the lowest index
//   w = scale * s[ids] (/ sum of s[ids])
//
// Two experts' scores can be closer than fp32 tells apart (256 scores of
// 16384 tokens: several such pairs per batch), and a choice that depends on
// rounding is not reproducible elsewhere, so keys are compared in double
// precision; without a bias both score functions rise with the logit and
// the logits themselves are compared.
#include "device.h"
#include "launch.h"

namespace fp8blk {

namespace {

constexpr float kFltMax = 3.402823466e38f;

__device__ __forceinline__ float load_logit(const void* l, bool f32, int64_t i) {
  if (f32) return reinterpret_cast<const float*>(l)[i];
  return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(l)[i] << 16);
}

// Orders a wave's own LDS reads and writes across its lanes (the hardware
// keeps them in order; this keeps the compiler to it).
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

// The two values of step STEP of a butterfly over 2^6 lanes, in either order:
// after the steps 0 .. n-1 of a commutative operation each run of 2^n lanes
// holds its result (the mirror steps pair lanes whose runs are complete
// already; the swap steps leave the lower run's value in one register and
// the upper run's in the other, for the lanes of both).
template <int STEP>
__device__ __forceinline__ void both(uint32_t v, uint32_t& a, uint32_t& b) {
  a = v;
  if constexpr (STEP == 0) b = dpp<kQuadSwap1>(v);
  if constexpr (STEP == 1) b = dpp<kQuadSwap2>(v);
  if constexpr (STEP == 2) b = dpp<kRowHalfMirror>(v);
  if constexpr (STEP == 3) b = dpp<kRowMirror>(v);
  if constexpr (STEP == 4) {
    const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(v, v, false, false));
    a = r.x;
    b = r.y;
  }
  if constexpr (STEP == 5) {
    const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(v, v, false, false));
    a = r.x;
    b = r.y;
  }
}
template <int STEP>
__device__ __forceinline__ void both(int v, int& a, int& b) {
  uint32_t x, y;
  both<STEP>((uint32_t)v, x, y);
  a = (int)x;
  b = (int)y;
}
template <int STEP>
__device__ __forceinline__ void both(float v, float& a, float& b) {
  uint32_t x, y;
  both<STEP>(__float_as_uint(v), x, y);
  a = __uint_as_float(x);
  b = __uint_as_float(y);
}
template <int STEP>
__device__ __forceinline__ void both(double v, double& a, double& b) {
  const u32x2 w = __builtin_bit_cast(u32x2, v);
  u32x2 x, y;
  uint32_t p, q;
  both<STEP>(w.x, p, q);
  x.x = p;
  y.x = q;
  both<STEP>(w.y, p, q);
  x.y = p;
  y.y = q;
  a = __builtin_bit_cast(double, x);
  b = __builtin_bit_cast(double, y);
}

__device__ __forceinline__ float larger(float a, float b) { return __builtin_fmaxf(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return __builtin_fminf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return a > b ? a : b; }
__device__ __forceinline__ double smaller(double a, double b) { return a < b ? a : b; }
__device__ __forceinline__ int larger(int a, int b) { return a > b ? a : b; }
__device__ __forceinline__ int smaller(int a, int b) { return a < b ? a : b; }

// A float as an int of the same order, and back.
__device__ __forceinline__ int ordered(float f) {
  const int i = (int)__float_as_uint(f);
  return i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float unordered(int i) { return __uint_as_float((uint32_t)(i ^ ((i >> 31) & 0x7FFFFFFF))); }

// A logit or bias as the ranking takes it: NaN masks, +inf is the largest
// float.
__device__ __forceinline__ float clean(float v) {
  v = v > -__builtin_inff() ? v : -__builtin_inff();
  return v > kFltMax ? kFltMax : v;
}

// e / per for e < 1024: the quotient's distance from an integer is at least
// 1 / (2 per) at e + 1/2, far above the product's rounding.
__device__ __forceinline__ int group_of(const RouteArgs& a, int e) { return (int)(((float)e + 0.5f) * a.inv_per); }

template <int G, typename T, int STEP = 0>
__device__ __forceinline__ T run_max(T v) {
  if constexpr ((1 << STEP) < G) {
    T a, b;
    both<STEP>(v, a, b);
    return run_max<G, T, STEP + 1>(larger(a, b));
  } else {
    return v;
  }
}
template <int G, typename T, int STEP = 0>
__device__ __forceinline__ T run_add(T v) {
  if constexpr ((1 << STEP) < G) {
    T a, b;
    both<STEP>(v, a, b);
    return run_add<G, T, STEP + 1>(a + b);
  } else {
    return v;
  }
}
// Best (key, index) of a run: highest key, lowest index among equals.
template <int G, int STEP = 0>
__device__ __forceinline__ void run_best(double& k, int& i) {
  if constexpr ((1 << STEP) < G) {
    double ka, kb;
    int ia, ib;
    both<STEP>(k, ka, kb);
    both<STEP>(i, ia, ib);
    const bool take = kb > ka || (kb == ka && ib < ia);
    k = take ? kb : ka;
    i = take ? ib : ia;
    run_best<G, STEP + 1>(k, i);
  }
}

// exp(l - base) for a softmax; sigmoid(l) exp(-base) for a sigmoid, base the
// best of the chosen logits where that is below 0 (then every l is), else 0:
// ratios of scores that would vanish by themselves.
__device__ __forceinline__ float choice_score(int score, float l, float base) {
  if (score == 0) return __expf(l - base);
  const float e = __expf(-__builtin_fabsf(l));
  return (l >= 0.f ? 1.f : base < 0.f ? __expf(l - base) : e) * __builtin_amdgcn_rcpf(1.f + e);
}

// The two largest values of runs of `width` (a power of two) lanes.
template <int STEP, typename T>
__device__ __forceinline__ void top2_step(T& k1, T& k2) {
  T a1, b1, a2, b2;
  both<STEP>(k1, a1, b1);
  both<STEP>(k2, a2, b2);
  k2 = larger(smaller(a1, b1), larger(a2, b2));
  k1 = larger(a1, b1);
}
template <typename T>
__device__ __forceinline__ void run_top2(T& k1, T& k2, int width) {
  if (width > 1) top2_step<0>(k1, k2);
  if (width > 2) top2_step<1>(k1, k2);
  if (width > 4) top2_step<2>(k1, k2);
  if (width > 8) top2_step<3>(k1, k2);
  if (width > 16) top2_step<4>(k1, k2);
  if (width > 32) top2_step<5>(k1, k2);
}

// Sorts a lane's EPL (key, index) pairs by falling key, equal keys in order
// (odd-even transposition: only neighbours change places).
template <int EPL, typename T, int R = 0, int I = 0>
__device__ __forceinline__ void sort_pairs(T* key, int* idx) {
  if constexpr (R < EPL) {
    if constexpr (I + 1 < EPL) {
      const bool sw = key[I + 1] > key[I];
      const T ka = larger(key[I], key[I + 1]), kb = smaller(key[I], key[I + 1]);
      const int ia = sw ? idx[I + 1] : idx[I], ib = sw ? idx[I] : idx[I + 1];
      key[I] = ka;
      key[I + 1] = kb;
      idx[I] = ia;
      idx[I + 1] = ib;
      sort_pairs<EPL, T, R, I + 2>(key, idx);
    } else {
      sort_pairs<EPL, T, R + 1, (R + 1) & 1>(key, idx);
    }
  }
}

// Sorts a lane's EPL keys by falling value: Batcher's odd-even merges (19
// exchanges of 8 keys), unrolled in the types so that keys stay in registers.
template <int EPL, int P = 1, int K = 1, int J = 0, int I = 0>
__device__ __forceinline__ void sort_keys(int* key) {
  if constexpr (P < EPL) {
    if constexpr (K < 1) {
      sort_keys<EPL, 2 * P, 2 * P, 0, 0>(key);
    } else if constexpr (J + K >= EPL) {
      sort_keys<EPL, P, K / 2, (K / 2) % P, 0>(key);
    } else if constexpr (I >= K || I + J + K >= EPL) {
      sort_keys<EPL, P, K, J + 2 * K, 0>(key);
    } else {
      if constexpr ((I + J) / (2 * P) == (I + J + K) / (2 * P)) {
        const int a = larger(key[I + J], key[I + J + K]), b = smaller(key[I + J], key[I + J + K]);
        key[I + J] = a;
        key[I + J + K] = b;
      }
      sort_keys<EPL, P, K, J, I + 1>(key);
    }
  }
}

// What a run of G lanes knows of its token: its groups ranked.  LDS lkey
// holds the token's ranking values (T), from which lane gl takes every
// width-th of group gl / width.  Leaves the group's two best values in k1
// and k2 of its lanes and returns its score.
template <int G, typename T>
__device__ __forceinline__ T group_scores(const RouteArgs& a, const T* lkey, bool top2, int gl, T& k1, T& k2) {
  const T none = -(T)__builtin_inff();
  const int width = 1 << a.log_width, grp = gl >> a.log_width;
  k1 = k2 = none;
  if (grp < a.groups)
#pragma clang loop unroll(disable)
    for (int i = gl - (grp << a.log_width); i < a.per; i += width) {
      const T k = lkey[grp * a.per + i];
      k2 = larger(k2, smaller(k1, k));
      k1 = larger(k1, k);
    }
  run_top2(k1, k2, width);
  return top2 && k2 > none ? k1 + k2 : k1;
}

// Bit g * width of the run's lanes: group g stays.
template <int EPL, typename T>
__device__ __forceinline__ void drop_groups(const RouteArgs& a, unsigned long long kept, int e0, int shift, T* key) {
  int g = group_of(a, e0), rem = e0 - g * a.per;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    if (g >= a.groups || !((kept >> (shift + (g << a.log_width))) & 1)) key[i] = -(T)__builtin_inff();
    if (++rem == a.per) {
      rem = 0;
      ++g;
    }
  }
}

// The top_k experts of a run whose lanes hold their keys as sort_pairs leaves
// them, above nokey where there is an expert: into sel, -1 where there is
// none.  Equal keys go by lane, and so by expert.
template <int G, int EPL, typename T>
__device__ __forceinline__ void choose(T* key, const int* idx, T nokey, int top_k, int e0, int gl, int sub, int* sel) {
  uint64_t order = 0;                 // the lane's experts in the order of its keys, 4 bits each
#pragma unroll
  for (int i = 0; i < EPL; ++i) order |= (uint64_t)(uint32_t)idx[i] << (4 * i);
#pragma clang loop unroll(disable)
  for (int r = gl; r < top_k; r += G) sel[r] = -1;
  wave_fence();
#pragma clang loop unroll(disable)
  for (int r = 0; r < top_k; ++r) {
    const T w = run_max<G>(key[0]);
    const bool best = w > nokey && key[0] == w;
    const unsigned long long eq = __builtin_amdgcn_ballot_w64(best);
    const unsigned long long run = G == 64 ? eq : (eq >> (sub * G)) & ((1ull << (G & 63)) - 1);
    if (best && __builtin_ctzll(run) == gl) {
      sel[r] = e0 + (int)(order & 15);
      order >>= 4;
#pragma unroll
      for (int i = 0; i + 1 < EPL; ++i) key[i] = key[i + 1];
      key[EPL - 1] = nokey;
    }
  }
}

// The wave's tokens again with keys in double precision: sel as the fp32
// pass below leaves it.
template <int G, int EPL, bool SCORED, bool GROUPS>
__device__ __forceinline__ void select_exact(const RouteArgs& a, const float* l, const float* bias, float mx, int gl,
                                             int sub, double* lkey, int* sel) {
  const double none = -__builtin_inf();
  const int e0 = gl * EPL;
  const bool top2 = GROUPS && a.group_score == 1;
  double key[EPL], z = 0.0;
  if (a.score == 0) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      key[i] = l[i] > -__builtin_inff() ? exp((double)l[i] - (double)mx) : 0.0;
      z += key[i];
    }
    z = run_add<G>(z);
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = key[i] / z;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = 1.0 / (1.0 + exp(-(double)l[i]));
  }
  const bool heads = SCORED && GROUPS && a.log_heads >= 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const bool in = l[i] > -__builtin_inff();
    const double rank = in ? (SCORED ? key[i] + (double)bias[i] : top2 ? key[i] : (double)l[i]) : none;
    if (GROUPS && !heads) lkey[e0 + i] = rank;
    key[i] = SCORED ? rank : (double)l[i];
  }
  int idx[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) idx[i] = i;
  if (heads) sort_pairs<EPL>(key, idx);
  if constexpr (GROUPS) {
    wave_fence();
    const int log_width = heads ? a.log_heads : a.log_width, grp = gl >> log_width;
    double k1, k2, score;
    if (heads) {
      k1 = key[0];
      k2 = key[1];
      run_top2(k1, k2, 1 << log_width);
      score = top2 && k2 > none ? k1 + k2 : k1;
    } else {
      score = group_scores<G>(a, lkey, top2, gl, k1, k2);
    }
    int better = 0;
#pragma clang loop unroll(disable)
    for (int j = 0; j < a.groups; ++j) {
      const double o = __shfl(score, sub * G + (j << log_width), 64);
      better += o > score || (o == score && j < grp);
    }
    const bool stays = grp < a.groups && better < a.topk_groups;
    if (heads)
      key[0] = stays ? key[0] : none;
    else
      drop_groups<EPL>(a, __builtin_amdgcn_ballot_w64(stays), e0, sub * G, key);
  }
  if (!heads) sort_pairs<EPL>(key, idx);
  choose<G, EPL>(key, idx, none, a.top_k, e0, gl, sub, sel);
}

// EPL consecutive values of a row from expert e0 on, -inf past the last
// expert.  vec: experts % 4 == 0 and aligned for four values at a time, which
// are then all within the row or all past it.
template <int EPL>
__device__ __forceinline__ void load_logits(const void* logits, bool f32, int E, int64_t row, int e0, bool vec,
                                            float* l) {
  static_assert(EPL % 4 == 0, "four at a time");
  if (vec) {
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
      const bool in = e0 + i < E;
      const int64_t at = row + (in ? e0 + i : E - 4);
      if (f32) {
        const v4f v = *reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(logits) + at);
#pragma unroll
        for (int j = 0; j < 4; ++j) l[i + j] = v[j];
      } else {
        const u32x2 w = *reinterpret_cast<const u32x2*>(reinterpret_cast<const uint16_t*>(logits) + at);
        l[i] = bf_lo(w.x);
        l[i + 1] = bf_hi(w.x);
        l[i + 2] = bf_lo(w.y);
        l[i + 3] = bf_hi(w.y);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) l[i + j] = in ? l[i + j] : -__builtin_inff();
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      l[i] = load_logit(logits, f32, row + (e0 + i < E ? e0 + i : E - 1));
      l[i] = e0 + i < E ? l[i] : -__builtin_inff();
    }
  }
}

// Bound by the vector instructions and the latency of top_k dependent
// rounds, not by reading the logits: 16384 tokens of 256 experts, top 8, take
// 11 us (1.5 TB/s) plain and 18 us with a bias and groups.
//
// G lanes per token (64 / G tokens per wave), EPL consecutive experts per
// lane.  Keys are ints of the order of the fp32 ranking values, sorted within
// each lane; a round takes the largest head of a run of G lanes (a butterfly)
// and moves that lane's list on.
//
// Where keys are scores, the low bits of a key hold its expert's place in the
// lane, which makes an exchange of the sort two instructions (with the place
// beside the key, five) and leaves kKeyErr of the key's precision; the fp32
// score is off by at most serr (below).  A choice between keys further apart
// than twice both is the one double precision makes; a wave with a closer one
// chooses again in double precision (about a hundred of 16384 tokens of 256
// experts, whose tail is 4 of the 18 us).  Groups that whole lanes make up
// are ranked from the heads of the sorted lists (16384 tokens, 8 groups of
// 32: 18.7 us, through LDS 22.4), others through LDS.
template <int G, int EPL, bool SCORED, bool GROUPS>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a, int vec, int64_t t0) {
  extern __shared__ double smem[];
  constexpr int TPW = 64 / G;
  const int lane = (int)(threadIdx.x & 63), wave = (int)(threadIdx.x >> 6);
  const int gl = lane & (G - 1), sub = lane / G;
  const float none = -__builtin_inff();
  const int E = a.experts;
  // per wave: 64 EPL keys (floats, or doubles where it chooses again), TPW * 64 choices
  constexpr int kKeyBytes = 64 * EPL * 8;
  uint8_t* mine = reinterpret_cast<uint8_t*>(smem) + wave * (kKeyBytes + TPW * 256);
  float* lkey = reinterpret_cast<float*>(mine) + sub * (G * EPL);
  int* sel = reinterpret_cast<int*>(mine + kKeyBytes) + sub * 64;
  const bool top2 = GROUPS && a.group_score == 1;
  const int e0 = gl * EPL;
  // a ranking value's distance from its key, relative
  constexpr float kKeyErr = SCORED ? EPL * 0x1p-23f : 0.f;

  const int64_t tw = t0 + ((int64_t)blockIdx.x * 4 + wave) * TPW;    // this wave's first token
  if (tw >= a.tokens) return;
  const int64_t t = tw + sub;
  const bool live = t < a.tokens;
  float l[EPL], bias[EPL], rank[EPL], s[EPL];
  load_logits<EPL>(a.logits, a.logits_f32, E, (live ? t : a.tokens - 1) * E, e0, (vec & 1) != 0, l);
  if constexpr (SCORED) load_logits<EPL>(a.bias, true, E, 0, e0, (vec & 2) != 0, bias);
#pragma unroll
  for (int i = 0; i < EPL; ++i) l[i] = clean(l[i]);
  float mx = l[0];
#pragma unroll
  for (int i = 1; i < EPL; ++i) mx = __builtin_fmaxf(mx, l[i]);
  float z = 1.f, pmax = 1.f;
  if (a.score == 0) {
    mx = run_max<G>(mx);
    z = 0.f;
    const float m = mx > none ? mx : 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      s[i] = __expf(l[i] - m);
      z += s[i];
    }
    z = run_add<G>(z);
    const float r = 1.f / z;
    pmax = r;
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] *= r;
  } else if (SCORED || top2) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] = __builtin_amdgcn_rcpf(1.f + __expf(-l[i]));
  }
  // |fp32 score - score| : sigmoid, s (1 - s) (|l| + 1) 2^-23 and two
  // roundings of s, below 2^-22; softmax, a probability p from a logit d
  // below the best is off by p (|d| + 8 + 22) 2^-23 (the difference's and
  // the exponential's rounding, the others' through the sum, the sum
  // itself), below pmax 2^-17.  The bias adds half a step of the key.
  const float serr = a.score == 0 ? pmax * 0x1p-17f + 0x1p-23f : 0x1p-21f;
  bool close = false;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    if constexpr (SCORED) bias[i] = clean(bias[i]);
    rank[i] = SCORED ? (l[i] > none ? s[i] + bias[i] : none) : l[i] + 0.f;      // -0 is 0
  }
  int key[EPL], idx[EPL];
  const int nokey = ordered(none);       // keys up to this one are no keys
  const bool heads = SCORED && GROUPS && a.log_heads >= 0;
  auto make_keys = [&]() {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      key[i] = SCORED ? (ordered(rank[i]) & -EPL) | i : ordered(rank[i]);
      idx[i] = i;
    }
    if constexpr (SCORED)
      sort_keys<EPL>(key);
    else
      sort_pairs<EPL>(key, idx);
  };
  if constexpr (GROUPS) {
    const int log_width = heads ? a.log_heads : a.log_width, grp = gl >> log_width;
    float score, k1, k2;
    if (heads) {
      make_keys();
      int i1 = key[0], i2 = key[1];
      run_top2(i1, i2, 1 << log_width);
      k1 = i1 > nokey ? unordered(i1) : none;
      k2 = i2 > nokey ? unordered(i2) : none;
      score = top2 && k2 > none ? k1 + k2 : k1;
    } else {
      // keys to LDS, then `width` lanes per group
      wave_fence();
#pragma unroll
      for (int i = 0; i < EPL; ++i) lkey[e0 + i] = SCORED || !top2 ? rank[i] : (l[i] > none ? s[i] : none);
      wave_fence();
      score = group_scores<G>(a, lkey, top2, gl, k1, k2);
    }
    // twice a group's error: two keys' and half a step of their sum, at most
    // a step of the larger (each pair of groups is looked at from both sides)
    const float size = __builtin_fmaxf(__builtin_fabsf(k1), k2 > none ? __builtin_fabsf(k2) : 0.f);
    const float gerr = (SCORED || top2) ? 4.f * (serr + (kKeyErr + 0x1p-23f) * size) : -1.f;
    int better = 0, near = 0;
#pragma clang loop unroll(disable)
    for (int j = 0; j < a.groups; ++j) {
      const float o = __shfl(score, sub * G + (j << log_width), 64);
      better += o > score || (o == score && j < grp);
      // sums that leave the fp32 range differ by NaN and are close
      near += !(__builtin_fabsf(o - score) > gerr);
    }
    close = near > 1 && grp < a.groups && k1 > none;        // one of them is the group itself
    const bool stays = grp < a.groups && better < a.topk_groups;
    if (heads) {
      key[0] = stays ? key[0] : nokey;
    } else {
      drop_groups<EPL>(a, __builtin_amdgcn_ballot_w64(stays), e0, sub * G, rank);
      make_keys();
    }
  } else {
    make_keys();
  }
  if constexpr (SCORED) {
    float last = __builtin_inff(), gap = __builtin_inff();
    auto look = [&](int w) {
      const float f = unordered(w);       // NaN where there is no key, which fminf passes over
      gap = __builtin_fminf(gap, __builtin_fmaf(-2.f * kKeyErr - 0x1p-22f, __builtin_fabsf(f), last - f));
      last = f;
    };
    bool tie = false;
#pragma clang loop unroll(disable)
    for (int r = gl; r < a.top_k; r += G) sel[r] = -1;
    wave_fence();
#pragma clang loop unroll(disable)
    for (int r = 0; r < a.top_k; ++r) {
      const int w = run_max<G>(key[0]);
      look(w);
      const bool any = w > nokey, first = any && key[0] == w;
      // runs with a key have one lane with it, or a tie
      tie = tie || __builtin_popcountll(__builtin_amdgcn_ballot_w64(first)) * G !=
                       __builtin_popcountll(__builtin_amdgcn_ballot_w64(any));
      if (first) {
        sel[r] = e0 + (key[0] & (EPL - 1));
#pragma unroll
        for (int i = 0; i + 1 < EPL; ++i) key[i] = key[i + 1];
        key[EPL - 1] = nokey;
      }
    }
    look(run_max<G>(key[0]));   // the first one left out
    close = close || tie || gap <= 2.f * serr;
  } else {
    choose<G, EPL>(key, idx, nokey, a.top_k, e0, gl, sub, sel);
  }
  wave_fence();
  if constexpr (SCORED || GROUPS) {
    if (__builtin_amdgcn_ballot_w64(close && live) != 0) {
      select_exact<G, EPL, SCORED, GROUPS>(a, l, bias, mx, gl, sub,
                                           reinterpret_cast<double*>(mine) + sub * (G * EPL), sel);
      wave_fence();
    }
  }
  // weights: lane gl has choice gl, and gl + G, ... where top_k is larger
  const int64_t row = (live ? t : 0) * E;
  auto chosen_logit = [&](int r) {
    const int e = r < a.top_k ? sel[r] : -1;
    return e >= 0 ? clean(load_logit(a.logits, a.logits_f32, row + e)) : none;
  };
  auto choice = [&](float v, float base) { return v > none ? choice_score(a.score, v, base) : 0.f; };
  const float c0 = chosen_logit(gl);
  float base = a.score == 0 ? mx : 0.f, norm = a.score == 0 ? a.scale / z : a.scale;
  if (a.renorm) {
    float top = c0;
#pragma clang loop unroll(disable)
    for (int r = gl + G; r < a.top_k; r += G) top = __builtin_fmaxf(top, chosen_logit(r));
    top = run_max<G>(top);
    base = a.score == 0 || top < 0.f ? top : 0.f;
    float sum = choice(c0, base);
#pragma clang loop unroll(disable)
    for (int r = gl + G; r < a.top_k; r += G) sum += choice(chosen_logit(r), base);
    sum = run_add<G>(sum);
    norm = a.scale / sum;
  }
  if (live)
#pragma clang loop unroll(disable)
    for (int r = gl; r < a.top_k; r += G) {
      const float c = r == gl ? c0 : chosen_logit(r);
      a.ids[t * a.top_k + r] = sel[r];
      a.weights[t * a.top_k + r] = c > none ? choice(c, base) * norm : 0.f;
    }
}

// With v_j = scale * dw_j over the valid choices:
//   sigmoid: dl = (v_j - [renorm] <v, s> / S) / [renorm] S * s (1 - s)
//   softmax: dl = s (ds - <ds, s>), ds as above; with renorm <ds, s> = 0
//            and the weights are a softmax over the choices alone
// G lanes per token (at least top_k: lane gl holds choice gl), EPL
// consecutive experts per lane, as in route_kernel; chosen logits and their
// gradients change lanes through LDS.  Bound by latency for a few thousand
// tokens (4099 x 160 bf16: 4.8 us), then by its instructions: 16384 x 256
// fp32 takes 13 us with softmax (2.6 TB/s) and 11 us renormalized.
template <int G, int EPL>
__global__ __launch_bounds__(256) void route_bwd_kernel(RouteBwdArgs a, int vec, int64_t t0) {
  extern __shared__ float smemf[];
  constexpr int TPW = 64 / G;
  const int lane = (int)(threadIdx.x & 63), wave = (int)(threadIdx.x >> 6);
  const int gl = lane & (G - 1), sub = lane / G;
  const float none = -__builtin_inff();
  const int E = a.experts, e0 = gl * EPL;
  float* mine = smemf + (size_t)(wave * TPW + sub) * (G * EPL);
  const int64_t tw = t0 + ((int64_t)blockIdx.x * 4 + wave) * TPW;    // this wave's first token
  if (tw >= a.tokens) return;
  const bool live = tw + sub < a.tokens;
  const int64_t t = live ? tw + sub : a.tokens - 1;
  float l[EPL];
  load_logits<EPL>(a.logits, a.logits_f32, E, t * E, e0, vec != 0, l);
  int id = -1;
  float v = 0.f;
  if (gl < a.top_k) {
    id = a.ids[t * a.top_k + gl];
    v = a.scale * a.dweights[t * a.top_k + gl];
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    l[i] = clean(l[i]);
    mine[e0 + i] = l[i];
  }
  wave_fence();
  float cl = none;
  if (id >= 0 && id < E) cl = mine[id];
  const bool ok = cl > none;        // neither left out nor masked
  wave_fence();
#pragma unroll
  for (int i = 0; i < EPL; ++i) mine[e0 + i] = 0.f;
  float mx = 0.f, z = 1.f;
  float s[EPL];
  const bool whole = a.score == 0 && !a.renorm;     // the gradient reaches every expert
  if (whole) {
    mx = l[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) mx = __builtin_fmaxf(mx, l[i]);
    mx = run_max<G>(mx);
    mx = mx > none ? mx : 0.f;
    z = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      s[i] = expf(l[i] - mx);
      z += s[i];
    }
    z = run_add<G>(z);
  }
  float dl = 0.f, back = 0.f;
  if (a.renorm) {
    const float top = run_max<G>(cl);
    const float base = a.score == 0 || top < 0.f ? top : 0.f;
    const float c = ok ? choice_score(a.score, cl, base) : 0.f;
    const float sum = run_add<G>(c);
    const float p = ok ? c / sum : 0.f;            // the weight before scale
    const float mean = run_add<G>(ok ? v * p : 0.f);
    dl = ok ? p * (v - mean) : 0.f;
    if (a.score == 1 && ok) dl *= 1.f / (1.f + expf(cl));
  } else if (ok) {
    const float c = a.score == 0 ? expf(cl - mx) / z : 1.f / (1.f + expf(-cl));
    dl = v * c;
    if (a.score == 1) dl *= 1.f / (1.f + expf(cl));
  }
  if (whole) back = run_add<G>(dl);
  wave_fence();
  // An expert listed twice adds up: its first lane takes the sum, in the
  // order of the choices.
  bool twice = false;
  for (int j = 1; j < a.top_k; ++j) {
    const int other = __shfl(id, sub * G + ((gl + j) & (G - 1)), 64);
    twice = twice || (ok && other == id && ((gl + j) & (G - 1)) < a.top_k);
  }
  if (__builtin_amdgcn_ballot_w64(twice) == 0) {
    if (ok) mine[id] = dl;
  } else {
#pragma clang loop unroll(disable)
    for (int j = 0; j < a.top_k; ++j) {
      if (gl == j && ok) mine[id] += dl;
      wave_fence();
    }
  }
  wave_fence();
  if (!live) return;
  float d[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    d[i] = mine[e0 + i];
    if (whole && l[i] > none) d[i] -= back * (s[i] / z);
  }
  if (vec) {
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
      if (e0 + i >= E) continue;
      if (a.logits_f32) {
        *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.dlogits) + t * E + e0 + i) =
            (v4f){d[i], d[i + 1], d[i + 2], d[i + 3]};
      } else {
        *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(a.dlogits) + t * E + e0 + i) =
            (u32x2){pack_bf16x2(d[i], d[i + 1]), pack_bf16x2(d[i + 2], d[i + 3])};
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if (e0 + i >= E) continue;
      if (a.logits_f32)
        reinterpret_cast<float*>(a.dlogits)[t * E + e0 + i] = d[i];
      else
        reinterpret_cast<uint16_t*>(a.dlogits)[t * E + e0 + i] = (uint16_t)pack_bf16x2(d[i], 0.f);
    }
  }
}

// ---------------------------------------------------------------------- plan

// A stable counting sort of the pairs by expert, 2048 pairs (a run) per
// workgroup: plan_count_kernel counts each run's pairs per expert, then
// plan_place_kernel places them after those of lower experts and of earlier
// runs.  Up to kDirectRuns runs a workgroup adds up the other runs' counts
// by itself (64 runs of 256 experts: fewer launches and 64 loads per
// thread); for more, plan_scan_kernel turns the counts into running sums
// first.  A single run counts and places in one launch.  Bound by latency and
// LDS: 131072 pairs of 256 experts, count 3.9 us and place 7.9 us.
constexpr int kPlanThreads = 512;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPlanItems = 4;                              // pairs per lane
constexpr int kPlanRun = kPlanThreads * kPlanItems;
constexpr int kDirectRuns = 128;

__global__ __launch_bounds__(kPlanThreads) void plan_count_kernel(const int32_t* __restrict__ ids, int pairs, int E,
                                                                  int32_t* __restrict__ counts) {
  __shared__ int hist[1024];
  const int t = (int)threadIdx.x;
  const int64_t lo = (int64_t)blockIdx.x * kPlanRun;
  int id[kPlanItems];
#pragma unroll
  for (int k = 0; k < kPlanItems; ++k) {
    const int64_t i = lo + k * kPlanThreads + t;
    id[k] = i < pairs ? ids[i] : -1;
  }
  for (int e = t; e < E; e += kPlanThreads) hist[e] = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPlanItems; ++k)
    if (id[k] >= 0 && id[k] < E) atomicAdd(&hist[id[k]], 1);
  __syncthreads();
  for (int e = t; e < E; e += kPlanThreads) counts[(int64_t)blockIdx.x * E + e] = hist[e];
}

// Counts of `runs` runs into the sums of the runs before, and their total
// into row `runs`: 64 experts per workgroup, each of its 16 waves a stretch
// of the runs.
__global__ __launch_bounds__(1024) void plan_scan_kernel(int32_t* __restrict__ counts, int runs, int E) {
  __shared__ int part[16][64];
  const int lane = (int)(threadIdx.x & 63), wave = (int)(threadIdx.x >> 6);
  const int e = (int)blockIdx.x * 64 + lane;
  const int len = (runs + 15) / 16;
  const int lo = wave * len, hi = lo + len < runs ? lo + len : runs;
  int sum = 0;
  if (e < E)
    for (int r = lo; r < hi; ++r) sum += counts[(int64_t)r * E + e];
  part[wave][lane] = sum;
  __syncthreads();
  int at = 0, total = 0;
  for (int w = 0; w < 16; ++w) {
    at += w < wave ? part[w][lane] : 0;
    total += part[w][lane];
  }
  if (e >= E) return;
  for (int r = lo; r < hi; ++r) {
    const int c = counts[(int64_t)r * E + e];
    counts[(int64_t)r * E + e] = at;
    at += c;
  }
  if (wave == 0) counts[(int64_t)runs * E + e] = total;
}

// scanned: counts hold running sums (plan_scan_kernel).
__global__ __launch_bounds__(kPlanThreads) void plan_place_kernel(const int32_t* __restrict__ ids, int pairs,
                                                                  int top_k, int E, int bits, int scanned,
                                                                  const int32_t* __restrict__ counts,
                                                                  int32_t* __restrict__ offsets,
                                                                  int32_t* __restrict__ row_index,
                                                                  int32_t* __restrict__ slot) {
  extern __shared__ int smemi[];
  __shared__ int all;                      // rows of all experts
  int* total = smemi;                      // [E] rows of each expert, then those of the experts before it
  int* before = smemi + E;                 // [E] rows of each expert in the runs before this one
  const int t = (int)threadIdx.x, lane = t & 63, wave = t >> 6;
  int* ctr = smemi + (2 + wave) * E;       // [E] of this wave
  const int runs = (int)gridDim.x, run = (int)blockIdx.x;
  // wave w holds the w-th eighth of the run, 64 pairs at a time, in order
  const int64_t lo = (int64_t)run * kPlanRun + wave * (64 * kPlanItems) + lane;
  int id[kPlanItems], rank[kPlanItems];
#pragma unroll
  for (int k = 0; k < kPlanItems; ++k) id[k] = lo + k * 64 < pairs ? ids[lo + k * 64] : -1;
  for (int e = lane; e < E; e += 64) ctr[e] = 0;
  for (int e = t; e < E; e += kPlanThreads) {
    int tot = 0, bef = 0;
    if (scanned) {
      bef = counts[(int64_t)run * E + e];
      tot = counts[(int64_t)runs * E + e];
    } else if (runs > 1) {
#pragma unroll 16
      for (int r = 0; r < runs; ++r) {
        const int c = counts[(int64_t)r * E + e];
        bef += r < run ? c : 0;
        tot += c;
      }
    }
    total[e] = tot;
    before[e] = bef;
  }
  wave_fence();
#pragma unroll
  for (int k = 0; k < kPlanItems; ++k) {
    const bool ok = id[k] >= 0 && id[k] < E;
    // lanes of the wave with the same expert
    unsigned long long same = __builtin_amdgcn_ballot_w64(ok);
    rank[k] = -1;
    if (same == 0) continue;
    for (int b = 0; b < bits; ++b) {
      const bool one = (id[k] >> b) & 1;
      const unsigned long long set = __builtin_amdgcn_ballot_w64(one);
      same &= one ? set : ~set;
    }
    if (ok) {
      rank[k] = ctr[id[k]] + __builtin_popcountll(same & ((1ull << lane) - 1));
      // the last of them moves the counter on (after every lane has read it)
      if ((same >> lane) == 1ull) ctr[id[k]] = rank[k] + 1;
    }
    wave_fence();
  }
  __syncthreads();
  // the waves' counters into their first ranks
  for (int e = t; e < E; e += kPlanThreads) {
    int at = 0;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      const int c = smemi[(2 + w) * E + e];
      smemi[(2 + w) * E + e] = at;
      at += c;
    }
    if (runs == 1) total[e] = at;
  }
  __syncthreads();
  if (wave == 0) {
    const int per = (E + 63) / 64, e0 = lane * per;
    int sum = 0;
    for (int i = 0; i < per; ++i) sum += e0 + i < E ? total[e0 + i] : 0;
    int upto = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(upto, d, 64);
      upto += lane >= d ? o : 0;
    }
    int at = upto - sum;
    for (int i = 0; i < per; ++i)
      if (e0 + i < E) {
        const int c = total[e0 + i];
        total[e0 + i] = at;
        if (run == 0) offsets[e0 + i] = at;
        at += c;
      }
    if (lane == 63) {
      all = upto;
      if (run == 0) offsets[E] = upto;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPlanItems; ++k) {
    const int64_t i = lo + k * 64;
    if (rank[k] >= 0) {
      const int at = total[id[k]] + before[id[k]] + ctr[id[k]] + rank[k];
      slot[i] = at;
      row_index[at] = (int)((uint32_t)i / (uint32_t)top_k);
    } else if (i < pairs) {
      slot[i] = -1;
    }
    // places behind the last row belong to nobody
    if (i >= all && i < pairs) row_index[i] = 0;
  }
}

int64_t plan_runs(int64_t pairs) { return pairs <= kPlanRun ? 1 : (pairs + kPlanRun - 1) / kPlanRun; }

}  // namespace

int64_t plan_workspace_bytes(int64_t pairs, int experts) {
  const int64_t runs = plan_runs(pairs);
  return runs == 1 ? 0 : (runs + 1) * experts * 4;
}

template <int G, int EPL, bool SCORED, bool GROUPS>
static void launch_route_as(const RouteArgs& a, int vec, hipStream_t stream) {
  constexpr int kTokens = 4 * (64 / G);
  for (int64_t t0 = 0; t0 < a.tokens; t0 += kMaxGrid * kTokens) {
    const int64_t wgs = (a.tokens - t0 + kTokens - 1) / kTokens;
    hipLaunchKernelGGL((route_kernel<G, EPL, SCORED, GROUPS>), dim3((unsigned)(wgs < kMaxGrid ? wgs : kMaxGrid)),
                       dim3(256), (size_t)4 * (64 * EPL * 8 + (64 / G) * 256), stream, a, vec, t0);
  }
}
template <int G, int EPL>
static void launch_route_as(const RouteArgs& a, int vec, hipStream_t stream) {
  if (a.bias && a.groups > 1) launch_route_as<G, EPL, true, true>(a, vec, stream);
  else if (a.bias) launch_route_as<G, EPL, true, false>(a, vec, stream);
  else if (a.groups > 1) launch_route_as<G, EPL, false, true>(a, vec, stream);
  else launch_route_as<G, EPL, false, false>(a, vec, stream);
}

hipError_t launch_route(const RouteArgs& args, hipStream_t stream) {
  RouteArgs a = args;
  const bool fours = a.experts % 4 == 0;
  const int vec = (fours && (reinterpret_cast<uintptr_t>(a.logits) & (a.logits_f32 ? 15 : 7)) == 0 ? 1 : 0) |
                  (fours && (reinterpret_cast<uintptr_t>(a.bias) & 15) == 0 ? 2 : 0);
  // Experts per lane: four up to 256 experts; eight for many tokens, where
  // the butterflies over fewer lanes count (16384 tokens of 256 experts: 11.0
  // us against 12.7, of 128: 6.3 against 7.3; sixteen: 12.9 us) and the longer
  // lists' latency does not (1024 tokens: 4.2 us against 3.8, 9.6 against 7.3
  // with groups).
  const int epl = a.experts > 512 ? 16 : a.experts > 256 || (a.experts > 64 && a.tokens >= 4096) ? 8 : 4;
  int lanes = 8;                        // per token, and one per group at least
  while (lanes < 64 && (lanes * epl < a.experts || lanes < a.groups)) lanes *= 2;
  a.per = a.experts / a.groups;
  a.inv_per = 1.0f / (float)a.per;
  a.log_width = 0;
  while ((2 << a.log_width) * a.groups <= lanes) ++a.log_width;
  a.log_heads = -1;
  for (int w = 0; epl << w <= a.per; ++w)
    if (epl << w == a.per) a.log_heads = w;
  if (epl == 16) launch_route_as<64, 16>(a, vec, stream);
  else if (epl == 8 && lanes == 64) launch_route_as<64, 8>(a, vec, stream);
  else if (epl == 8 && lanes == 32) launch_route_as<32, 8>(a, vec, stream);
  else if (epl == 8) launch_route_as<16, 8>(a, vec, stream);
  else if (lanes == 64) launch_route_as<64, 4>(a, vec, stream);
  else if (lanes == 32) launch_route_as<32, 4>(a, vec, stream);
  else if (lanes == 16) launch_route_as<16, 4>(a, vec, stream);
  else launch_route_as<8, 4>(a, vec, stream);
  return hipGetLastError();
}

template <int G, int EPL>
static void launch_route_bwd_as(const RouteBwdArgs& a, bool vec, hipStream_t stream) {
  constexpr int kTokens = 4 * (64 / G);
  for (int64_t t0 = 0; t0 < a.tokens; t0 += kMaxGrid * kTokens) {
    const int64_t wgs = (a.tokens - t0 + kTokens - 1) / kTokens;
    hipLaunchKernelGGL((route_bwd_kernel<G, EPL>), dim3((unsigned)(wgs < kMaxGrid ? wgs : kMaxGrid)), dim3(256),
                       (size_t)4 * 64 * EPL * 4, stream, a, vec ? 1 : 0, t0);
  }
}

hipError_t launch_route_bwd(const RouteBwdArgs& a, hipStream_t stream) {
  const uintptr_t both = reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.dlogits);
  const bool vec = a.experts % 4 == 0 && (both & (a.logits_f32 ? 15 : 7)) == 0;
  const int epl = a.experts > 512 ? 16 : a.experts > 256 ? 8 : 4;
  int lanes = 8;                        // per token: one per choice at least
  while (lanes < 64 && (lanes * epl < a.experts || lanes < a.top_k)) lanes *= 2;
  if (epl == 16) launch_route_bwd_as<64, 16>(a, vec, stream);
  else if (epl == 8) launch_route_bwd_as<64, 8>(a, vec, stream);
  else if (lanes == 64) launch_route_bwd_as<64, 4>(a, vec, stream);
  else if (lanes == 32) launch_route_bwd_as<32, 4>(a, vec, stream);
  else if (lanes == 16) launch_route_bwd_as<16, 4>(a, vec, stream);
  else launch_route_bwd_as<8, 4>(a, vec, stream);
  return hipGetLastError();
}

hipError_t launch_plan(const int32_t* ids, int64_t tokens, int top_k, int experts, void* workspace, int32_t* offsets,
                       int32_t* row_index, int32_t* slot, hipStream_t stream) {
  const int pairs = (int)(tokens * top_k);
  const int runs = (int)plan_runs(pairs);
  int bits = 0;
  while ((1 << bits) < experts) ++bits;
  int32_t* counts = reinterpret_cast<int32_t*>(workspace);
  const dim3 grid((unsigned)runs), block(kPlanThreads);
  const int scanned = runs > kDirectRuns ? 1 : 0;
  if (runs > 1) hipLaunchKernelGGL(plan_count_kernel, grid, block, 0, stream, ids, pairs, experts, counts);
  if (scanned)
    hipLaunchKernelGGL(plan_scan_kernel, dim3((unsigned)((experts + 63) / 64)), dim3(1024), 0, stream, counts, runs,
                       experts);
  hipLaunchKernelGGL(plan_place_kernel, grid, block, (size_t)(2 + kPlanWaves) * experts * 4, stream, ids, pairs, top_k,
                     experts, bits, scanned, counts, offsets, row_index, slot);
  return hipGetLastError();
}

}  // namespace fp8blk
