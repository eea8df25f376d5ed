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
constexpr int kTokensPerWg = 4;

__device__ __forceinline__ float load_logit(const void* l, bool f32, int64_t i) {
  if (f32) return reinterpret_cast<const float*>(l)[i];
  return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(l)[i] << 16);
}

template <typename T>
__device__ __forceinline__ T wave_add(T v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// Best (key, index) over the wave: highest key, lowest index among equals.
__device__ __forceinline__ void wave_best(double& k, int& i) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double ok = __shfl_xor(k, d, 64);
    const int oi = __shfl_xor(i, d, 64);
    if (ok > k || (ok == k && oi < i)) {
      k = ok;
      i = oi;
    }
  }
}

// One wave per token; its keys in LDS.
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
  extern __shared__ double smem[];
  const int lane = (int)(threadIdx.x & 63), wave = (int)(threadIdx.x >> 6);
  const int E = a.experts;
  double* key = smem + (size_t)wave * E;
  const double none = -__builtin_inf();
  for (int64_t t = (int64_t)blockIdx.x * kTokensPerWg + wave; t < a.tokens; t += (int64_t)gridDim.x * kTokensPerWg) {
  double mx = none;
  for (int e = lane; e < E; e += 64) {
    float l = load_logit(a.logits, a.logits_f32, t * E + e);
    if (!(l > -__builtin_inff())) l = -__builtin_inff();
    l = l > kFltMax ? kFltMax : l;
    key[e] = (double)l;
    mx = mx > (double)l ? mx : (double)l;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double o = __shfl_xor(mx, d, 64);
    mx = mx > o ? mx : o;
  }
  double z = 1.0;
  if (a.score == 0) {
    z = 0.0;
    for (int e = lane; e < E; e += 64)
      if (key[e] > none) z += exp(key[e] - mx);
    z = wave_add(z);
  }
  // a score from its logit (0 for a masked expert)
  auto score = [&](double l) -> double {
    if (!(l > none)) return 0.0;
    return a.score == 0 ? exp(l - mx) / z : 1.0 / (1.0 + exp(-l));
  };
  unsigned long long keep = ~0ull;
  if (a.bias)
    for (int e = lane; e < E; e += 64) {
      float b = a.bias[e];
      if (!(b > -__builtin_inff())) b = -__builtin_inff();
      b = b > kFltMax ? kFltMax : b;
      key[e] = key[e] > none ? score(key[e]) + (double)b : none;
    }
  __builtin_amdgcn_wave_barrier();
  __threadfence_block();
  if (a.groups > 1) {
    const int per = E / a.groups;
    double g = none;
    if (lane < a.groups) {
      double k1 = none, k2 = none;
      for (int i = 0; i < per; ++i) {
        const double k = key[lane * per + i];
        if (k > k1) {
          k2 = k1;
          k1 = k;
        } else if (k > k2) {
          k2 = k;
        }
      }
      g = k1;
      if (a.group_score == 1) {
        if (!a.bias) {
          k1 = k1 > none ? score(k1) : none;
          k2 = k2 > none ? score(k2) : none;
        }
        g = k2 > none ? k1 + k2 : k1;
      }
    }
    keep = 0ull;
    int gi = lane < a.groups ? lane : 64 + lane;
    for (int r = 0; r < a.topk_groups; ++r) {
      double bk = gi < 64 ? g : none;
      int bi = gi;
      wave_best(bk, bi);
      if (bi < 64) keep |= 1ull << bi;
      if (bi == gi) gi = 64 + lane;
    }
  }
  // top_k rounds of the wave's best remaining key
  const int per = E / a.groups;
  int chosen = -1;
  double cl = none;
  for (int r = 0; r < a.top_k; ++r) {
    double bk = none;
    int bi = 1 << 20;
    for (int e = lane; e < E; e += 64) {
      if (a.groups > 1 && !((keep >> (e / per)) & 1)) continue;
      if (key[e] > bk) {
        bk = key[e];
        bi = e;
      }
    }
    wave_best(bk, bi);
    if (!(bk > none)) break;
    if (lane == r) chosen = bi;
    if ((bi & 63) == lane) key[bi] = none;
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
  }
  float s = 0.f;
  if (chosen >= 0) {
    float l = load_logit(a.logits, a.logits_f32, t * E + chosen);
    cl = (double)(l > kFltMax ? kFltMax : l);
  }
  double w = chosen >= 0 ? score(cl) : 0.0;
  if (a.renorm) {
    // the ratio of scores, from logits so far below zero (or below the
    // token's best) that the scores themselves would vanish too
    double top = cl;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double o = __shfl_xor(top, d, 64);
      top = top > o ? top : o;
    }
    if (chosen >= 0) {
      const double base = a.score == 0 ? top : (top < 0.0 ? top : 0.0);
      w = a.score == 0 ? exp(cl - base) : (cl >= 0.0 ? 1.0 / (1.0 + exp(-cl)) : exp(cl - base) / (1.0 + exp(cl)));
    }
    const double sum = wave_add(w);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  s = (float)(w * (double)a.scale);
  if (lane < a.top_k) {
    a.ids[t * a.top_k + lane] = chosen;
    a.weights[t * a.top_k + lane] = chosen >= 0 ? s : 0.f;
  }
  }
}

// One wave per token.  With v_j = scale * dw_j over the valid choices:
//   sigmoid: dl = (v_j - [renorm] <v, s> / S) / [renorm] S * s (1 - s)
//   softmax: dl = s (ds - <ds, s>), ds as above; with renorm <ds, s> = 0
//            and the weights are a softmax over the choices alone
__global__ __launch_bounds__(256) void route_bwd_kernel(RouteBwdArgs a) {
  extern __shared__ float smemf[];
  const int lane = (int)(threadIdx.x & 63), wave = (int)(threadIdx.x >> 6);
  const int E = a.experts;
  float* acc = smemf + (size_t)wave * E;
  const float none = -__builtin_inff();
  for (int64_t t = (int64_t)blockIdx.x * kTokensPerWg + wave; t < a.tokens; t += (int64_t)gridDim.x * kTokensPerWg) {
  float mx = none;
  auto logit = [&](int e) -> float {
    float l = load_logit(a.logits, a.logits_f32, t * E + e);
    if (!(l > none)) l = none;
    return l > kFltMax ? kFltMax : l;
  };
  for (int e = lane; e < E; e += 64) {
    acc[e] = 0.f;
    const float l = logit(e);
    mx = mx > l ? mx : l;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) mx = __builtin_fmaxf(mx, __shfl_xor(mx, d, 64));
  int id = -1;
  float v = 0.f, cl = none;
  if (lane < a.top_k) {
    id = a.ids[t * a.top_k + lane];
    if (id < 0 || id >= E) id = -1;
    if (id >= 0) {
      cl = logit(id);
      if (!(cl > none)) id = -1;
    }
    if (id >= 0) v = a.scale * a.dweights[t * a.top_k + lane];
  }
  float top = cl;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, d, 64));
  float z = 1.f;
  if (a.score == 0 && !a.renorm) {
    z = 0.f;
    for (int e = lane; e < E; e += 64) {
      const float l = logit(e);
      if (l > none) z += expf(l - mx);
    }
    z = wave_add(z);
  }
  float dl = 0.f, back = 0.f;
  if (a.renorm) {
    float s = 0.f;
    const float base = a.score == 0 ? top : (top < 0.f ? top : 0.f);
    if (id >= 0)
      s = a.score == 0 ? expf(cl - base) : (cl >= 0.f ? 1.f / (1.f + expf(-cl)) : expf(cl - base) / (1.f + expf(cl)));
    const float sum = wave_add(s);
    const float p = id >= 0 ? s / sum : 0.f;       // the weight before scale
    const float mean = wave_add(v * p);
    dl = p * (v - mean);
    if (a.score == 1 && id >= 0) dl *= 1.f / (1.f + expf(cl));
  } else if (id >= 0) {
    const float s = a.score == 0 ? expf(cl - mx) / z : 1.f / (1.f + expf(-cl));
    dl = v * s;
    if (a.score == 1) dl *= 1.f / (1.f + expf(cl));
  }
  if (a.score == 0 && !a.renorm) back = wave_add(dl);
  // choices in order, so that an expert listed twice adds up the same way
  // every time
  for (int j = 0; j < a.top_k; ++j) {
    if (lane == j && id >= 0) acc[id] += dl;
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
  }
  for (int e = lane; e < E; e += 64) {
    float d = acc[e];
    if (a.score == 0 && !a.renorm) {
      const float l = logit(e);
      if (l > none) d -= back * (expf(l - mx) / z);
    }
    if (a.logits_f32)
      reinterpret_cast<float*>(a.dlogits)[t * E + e] = d;
    else
      reinterpret_cast<uint16_t*>(a.dlogits)[t * E + e] = (uint16_t)pack_bf16x2(d, 0.f);
  }
  }
}

// ---------------------------------------------------------------------- plan

// A stable counting sort of the pairs by expert: workgroup b counts its run
// of pairs per expert (plan_count_kernel), then every workgroup adds up the
// counts of the runs before its own and places its pairs in order
// (plan_place_kernel).  One workgroup counts and places in one launch.
constexpr int kPlanThreads = 256;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPlanRun = 2048;       // pairs per workgroup, at least
constexpr int kPlanMaxRuns = 256;    // longer runs beyond: every workgroup reads all runs' counts

__global__ __launch_bounds__(kPlanThreads) void plan_count_kernel(const int32_t* __restrict__ ids, int pairs, int run_len,
                                                                  int E, int32_t* __restrict__ counts) {
  __shared__ int hist[1024];
  for (int e = (int)threadIdx.x; e < E; e += kPlanThreads) hist[e] = 0;
  __syncthreads();
  const int lo = (int)blockIdx.x * run_len, hi = pairs - lo < run_len ? pairs : lo + run_len;
  for (int i = lo + (int)threadIdx.x; i < hi; i += kPlanThreads) {
    const int id = ids[i];
    if (id >= 0 && id < E) atomicAdd(&hist[id], 1);
  }
  __syncthreads();
  for (int e = (int)threadIdx.x; e < E; e += kPlanThreads) counts[(int64_t)blockIdx.x * E + e] = hist[e];
}

__global__ __launch_bounds__(kPlanThreads) void plan_place_kernel(const int32_t* __restrict__ ids, int pairs,
                                                                  int run_len, int top_k, int E, int bits,
                                                                  const int32_t* __restrict__ counts,
                                                                  int32_t* __restrict__ offsets,
                                                                  int32_t* __restrict__ row_index,
                                                                  int32_t* __restrict__ slot) {
  __shared__ int ctr[kPlanWaves][1024];   // next row of each expert, per wave of this run
  __shared__ int total[1024];             // rows of each expert, then their running sums
  __shared__ int before[1024];            // rows of each expert in the runs before this one
  const int t = (int)threadIdx.x, lane = t & 63, wave = t >> 6;
  const int runs = (int)gridDim.x, run = (int)blockIdx.x;
  const int lo = run * run_len, hi = pairs - lo < run_len ? pairs : lo + run_len;
  for (int e = t; e < E; e += kPlanThreads) {
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) ctr[w][e] = 0;
    int tot = 0, bef = 0;
    if (runs > 1)
      for (int r = 0; r < runs; ++r) {
        const int c = counts[(int64_t)r * E + e];
        bef += r < run ? c : 0;
        tot += c;
      }
    total[e] = tot;
    before[e] = bef;
  }
  __syncthreads();
  // wave w takes the w-th quarter of the run, so earlier waves hold earlier pairs
  const int quarter = run_len / kPlanWaves;
  const int wlo = lo + wave * quarter;
  const int whi = wlo + quarter < hi ? wlo + quarter : hi;
  for (int i = wlo + lane; i < whi; i += 64) {
    const int id = ids[i];
    if (id >= 0 && id < E) atomicAdd(&ctr[wave][id], 1);
  }
  __syncthreads();
  if (runs == 1) {
    for (int e = t; e < E; e += kPlanThreads) {
      int c = 0;
#pragma unroll
      for (int w = 0; w < kPlanWaves; ++w) c += ctr[w][e];
      total[e] = c;
    }
    __syncthreads();
  }
  // inclusive running sums of the totals
  for (int d = 1; d < E; d <<= 1) {
    int v[1024 / kPlanThreads];
    int n = 0;
    for (int e = t; e < E; e += kPlanThreads) v[n++] = e >= d ? total[e - d] : 0;
    __syncthreads();
    n = 0;
    for (int e = t; e < E; e += kPlanThreads) total[e] += v[n++];
    __syncthreads();
  }
  for (int e = t; e < E; e += kPlanThreads) {
    int at = (e > 0 ? total[e - 1] : 0) + before[e];
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      const int c = ctr[w][e];
      ctr[w][e] = at;
      at += c;
    }
  }
  if (run == 0) {
    if (t == 0) offsets[0] = 0;
    for (int e = t; e < E; e += kPlanThreads) offsets[e + 1] = total[e];
  }
  __syncthreads();
  for (int i0 = wlo; i0 < whi; i0 += 64) {
    const int i = i0 + lane;
    int id = i < whi ? ids[i] : -1;
    const bool ok = id >= 0 && id < E;
    // lanes of the wave with the same expert
    unsigned long long same = __builtin_amdgcn_ballot_w64(ok);
    for (int b = 0; b < bits; ++b) {
      const unsigned long long set = __builtin_amdgcn_ballot_w64((id >> b) & 1);
      same &= ((id >> b) & 1) ? set : ~set;
    }
    if (ok) {
      const unsigned long long below = same & ((1ull << lane) - 1);
      const int at = ctr[wave][id] + __builtin_popcountll(below);
      __builtin_amdgcn_wave_barrier();
      // the last of them moves the counter on (after every lane has read it)
      if ((same >> lane) == 1ull) ctr[wave][id] = at + 1;
      slot[i] = at;
      row_index[at] = i / top_k;
    } else if (i < whi) {
      slot[i] = -1;
    }
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
  }
  for (int i = total[E - 1] + run * kPlanThreads + t; i < pairs; i += runs * kPlanThreads) row_index[i] = 0;
}

// Pairs per run (a multiple of the workgroup) and runs.
int plan_run_len(int64_t pairs) {
  const int64_t len = ((pairs + kPlanMaxRuns - 1) / kPlanMaxRuns + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
  return (int)(len < kPlanRun ? kPlanRun : len);
}
int plan_runs(int64_t pairs) {
  const int len = plan_run_len(pairs);
  return pairs <= len ? 1 : (int)((pairs + len - 1) / len);
}

}  // namespace

int64_t plan_workspace_bytes(int64_t pairs, int experts) {
  const int runs = plan_runs(pairs);
  return runs == 1 ? 0 : (int64_t)runs * experts * 4;
}

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
  const int64_t wgs = (a.tokens + kTokensPerWg - 1) / kTokensPerWg;
  const dim3 grid((unsigned)(wgs < kMaxGrid ? wgs : kMaxGrid));
  hipLaunchKernelGGL(route_kernel, grid, dim3(64 * kTokensPerWg), (size_t)kTokensPerWg * a.experts * sizeof(double),
                     stream, a);
  return hipGetLastError();
}

hipError_t launch_route_bwd(const RouteBwdArgs& a, hipStream_t stream) {
  const int64_t wgs = (a.tokens + kTokensPerWg - 1) / kTokensPerWg;
  const dim3 grid((unsigned)(wgs < kMaxGrid ? wgs : kMaxGrid));
  hipLaunchKernelGGL(route_bwd_kernel, grid, dim3(64 * kTokensPerWg), (size_t)kTokensPerWg * a.experts * sizeof(float),
                     stream, a);
  return hipGetLastError();
}

hipError_t launch_plan(const int32_t* ids, int64_t tokens, int top_k, int experts, void* workspace, int32_t* offsets,
                       int32_t* row_index, int32_t* slot, hipStream_t stream) {
  const int64_t pairs = tokens * top_k;
  const int runs = plan_runs(pairs);
  int bits = 0;
  while ((1 << bits) < experts) ++bits;
  int32_t* counts = reinterpret_cast<int32_t*>(workspace);
  if (runs > 1)
    hipLaunchKernelGGL(plan_count_kernel, dim3((unsigned)runs), dim3(kPlanThreads), 0, stream, ids, (int)pairs,
                       plan_run_len(pairs), experts, counts);
  hipLaunchKernelGGL(plan_place_kernel, dim3((unsigned)runs), dim3(kPlanThreads), 0, stream, ids, (int)pairs,
                     plan_run_len(pairs), top_k, experts, bits, counts, offsets, row_index, slot);
  return hipGetLastError();
}

}  // namespace fp8blk
