// Kernel launchers of the fp8blk library (internal; arguments are already
// validated by abi.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8blk {

hipError_t launch_quant_rows(const uint16_t* x, int64_t rows, int64_t cols, int blk, bool floor_rule, uint8_t* q,
                             void* scale, uint16_t* xdq, int num_cu, hipStream_t stream);
hipError_t launch_quant_128(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* q, float* scale, uint16_t* xdq,
                            hipStream_t stream);
// Batched quantize: jobs already validated (at most kMaxQuantJobs).
constexpr int kMaxQuantJobs = 16;
// 8-chunk groups a rows-kind (1x32, 1x128) batch workgroup covers in its one
// pass: 8 waves x 64 lanes x 2 chunks.
constexpr int64_t kQuantBatchRowsChunks = 1024;
struct QuantJobIn {
  const uint16_t* x;
  int64_t rows, cols;
  int kind;           // 0 = 1x32 E8M0, 1 = 1x128 fp32, 2 = 128x128 fp32
  bool floor_rule;
  uint8_t* q;
  void* scale;
  uint16_t* xdq;
};
struct QuantJob {
  const uint16_t* x;
  int64_t rows, cols;
  uint8_t* q;
  void* scale;
  uint16_t* xdq;
  int kind, floor_rule, cached, blocks_x, wg0, wgs;
};
struct QuantBatch {
  QuantJob job[kMaxQuantJobs];
  int count;
};
hipError_t launch_quant_batch(const QuantJobIn* jobs, int count, hipStream_t stream);
hipError_t launch_dequant(const uint8_t* q, const void* scale, int64_t rows, int64_t cols, int kind, uint16_t* x,
                          hipStream_t stream);
hipError_t launch_merge(const uint16_t* w, const uint16_t* lb, const uint16_t* la, int64_t n, int64_t k, int64_t r,
                        uint8_t* q, float* scale, uint16_t* wdq, hipStream_t stream);
hipError_t launch_gemm(const uint8_t* a, const void* sa, int a_kind, const uint8_t* b, const void* sb, int b_kind,
                       int64_t m, int64_t n, int64_t k, void* y, bool out_f32, int num_cu, hipStream_t stream);
hipError_t launch_grouped_gemm(const uint8_t* a, const void* sa, int a_kind, const int32_t* row_index,
                               int64_t a_rows, const uint8_t* b, const void* sb, int b_kind, const int32_t* offsets, int64_t groups,
                               int64_t total_m, int64_t n, int64_t k, void* y, bool out_f32, int num_cu,
                               hipStream_t stream);

int64_t lora_bwd_workspace_bytes(int64_t m, int64_t n, int64_t k, int64_t r);
// Fixed scratch of the no-allocation LoRA backward (one array per device):
// 40 MiB holds the workspace of 8192 tokens at hidden sizes 7168 and rank
// 64 (36.4 MiB).
constexpr int64_t kLoraScratchBytes = int64_t(40) << 20;
constexpr int kMaxScratchDevices = 64;
// The device address of `dev`'s scratch array (looked up once per device,
// with `dev` current).
hipError_t lora_bwd_scratch(int dev, void** ptr);
hipError_t launch_lora_bwd(const uint16_t* dy, const uint16_t* x, const uint16_t* lb, const uint16_t* la, int64_t m,
                           int64_t n, int64_t k, int64_t r, void* workspace, void* d_b, void* d_a, bool out_f32,
                           int num_cu, hipStream_t stream);

hipError_t launch_nvfp4_quant(const uint16_t* x, int64_t rows, int64_t cols, int64_t rpt, float* amax,
                              bool amax_given, uint8_t* q, uint8_t* bs, float* gs, uint16_t* xdq,
                              hipStream_t stream);
hipError_t launch_nvfp4_dequant(const uint8_t* q, const uint8_t* bs, const float* gs, int64_t rows, int64_t cols,
                                int64_t rpt, uint16_t* x, hipStream_t stream);

// ------------------------------------------------ mixture-of-experts operators

// Workgroups of a launch at most (a launch's threads have to stay below
// 2^32); kernels that take one row or token per workgroup walk on from there.
constexpr int64_t kMaxGrid = int64_t(1) << 20;

// Bytes of a call past which its accesses are nontemporal: what it reads and
// writes does not stay in the 256 MB of the Infinity Cache anyway, and that
// way its stores and loads disturb each other less.  16384 x 8 rows of 7168
// combined: 416 us, 460 with the cache's own policy; norm of 16384 x 7168: 180
// and 188, its gradient for 8192 x 7168: 90 and 96; NVFP4 weights of 52 experts
// of 4096 x 7168: 149 and 164.  Smaller calls find their inputs in the cache
// and leave their outputs there (2048 x 7168 normed, 132 MB: 23.0 us,
// nontemporal 27.9; weights of 8 such experts, two sets in turn: 25.8 and
// 27.4).
constexpr int64_t kCached = int64_t(256) << 20;

struct RmsNorm {
  const uint16_t* x;
  const uint16_t* residual;
  const void* weight;
  bool weight_f32;
  int64_t rows, cols;
  float eps;
  int blk;            // 32 or 128
  bool floor_rule;
  uint8_t* q;
  void* scale;
  uint16_t *h, *y, *ydq;
  float* rstd;
};
hipError_t launch_rmsnorm_quant(const RmsNorm& a, hipStream_t stream);
// Partial weight gradients the backward pass keeps: [parts][cols] floats.
int64_t rmsnorm_bwd_parts(int64_t rows, int64_t cols);
hipError_t launch_rmsnorm_bwd(const uint16_t* dy, const uint16_t* h, const void* w, bool w_f32, const float* rstd,
                              const uint16_t* dres, int64_t rows, int64_t cols, void* workspace, uint16_t* dx,
                              void* dw, hipStream_t stream);

struct RouteArgs {
  const void* logits;
  const float* bias;
  int64_t tokens;
  int experts, top_k, groups, topk_groups;
  int score, group_score, renorm, logits_f32;
  float scale;
  int32_t* ids;
  float* weights;
  // set by the launcher: experts per group, log2 of the lanes that rank a group through LDS, and of those whose
  // experts make up a group (-1 where lanes span groups)
  int per = 0, log_width = 0, log_heads = -1;
  float inv_per = 0.f;
};
hipError_t launch_route(const RouteArgs& a, hipStream_t stream);
struct RouteBwdArgs {
  const void* logits;
  const int32_t* ids;
  const float* dweights;
  int64_t tokens;
  int experts, top_k, score, renorm, logits_f32;
  float scale;
  void* dlogits;
};
hipError_t launch_route_bwd(const RouteBwdArgs& a, hipStream_t stream);
int64_t plan_workspace_bytes(int64_t pairs, int experts);
hipError_t launch_plan(const int32_t* ids, int64_t tokens, int top_k, int experts, void* workspace, int32_t* offsets,
                       int32_t* row_index, int32_t* slot, hipStream_t stream);

struct MatvecArgs {
  const uint16_t* x;
  int64_t x_rows;
  const int32_t* row_index;   // null = the row itself
  const uint8_t* q;
  const uint8_t* block_scale;
  const float* global_scale;
  int64_t rows_per_tensor;
  const int32_t* offsets;     // null = one group of all rows
  int64_t groups, total_m, n, k;
  void* y;
  bool out_f32;
  int64_t slice = 0;          // rows of x per workgroup without offsets (set by the launcher)
};
hipError_t launch_matvec(const MatvecArgs& a, hipStream_t stream);

struct CombineArgs {
  const void* rows;
  int64_t total_m;
  const int32_t* slot;
  const float* weights;
  const uint16_t* residual;
  int64_t tokens;
  int top_k;
  int64_t n;
  void* y;
  bool row_f32, out_f32;
};
hipError_t launch_combine(const CombineArgs& a, hipStream_t stream);
struct CombineBwdArgs {
  const void* dy;
  const void* rows;
  int64_t total_m;
  const int32_t* slot;
  const float* weights;
  int64_t tokens;
  int top_k;
  int64_t n;
  void* drows;
  float* dweights;
  bool dy_f32, row_f32;
};
hipError_t launch_combine_bwd(const CombineBwdArgs& a, hipStream_t stream);

// ------------------------------------------------------------ MXFP4 experts

hipError_t launch_mxfp4_quant(const uint16_t* x, int64_t rows, int64_t cols, bool floor_rule, uint8_t* q,
                              uint8_t* scale, uint16_t* xdq, hipStream_t stream);
hipError_t launch_mxfp4_dequant(const uint8_t* q, const uint8_t* scale, int64_t rows, int64_t cols, uint16_t* x,
                                hipStream_t stream);

struct MxProduct {
  const uint8_t* a;
  const uint8_t* a_scale;
  bool a_fp4;
  int64_t a_rows;
  const int32_t* row_index;   // null = the row itself
  const uint8_t* b;
  const uint8_t* b_scale;
  const int32_t* offsets;     // null = one group of all rows
  int groups;
  int64_t m, n, k;
  void* y;
  bool out_f32;
};
hipError_t launch_mx_product(const MxProduct& p, int num_cu, hipStream_t stream);

struct MxRows {
  const uint16_t* x;
  int64_t x_rows;
  const int32_t* row_index;   // null = the row itself
  const uint8_t* q;
  const uint8_t* scale;
  const int32_t* offsets;     // null = one group of all rows
  int64_t groups, total_m, n, k;
  void* y;
  bool out_f32;
};
hipError_t launch_mx_rows(const MxRows& a, hipStream_t stream);
// A product of few rows (of each group), for which launch_mx_product's tiles
// are too large.
hipError_t launch_mx_few(const MxProduct& p, hipStream_t stream);

struct GroupedGrad {
  const uint16_t* dy;
  const uint16_t* x;          // wgrad
  int64_t x_rows;
  const int32_t* row_index;   // wgrad; null = the row itself
  const uint16_t* w;          // dgrad
  const int32_t* offsets;
  int groups;
  int64_t total_m, n, k;
  void* out;
  bool out_f32;
};
hipError_t launch_grouped_dgrad(const GroupedGrad& a, int num_cu, hipStream_t stream);
hipError_t launch_grouped_wgrad(const GroupedGrad& a, int num_cu, hipStream_t stream);

}  // namespace fp8blk
