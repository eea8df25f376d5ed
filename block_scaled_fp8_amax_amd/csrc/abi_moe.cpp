// C-ABI entry points of the mixture-of-experts operators: argument
// validation and kernel dispatch.  The declarations and their contracts are
// in include/fp8blk_moe.h.
#include "fp8blk_moe.h"

#include <hip/hip_runtime.h>

#include <math.h>

#include "host.h"
#include "launch.h"

namespace {

using namespace fp8blk;

bool valid_type(int t) { return t == FP8_OUT_BF16 || t == FP8_OUT_F32; }
uintptr_t type_bytes(int t) { return t == FP8_OUT_F32 ? 4 : 2; }
hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

constexpr int64_t kMaxRows = 0x7FFFFFFFll;
constexpr int64_t kMaxNormCols = 32768;
constexpr int64_t kMaxPairs = int64_t(1) << 30;
constexpr int64_t kMaxWidth = int64_t(1) << 24;

int norm_shape(int64_t rows, int64_t cols, int64_t multiple) {
  if (rows < 0 || rows > kMaxRows || cols < 0 || cols > kMaxNormCols || cols % multiple) return FP8_ERR_SHAPE;
  return FP8_OK;
}

// tokens, top_k and experts of the routing calls.
int pair_shape(int64_t tokens, int top_k, int experts) {
  if (experts < 1 || experts > 1024 || top_k < 1 || top_k > 64) return FP8_ERR_INVALID_ARG;
  if (tokens < 0 || !product_at_most(tokens, top_k, kMaxPairs)) return FP8_ERR_SHAPE;
  return FP8_OK;
}

int combine_args(int row_type, int other_type, int64_t total_m, int64_t tokens, int top_k, int64_t n) {
  if (!valid_type(row_type) || !valid_type(other_type)) return FP8_ERR_INVALID_ARG;
  if (top_k < 1 || top_k > 64) return FP8_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > kMaxRows || total_m < 0 || total_m > kMaxRows) return FP8_ERR_SHAPE;
  if (n < 0 || n > kMaxWidth || n % 8) return FP8_ERR_SHAPE;
  return FP8_OK;
}

// x is read with 32-bit byte offsets.
constexpr int64_t kMaxMatvecX = (int64_t(1) << 30) - 1;

int matvec_shape(int64_t x_rows, int64_t rows_per_tensor, int64_t m, int64_t n, int64_t k, int y_type) {
  if (!valid_type(y_type)) return FP8_ERR_INVALID_ARG;
  if (m < 0 || m > kMaxRows || n < 0 || n > kMaxWidth || k <= 0 || k > kMaxWidth || k % 16) return FP8_ERR_SHAPE;
  if (rows_per_tensor < 1 || n % rows_per_tensor) return FP8_ERR_SHAPE;
  if (x_rows < 0 || !product_at_most(x_rows, k, kMaxMatvecX)) return FP8_ERR_SHAPE;
  return FP8_OK;
}

}  // namespace

extern "C" {

int fp8_moe_abi_version(void) { return FP8BLK_MOE_ABI_VERSION; }

int fp8_rmsnorm_quantize(const uint16_t* x, const uint16_t* residual, const void* weight, int weight_type,
                         int64_t rows, int64_t cols, float eps, int kind, int rule, uint8_t* q, void* scale,
                         uint16_t* h, uint16_t* y, uint16_t* ydq, float* rstd, void* stream) {
  if (kind != FP8_BLOCK_1x32_E8M0 && kind != FP8_BLOCK_1x128_F32)
    return kind == FP8_BLOCK_128x128_F32 ? FP8_ERR_UNSUPPORTED : FP8_ERR_INVALID_ARG;
  const bool mx = kind == FP8_BLOCK_1x32_E8M0;
  if (mx && rule != FP8_E8M0_CEIL && rule != FP8_E8M0_FLOOR) return FP8_ERR_INVALID_ARG;
  if (!valid_type(weight_type) || !(eps >= 1e-20f) || !(eps < INFINITY)) return FP8_ERR_INVALID_ARG;
  if ((residual != nullptr) != (h != nullptr)) return FP8_ERR_INVALID_ARG;
  if (int s = norm_shape(rows, cols, mx ? 32 : 128)) return s;
  if (rows == 0 || cols == 0) return FP8_OK;
  if (!x || !weight || !q || !scale) return FP8_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(q, 16) || !aligned(h, 16) ||
      !aligned(y, 16) || !aligned(ydq, 16) || !aligned(rstd, 4) || !aligned(scale, mx ? 1 : 4))
    return FP8_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if (int s = current_device(&dev)) return s;
  RmsNorm a{x, residual, weight, weight_type == FP8_OUT_F32, rows, cols, eps, mx ? 32 : 128,
            mx && rule == FP8_E8M0_FLOOR, q, scale, h, y, ydq, rstd};
  return hip_status(launch_rmsnorm_quant(a, as_stream(stream)));
}

int fp8_rmsnorm_backward_workspace(int64_t rows, int64_t cols, size_t* bytes) {
  if (!bytes) return FP8_ERR_INVALID_ARG;
  if (int s = norm_shape(rows, cols, 8)) return s;
  *bytes = (size_t)(rmsnorm_bwd_parts(rows, cols) * cols * 4);
  return FP8_OK;
}

int fp8_rmsnorm_backward(const uint16_t* dy, const uint16_t* h, const void* weight, int weight_type,
                         const float* rstd, const uint16_t* dres, int64_t rows, int64_t cols, void* workspace,
                         size_t workspace_bytes, uint16_t* dx, void* dweight, void* stream) {
  if (!valid_type(weight_type)) return FP8_ERR_INVALID_ARG;
  if (int s = norm_shape(rows, cols, 8)) return s;
  if (cols == 0) return FP8_OK;
  if (!weight || !dweight) return FP8_ERR_INVALID_ARG;
  if (rows > 0 && (!dy || !h || !rstd || !dx || !workspace)) return FP8_ERR_INVALID_ARG;
  if (workspace_bytes < (size_t)(rmsnorm_bwd_parts(rows, cols) * cols * 4)) return FP8_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(h, 16) || !aligned(weight, 16) || !aligned(rstd, 4) || !aligned(dres, 16) ||
      !aligned(workspace, 256) || !aligned(dx, 16) || !aligned(dweight, type_bytes(weight_type)))
    return FP8_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if (int s = current_device(&dev)) return s;
  return hip_status(launch_rmsnorm_bwd(dy, h, weight, weight_type == FP8_OUT_F32, rstd, dres, rows, cols, workspace,
                                       dx, dweight, as_stream(stream)));
}

int fp8_moe_route(const void* logits, int logits_type, const float* bias, int64_t tokens, int experts, int top_k,
                  int score, int groups, int topk_groups, int group_score, int renorm, float scale, int32_t* ids,
                  float* weights, void* stream) {
  if (!valid_type(logits_type)) return FP8_ERR_INVALID_ARG;
  if (score != FP8_SCORE_SOFTMAX && score != FP8_SCORE_SIGMOID) return FP8_ERR_INVALID_ARG;
  if (group_score != FP8_GROUP_MAX && group_score != FP8_GROUP_TOP2) return FP8_ERR_INVALID_ARG;
  if ((renorm != 0 && renorm != 1) || !isfinite(scale)) return FP8_ERR_INVALID_ARG;
  if (int s = pair_shape(tokens, top_k, experts)) return s;
  if (groups < 1 || groups > 64 || experts % groups || topk_groups < 1 || topk_groups > groups)
    return FP8_ERR_INVALID_ARG;
  if (top_k > topk_groups * (experts / groups)) return FP8_ERR_INVALID_ARG;
  if (tokens == 0) return FP8_OK;
  if (!logits || !ids || !weights) return FP8_ERR_INVALID_ARG;
  if (!aligned(logits, type_bytes(logits_type)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
    return FP8_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if (int s = current_device(&dev)) return s;
  RouteArgs a{logits, bias, tokens, experts, top_k, groups, topk_groups, score, group_score, renorm,
              logits_type == FP8_OUT_F32 ? 1 : 0, scale, ids, weights};
  return hip_status(launch_route(a, as_stream(stream)));
}

int fp8_moe_route_backward(const void* logits, int logits_type, const int32_t* ids, const float* dweights,
                           int64_t tokens, int experts, int top_k, int score, int renorm, float scale, void* dlogits,
                           void* stream) {
  if (!valid_type(logits_type)) return FP8_ERR_INVALID_ARG;
  if (score != FP8_SCORE_SOFTMAX && score != FP8_SCORE_SIGMOID) return FP8_ERR_INVALID_ARG;
  if ((renorm != 0 && renorm != 1) || !isfinite(scale)) return FP8_ERR_INVALID_ARG;
  if (int s = pair_shape(tokens, top_k, experts)) return s;
  if (tokens == 0) return FP8_OK;
  if (!logits || !ids || !dweights || !dlogits) return FP8_ERR_INVALID_ARG;
  if (!aligned(logits, type_bytes(logits_type)) || !aligned(dlogits, type_bytes(logits_type)) || !aligned(ids, 4) ||
      !aligned(dweights, 4))
    return FP8_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if (int s = current_device(&dev)) return s;
  RouteBwdArgs a{logits, ids, dweights, tokens, experts, top_k, score, renorm, logits_type == FP8_OUT_F32 ? 1 : 0,
                 scale, dlogits};
  return hip_status(launch_route_bwd(a, as_stream(stream)));
}

int fp8_moe_plan_workspace(int64_t tokens, int top_k, int experts, size_t* bytes) {
  if (!bytes) return FP8_ERR_INVALID_ARG;
  if (int s = pair_shape(tokens, top_k, experts)) return s;
  *bytes = (size_t)plan_workspace_bytes(tokens * top_k, experts);
  return FP8_OK;
}

int fp8_moe_plan(const int32_t* ids, int64_t tokens, int top_k, int experts, void* workspace, size_t workspace_bytes,
                 int32_t* offsets, int32_t* row_index, int32_t* slot, void* stream) {
  if (int s = pair_shape(tokens, top_k, experts)) return s;
  if (!offsets || (tokens > 0 && (!ids || !row_index || !slot))) return FP8_ERR_INVALID_ARG;
  const size_t need = (size_t)plan_workspace_bytes(tokens * top_k, experts);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FP8_ERR_INVALID_ARG;
  if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(row_index, 4) || !aligned(slot, 4) ||
      (need > 0 && !aligned(workspace, 16)))
    return FP8_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if (int s = current_device(&dev)) return s;
  return hip_status(launch_plan(ids, tokens, top_k, experts, workspace, offsets, row_index, slot, as_stream(stream)));
}

int fp8_nvfp4_matvec(const uint16_t* x, const uint8_t* q, const uint8_t* block_scale, const float* global_scale,
                     int64_t rows_per_tensor, int64_t m, int64_t n, int64_t k, void* y, int y_type, void* stream) {
  if (int s = matvec_shape(m, rows_per_tensor, m, n, k, y_type)) return s;
  if (m == 0 || n == 0) return FP8_OK;
  if (!x || !q || !block_scale || !global_scale || !y) return FP8_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 8) || !aligned(global_scale, 4) || !aligned(y, type_bytes(y_type)))
    return FP8_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if (int s = current_device(&dev)) return s;
  MatvecArgs a{x, m, nullptr, q, block_scale, global_scale, rows_per_tensor, nullptr, 1, m, n, k, y,
               y_type == FP8_OUT_F32};
  return hip_status(launch_matvec(a, as_stream(stream)));
}

int fp8_nvfp4_grouped_matvec(const uint16_t* x, int64_t x_rows, const int32_t* row_index, const uint8_t* q,
                             const uint8_t* block_scale, const float* global_scale, int64_t rows_per_tensor,
                             const int32_t* group_offsets, int64_t groups, int64_t total_m, int64_t n, int64_t k,
                             void* y, int y_type, void* stream) {
  if (int s = matvec_shape(x_rows, rows_per_tensor, total_m, n, k, y_type)) return s;
  if (groups < 1 || groups > 1024) return FP8_ERR_INVALID_ARG;
  if (total_m == 0 || n == 0) return FP8_OK;
  if (x_rows == 0 || (!row_index && x_rows != total_m)) return FP8_ERR_SHAPE;
  if (!x || !q || !block_scale || !global_scale || !group_offsets || !y) return FP8_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 8) || !aligned(global_scale, 4) || !aligned(group_offsets, 4) ||
      !aligned(row_index, 4) || !aligned(y, type_bytes(y_type)))
    return FP8_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if (int s = current_device(&dev)) return s;
  MatvecArgs a{x, x_rows, row_index, q, block_scale, global_scale, rows_per_tensor, group_offsets, groups, total_m,
               n, k, y, y_type == FP8_OUT_F32};
  return hip_status(launch_matvec(a, as_stream(stream)));
}

int fp8_moe_combine(const void* rows, int row_type, int64_t total_m, const int32_t* slot, const float* weights,
                    const uint16_t* residual, int64_t tokens, int top_k, int64_t n, void* y, int y_type,
                    void* stream) {
  if (int s = combine_args(row_type, y_type, total_m, tokens, top_k, n)) return s;
  if (tokens == 0 || n == 0) return FP8_OK;
  if ((!rows && total_m > 0) || !slot || !weights || !y) return FP8_ERR_INVALID_ARG;
  if (!aligned(rows, 16) || !aligned(slot, 4) || !aligned(weights, 4) || !aligned(residual, 16) || !aligned(y, 16))
    return FP8_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if (int s = current_device(&dev)) return s;
  CombineArgs a{rows, total_m, slot, weights, residual, tokens, top_k, n, y, row_type == FP8_OUT_F32,
                y_type == FP8_OUT_F32};
  return hip_status(launch_combine(a, as_stream(stream)));
}

int fp8_moe_combine_backward(const void* dy, int dy_type, const void* rows, int row_type, int64_t total_m,
                             const int32_t* slot, const float* weights, int64_t tokens, int top_k, int64_t n,
                             void* drows, float* dweights, void* stream) {
  if (int s = combine_args(row_type, dy_type, total_m, tokens, top_k, n)) return s;
  if (tokens == 0) return FP8_OK;
  if ((n > 0 && (!dy || (total_m > 0 && (!rows || !drows)))) || !slot || !weights || !dweights)
    return FP8_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(rows, 16) || !aligned(slot, 4) || !aligned(weights, 4) || !aligned(drows, 16) ||
      !aligned(dweights, 4))
    return FP8_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if (int s = current_device(&dev)) return s;
  CombineBwdArgs a{dy, rows, total_m, slot, weights, tokens, top_k, n, drows, dweights, dy_type == FP8_OUT_F32,
                   row_type == FP8_OUT_F32};
  return hip_status(launch_combine_bwd(a, as_stream(stream)));
}

}  // extern "C"
