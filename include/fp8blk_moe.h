/*
 * fp8blk_moe -- the operators of a mixture-of-experts layer around the
 * block-scaled FP8 and NVFP4 products of fp8blk.h: residual addition and
 * root-mean-square norm with FP8 output, routing to experts, products with
 * NVFP4 weights, and the weighted combination of the experts' rows.  Same
 * library (libfp8blk.so), same device (gfx950).  C ABI.
 *
 * The conventions of fp8blk.h hold here too: device pointers to dense
 * row-major matrices, bf16 as uint16_t, caller-owned buffers and
 * workspaces, arguments checked on the host before anything is enqueued,
 * fp8_status results, no allocation, no synchronization, only kernels on
 * `stream` (so calls can be captured into a HIP graph), identical bytes for
 * identical inputs.  Element types of arguments that allow both are given
 * as fp8_out values (FP8_OUT_BF16, FP8_OUT_F32).  bf16 and float inputs are
 * finite unless a call says otherwise.  Buffers of one call do not overlap
 * unless the call says so.  Calls that share a workspace are ordered by the
 * caller (one stream, or events).
 *
 * A prompt passes an MoE layer as
 *   fp8_rmsnorm_quantize -> (router product) -> fp8_moe_route -> fp8_moe_plan
 *   -> fp8_grouped_gemm_gather(row_index, offsets) -> activation, quantize
 *   -> fp8_grouped_gemm -> fp8_moe_combine(slot, weights, residual)
 * and decoded tokens with NVFP4 experts take fp8_nvfp4_grouped_matvec in
 * place of the two grouped GEMMs.
 */
#ifndef FP8BLK_MOE_H
#define FP8BLK_MOE_H

#include "fp8blk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FP8BLK_MOE_ABI_VERSION 1

/* How a router turns logits into scores. */
typedef enum { FP8_SCORE_SOFTMAX = 0, FP8_SCORE_SIGMOID = 1 } fp8_score;

/* How a group of experts is ranked: by its best key, or by the sum of its
 * two best keys (its only key where it has one). */
typedef enum { FP8_GROUP_MAX = 0, FP8_GROUP_TOP2 = 1 } fp8_group_score;

/*
 * fp8_rmsnorm_quantize -- residual addition, root-mean-square norm and FP8
 * quantization of the normed rows, in one pass.
 *
 *   h    = RN_bf16(x + residual)            (h = x without a residual)
 *   rstd = 1 / sqrt(mean_j h[j]^2 + eps)    (fp32; rows whose squares leave
 *                                            the fp32 range are rescaled)
 *   y[j] = h[j] * rstd * weight[j]          (fp32, not rounded further)
 * and y is quantized per row in 1x128 tiles (scale = RN32(amax / 448),
 * code = e4m3(y / scale)) or 1x32 blocks (E8M0 exponent X by `rule`, code =
 * e4m3(y * 2^-X)) as fp8_block_quantize does, but from the fp32 y.  A tile
 * whose fp32 scale is 0 gets codes +-0.  Rows whose h or y leaves its range
 * (bf16, fp32) have no defined codes; a NaN in a row shows in its y and rstd,
 * not in its codes.
 *
 * x        [rows x cols] bf16 (16-byte aligned);
 * residual optional (NULL = none) [rows x cols] bf16 (16-byte aligned);
 * weight   [cols] bf16 or float per weight_type (16-byte aligned);
 * eps      finite, >= 1e-20;
 * kind     FP8_BLOCK_1x32_E8M0 or FP8_BLOCK_1x128_F32; rule as in
 *          fp8_block_quantize;
 * q        [rows x cols] codes out (16-byte aligned); scale as
 *          fp8_block_quantize writes it for `kind`;
 * h        [rows x cols] bf16 out, required with a residual (it may be x or
 *          residual itself) and NULL without one;
 * y        optional [rows x cols] bf16 out, RN_bf16(y) (for the router and
 *          other bf16 products);
 * ydq      optional [rows x cols] bf16 out, the fake-quant value
 *          RN_bf16(RN32(decode(q) * scale));
 * rstd     optional [rows] float out (fp8_rmsnorm_backward reads it).
 * Shape: 0 <= rows < 2^31, 0 <= cols <= 32768, cols % 32 == 0 (1x32) or
 *        cols % 128 == 0 (1x128).  rows == 0 or cols == 0 enqueues nothing.
 */
int fp8_rmsnorm_quantize(const uint16_t* x, const uint16_t* residual, const void* weight, int weight_type,
                         int64_t rows, int64_t cols, float eps, int kind, int rule, uint8_t* q, void* scale,
                         uint16_t* h, uint16_t* y, uint16_t* ydq, float* rstd, void* stream);

/*
 * fp8_rmsnorm_backward -- gradients of y = h * rstd * weight, straight
 * through the quantization.
 *
 *   xh = h * rstd,  c = mean_j(weight dy xh)
 *   dx = rstd * (weight dy - xh c) + dres   (the gradient of x and of the
 *                                            residual alike)
 *   dweight = sum over rows of dy xh
 * dres is the gradient that reaches h past the norm (the residual stream).
 * Sums are fp32: a row of which the |weight dy| or the |weight dy xh| add up
 * past that range has no defined dx, a column of which the |dy xh| do no
 * defined dweight.
 *
 * dy     [rows x cols] bf16 (16-byte aligned); h [rows x cols] bf16, the h
 *        of the forward call (x where it had no residual); weight as there;
 * rstd   [rows] float of the forward call (4-byte aligned);
 * dres   optional [rows x cols] bf16;
 * workspace: at least the bytes fp8_rmsnorm_backward_workspace reports,
 *        256-byte aligned, garbage before and after;
 * dx     [rows x cols] bf16 out (it may be dy or dres itself);
 * dweight [cols] out, bf16 or float per weight_type (rows == 0 writes zeros).
 * Shape: 0 <= rows < 2^31, 0 <= cols <= 32768, cols % 8 == 0.
 */
int fp8_rmsnorm_backward(const uint16_t* dy, const uint16_t* h, const void* weight, int weight_type,
                         const float* rstd, const uint16_t* dres, int64_t rows, int64_t cols, void* workspace,
                         size_t workspace_bytes, uint16_t* dx, void* dweight, void* stream);
int fp8_rmsnorm_backward_workspace(int64_t rows, int64_t cols, size_t* bytes);

/*
 * fp8_moe_route -- the top_k experts of every token and their weights.
 *
 *   s = softmax(logits) over the experts, or sigmoid(logits)
 *   key = s + bias (s without a bias)
 *   groups > 1: the experts form `groups` equal runs of consecutive indices;
 *     the topk_groups groups ranked highest (group_score) stay
 *   ids = the top_k experts of the highest keys, highest first
 *   weights = s[ids] (the bias ranks only), divided by their sum with
 *     renorm, times `scale`
 * Ties go to the lowest index, of groups and of experts.  Choices are those
 * of the scores in double precision (without a bias: of the logits
 * themselves); weights are computed in fp32, off by at most 2^-18 + 2^-22 L
 * of their value, L the largest difference of two finite logits of the token
 * (about 2^-24 for usual logits).
 *
 * logits [tokens x experts] bf16 or float per logits_type (4-byte aligned,
 *        bf16 2-byte).  An expert whose logit is -inf or NaN is masked: its
 *        score is 0 and it is never chosen.  One whose bias is -inf or NaN
 *        is never chosen either (a softmax still counts it).  +inf counts as
 *        the largest float.  A group's two best keys are those of experts
 *        that can be chosen; a group with none ranks last.  A token with
 *        fewer than top_k experts to choose from gets id -1 and weight 0 in
 *        the places that remain.
 * bias   optional (NULL = none) [experts] float (4-byte aligned);
 * ids    [tokens x top_k] int32 out; weights [tokens x top_k] float out.
 * Shape: tokens >= 0, tokens * top_k <= 2^30, 1 <= experts <= 1024, 1 <=
 *        groups <= 64, experts % groups == 0, 1 <= topk_groups <= groups,
 *        1 <= top_k <= 64, top_k <= topk_groups * (experts / groups);
 *        renorm 0 or 1; scale finite.
 */
int fp8_moe_route(const void* logits, int logits_type, const float* bias, int64_t tokens, int experts, int top_k,
                  int score, int groups, int topk_groups, int group_score, int renorm, float scale, int32_t* ids,
                  float* weights, void* stream);

/*
 * fp8_moe_route_backward -- gradient of the weights with respect to the
 * logits (the choice itself has none, nor has the bias).
 *
 * logits, score, renorm, scale as in the forward call; ids its output (ids
 * outside [0, experts) carry no weight; an expert listed twice collects
 * both gradients); dweights [tokens x top_k] float; dlogits [tokens x
 * experts] out, of the logits' type, every element written (masked experts
 * get 0).
 */
int fp8_moe_route_backward(const void* logits, int logits_type, const int32_t* ids, const float* dweights,
                           int64_t tokens, int experts, int top_k, int score, int renorm, float scale, void* dlogits,
                           void* stream);

/*
 * fp8_moe_plan -- sorts the routed (token, choice) pairs by expert, for the
 * grouped products and the combination.
 *
 * ids [tokens x top_k] int32: expert of each pair; values outside
 *     [0, experts) leave the pair out;
 * offsets   [experts + 1] int32 out: rows of expert e are [off[e], off[e+1]);
 *     off[experts] is the number of pairs that take part;
 * row_index [tokens * top_k] int32 out: the token of each grouped row, rows
 *     of one expert in the order of their pairs; 0 behind off[experts];
 * slot      [tokens x top_k] int32 out: grouped row of each pair, -1 for a
 *     pair left out;
 * workspace: at least the bytes fp8_moe_plan_workspace reports (which can
 *     be 0; then NULL will do), 16-byte aligned, garbage before and after.
 * Shape: tokens >= 0, 1 <= top_k <= 64, tokens * top_k <= 2^30, 1 <= experts
 *     <= 1024.  tokens == 0 writes offsets of 0.
 */
int fp8_moe_plan(const int32_t* ids, int64_t tokens, int top_k, int experts, void* workspace, size_t workspace_bytes,
                 int32_t* offsets, int32_t* row_index, int32_t* slot, void* stream);
int fp8_moe_plan_workspace(int64_t tokens, int top_k, int experts, size_t* bytes);

/*
 * fp8_nvfp4_matvec -- products of a few bf16 rows with an NVFP4 matrix:
 *   y[i][j] = sum over k of x[i][k] * e2m1(code[j][k]) * e4m3(S[j][k / 16]) * g[j / rows_per_tensor]
 * with exact products, fp32 sums (the scale g multiplies the sum) and one
 * rounding to y's type.  Meant for 1 to about 32 rows (of each group, in the
 * grouped call); more are taken 16 or 32 at a time and read the weights
 * again for each.  The order of a row's sum depends on the sizes of the call
 * and of its group, so a row can differ in its last bits from the same row
 * in a call of another size.  A scale byte that is NaN makes its products
 * NaN.
 *
 * x [m x k] bf16 (16-byte aligned); q [n x k/2] codes, block_scale
 * [n x k/16], global_scale [n / rows_per_tensor] float as written by
 * fp8_nvfp4_quantize (q 8-byte aligned); y [m x n] out, bf16 or float per
 * y_type (aligned to its element).
 * Shape: 0 <= m < 2^31, 0 <= n <= 2^24, rows_per_tensor >= 1, n %
 *        rows_per_tensor == 0, k % 16 == 0, 0 < k <= 2^24, m * k < 2^30;
 *        m == 0 or n == 0 enqueues nothing.
 */
int fp8_nvfp4_matvec(const uint16_t* x, const uint8_t* q, const uint8_t* block_scale, const float* global_scale,
                     int64_t rows_per_tensor, int64_t m, int64_t n, int64_t k, void* y, int y_type, void* stream);

/*
 * fp8_nvfp4_grouped_matvec -- the same over routed experts: rows
 * [off[g], off[g+1]) of y take matrix g of q [groups x n x k/2], block_scale
 * [groups x n x k/16] and global_scale [groups * n / rows_per_tensor], and
 * row i reads x[row_index[i]] (x[i] where row_index is NULL).
 *
 * group_offsets, row_index, total_m and x_rows behave as in
 * fp8_grouped_gemm_gather: device int32 arrays that are not checked on the
 * host, with offsets clamped into [0, total_m] and indices into [0, x_rows).
 * Rows of y at or behind off[groups] are left as they were.
 * Shape: 1 <= groups <= 1024, 0 <= total_m < 2^31, x_rows >= 1 where there
 *        are rows (x_rows == total_m without row_index), x_rows * k < 2^30;
 *        n, k as above.
 */
int fp8_nvfp4_grouped_matvec(const uint16_t* x, int64_t x_rows, const int32_t* row_index, const uint8_t* q,
                             const uint8_t* block_scale, const float* global_scale, int64_t rows_per_tensor,
                             const int32_t* group_offsets, int64_t groups, int64_t total_m, int64_t n, int64_t k,
                             void* y, int y_type, void* stream);

/*
 * fp8_moe_combine -- the experts' rows back into tokens:
 *   y[t] = residual[t] + sum over j of weights[t][j] * rows[slot[t][j]]
 * in fp32, j ascending, rounded once to y's type.  Slots outside
 * [0, total_m) take no part (their weight is not looked at).
 *
 * rows [total_m x n] bf16 or float per row_type (16-byte aligned; NULL where
 * total_m == 0); slot [tokens x top_k] int32 (fp8_moe_plan's); weights
 * [tokens x top_k] float; residual optional (NULL = none) [tokens x n] bf16
 * (16-byte aligned); y [tokens x n] out, bf16 or float per y_type (16-byte
 * aligned; of type bf16 it may be residual itself).
 * Shape: tokens >= 0, total_m >= 0, both < 2^31, 1 <= top_k <= 64,
 *        n % 8 == 0, 0 <= n <= 2^24.
 */
int fp8_moe_combine(const void* rows, int row_type, int64_t total_m, const int32_t* slot, const float* weights,
                    const uint16_t* residual, int64_t tokens, int top_k, int64_t n, void* y, int y_type,
                    void* stream);

/*
 * fp8_moe_combine_backward -- gradients of the combination:
 *   drows[slot[t][j]] = weights[t][j] * dy[t],  dweights[t][j] = <dy[t], rows[slot[t][j]]>
 * (the residual's gradient is dy itself).  drows is of row_type, rounded
 * once; rows that no slot names are left as they were.  Slots are distinct,
 * as fp8_moe_plan's are; a row that two slots name ends with elements of
 * either gradient.  A slot outside [0, total_m) gets dweight 0, whatever dy
 * holds.
 *
 * dy [tokens x n] bf16 or float per dy_type; other arguments as above.
 */
int fp8_moe_combine_backward(const void* dy, int dy_type, const void* rows, int row_type, int64_t total_m,
                             const int32_t* slot, const float* weights, int64_t tokens, int top_k, int64_t n,
                             void* drows, float* dweights, void* stream);

/* FP8BLK_MOE_ABI_VERSION of the loaded library. */
int fp8_moe_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8BLK_MOE_H */
