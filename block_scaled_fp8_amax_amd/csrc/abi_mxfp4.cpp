// C-ABI entry points of the MXFP4 codec and products and of the experts'
// gradients: argument validation and kernel dispatch.  The declarations and
// their contracts are in include/fp8blk_mxfp4.h.
#include "fp8blk_mxfp4.h"

#include <hip/hip_runtime.h>

#include "host.h"
#include "launch.h"

namespace {

using namespace fp8blk;

bool valid_type(int t) { return t == FP8_OUT_BF16 || t == FP8_OUT_F32; }
uintptr_t type_bytes(int t) { return t == FP8_OUT_F32 ? 4 : 2; }
hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

constexpr int64_t kMaxRows = 0x7FFFFFFFll;
constexpr int64_t kMaxWidth = int64_t(1) << 24;
// Blocks of 32 elements of a codec call: their number fits 32 bits.
constexpr int64_t kMaxBlocks = (int64_t(1) << 32) - (int64_t(1) << 20);
// Rows of a gradient's tile are read with 32-bit byte offsets.
constexpr int64_t kMaxGradWidth = int64_t(1) << 22;
// x of a matvec is read with 32-bit byte offsets whose top bit is free.
constexpr int64_t kMaxMatvecX = (int64_t(1) << 30) - 1;

int codec_shape(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || cols % 32 || !product_at_most(rows, cols / 32, kMaxBlocks)) return FP8_ERR_SHAPE;
  return FP8_OK;
}

int product_shape(int64_t m, int64_t n, int64_t k, int64_t multiple, int y_type) {
  if (!valid_type(y_type)) return FP8_ERR_INVALID_ARG;
  if (m < 0 || m > kMaxRows || n < 0 || n > kMaxWidth || k <= 0 || k > kMaxWidth || k % multiple) return FP8_ERR_SHAPE;
  return FP8_OK;
}

int gradient_shape(int64_t groups, int64_t total_m, int64_t n, int64_t k, int type) {
  if (!valid_type(type)) return FP8_ERR_INVALID_ARG;
  if (groups < 1 || groups > 1024) return FP8_ERR_INVALID_ARG;
  if (total_m < 0 || total_m > kMaxRows || n < 0 || n > kMaxGradWidth || k < 0 || k > kMaxGradWidth || n % 8 || k % 8 ||
      n * k > kMaxRows)
    return FP8_ERR_SHAPE;
  return FP8_OK;
}

// Rows that grouped rows are read from: as many as there are, or gathered.
int source_rows(int64_t rows, const int32_t* row_index, int64_t total_m, int64_t k, int64_t most) {
  if (rows < 1 || rows > kMaxRows || (!row_index && rows != total_m)) return FP8_ERR_SHAPE;
  if (row_index && !product_at_most(rows, k, most)) return FP8_ERR_SHAPE;
  return FP8_OK;
}

}  // namespace

extern "C" {

int fp8_mxfp4_abi_version(void) { return FP8BLK_MXFP4_ABI_VERSION; }

int fp8_mxfp4_quantize(const uint16_t* x, int64_t rows, int64_t cols, int rule, uint8_t* q, uint8_t* scale,
                       uint16_t* xdq, void* stream) {
  if (rule != FP8_E8M0_CEIL && rule != FP8_E8M0_FLOOR) return FP8_ERR_INVALID_ARG;
  if (int s = codec_shape(rows, cols)) return s;
  if (rows == 0 || cols == 0) return FP8_OK;
  if (!x || !q || !scale) return FP8_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(xdq, 16)) return FP8_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if (int s = current_device(&dev)) return s;
  return hip_status(launch_mxfp4_quant(x, rows, cols, rule == FP8_E8M0_FLOOR, q, scale, xdq, as_stream(stream)));
}

int fp8_mxfp4_dequantize(const uint8_t* q, const uint8_t* scale, int64_t rows, int64_t cols, uint16_t* x,
                         void* stream) {
  if (int s = codec_shape(rows, cols)) return s;
  if (rows == 0 || cols == 0) return FP8_OK;
  if (!x || !q || !scale) return FP8_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 16)) return FP8_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if (int s = current_device(&dev)) return s;
  return hip_status(launch_mxfp4_dequant(q, scale, rows, cols, x, as_stream(stream)));
}

static int mx_product(const uint8_t* a_q, const uint8_t* a_scale, int a_elem, int64_t a_rows,
                      const int32_t* row_index, const uint8_t* b_q, const uint8_t* b_scale, const int32_t* offsets,
                      int64_t groups, int64_t m, int64_t n, int64_t k, void* y, int y_type, void* stream) {
  if (!a_q || !a_scale || !b_q || !b_scale || !y) return FP8_ERR_INVALID_ARG;
  if (!aligned(a_q, 16) || !aligned(b_q, 16) || !aligned(a_scale, 4) || !aligned(b_scale, 4) || !aligned(y, 16) ||
      !aligned(row_index, 4) || !aligned(offsets, 4))
    return FP8_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if (int s = current_device(&dev)) return s;
  MxProduct p{a_q, a_scale, a_elem == FP8_MX_E2M1, a_rows, row_index, b_q, b_scale, offsets, (int)groups, m, n, k, y,
              y_type == FP8_OUT_F32};
  return hip_status(launch_mx_product(p, dev->num_cu, as_stream(stream)));
}

int fp8_mxfp4_gemm(const uint8_t* a_q, const uint8_t* a_scale, int a_elem, const uint8_t* b_q,
                   const uint8_t* b_scale, int64_t m, int64_t n, int64_t k, void* y, int y_type, void* stream) {
  if (a_elem != FP8_MX_E4M3 && a_elem != FP8_MX_E2M1) return FP8_ERR_INVALID_ARG;
  if (int s = product_shape(m, n, k, 128, y_type)) return s;
  if (m == 0 || n == 0) return FP8_OK;
  return mx_product(a_q, a_scale, a_elem, m, nullptr, b_q, b_scale, nullptr, 1, m, n, k, y, y_type, stream);
}

int fp8_mxfp4_grouped_gemm(const uint8_t* a_q, const uint8_t* a_scale, int a_elem, int64_t a_rows,
                           const int32_t* row_index, const uint8_t* b_q, const uint8_t* b_scale,
                           const int32_t* group_offsets, int64_t groups, int64_t total_m, int64_t n, int64_t k,
                           void* y, int y_type, void* stream) {
  if (a_elem != FP8_MX_E4M3 && a_elem != FP8_MX_E2M1) return FP8_ERR_INVALID_ARG;
  if (int s = product_shape(total_m, n, k, 128, y_type)) return s;
  if (groups < 1 || groups > 1024) return FP8_ERR_INVALID_ARG;
  if (total_m == 0 || n == 0) return FP8_OK;
  if (int s = source_rows(a_rows, row_index, total_m, k, 0xFFFFFFFFll)) return s;
  if (!group_offsets) return FP8_ERR_INVALID_ARG;
  return mx_product(a_q, a_scale, a_elem, a_rows, row_index, b_q, b_scale, group_offsets, groups, total_m, n, k, y,
                    y_type, stream);
}

static int mx_rows(const uint16_t* x, int64_t x_rows, const int32_t* row_index, const uint8_t* q,
                   const uint8_t* scale, const int32_t* offsets, int64_t groups, int64_t m, int64_t n, int64_t k,
                   void* y, int y_type, void* stream) {
  if (!x || !q || !scale || !y) return FP8_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(y, type_bytes(y_type)) || !aligned(row_index, 4) ||
      !aligned(offsets, 4))
    return FP8_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if (int s = current_device(&dev)) return s;
  MxRows a{x, x_rows, row_index, q, scale, offsets, groups, m, n, k, y, y_type == FP8_OUT_F32};
  return hip_status(launch_mx_rows(a, as_stream(stream)));
}

int fp8_mxfp4_matvec(const uint16_t* x, const uint8_t* q, const uint8_t* scale, int64_t m, int64_t n, int64_t k,
                     void* y, int y_type, void* stream) {
  if (int s = product_shape(m, n, k, 32, y_type)) return s;
  if (!product_at_most(m, k, kMaxMatvecX)) return FP8_ERR_SHAPE;
  if (m == 0 || n == 0) return FP8_OK;
  return mx_rows(x, m, nullptr, q, scale, nullptr, 1, m, n, k, y, y_type, stream);
}

int fp8_mxfp4_grouped_matvec(const uint16_t* x, int64_t x_rows, const int32_t* row_index, const uint8_t* q,
                             const uint8_t* scale, const int32_t* group_offsets, int64_t groups, int64_t total_m,
                             int64_t n, int64_t k, void* y, int y_type, void* stream) {
  if (int s = product_shape(total_m, n, k, 32, y_type)) return s;
  if (groups < 1 || groups > 1024) return FP8_ERR_INVALID_ARG;
  if (x_rows < 0 || !product_at_most(x_rows, k, kMaxMatvecX)) return FP8_ERR_SHAPE;
  if (total_m == 0 || n == 0) return FP8_OK;
  if (int s = source_rows(x_rows, row_index, total_m, k, kMaxMatvecX)) return s;
  if (!group_offsets) return FP8_ERR_INVALID_ARG;
  return mx_rows(x, x_rows, row_index, q, scale, group_offsets, groups, total_m, n, k, y, y_type, stream);
}

int fp8_grouped_dgrad(const uint16_t* dy, const uint16_t* w, const int32_t* group_offsets, int64_t groups,
                      int64_t total_m, int64_t n, int64_t k, void* dx, int dx_type, void* stream) {
  if (int s = gradient_shape(groups, total_m, n, k, dx_type)) return s;
  if (total_m == 0 || k == 0) return FP8_OK;
  if ((n > 0 && (!dy || !w)) || !group_offsets || !dx) return FP8_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(w, 16) || !aligned(group_offsets, 4) || !aligned(dx, 16)) return FP8_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if (int s = current_device(&dev)) return s;
  GroupedGrad a{dy, nullptr, 0, nullptr, w, group_offsets, (int)groups, total_m, n, k, dx, dx_type == FP8_OUT_F32};
  return hip_status(launch_grouped_dgrad(a, dev->num_cu, as_stream(stream)));
}

int fp8_grouped_wgrad(const uint16_t* dy, const uint16_t* x, int64_t x_rows, const int32_t* row_index,
                      const int32_t* group_offsets, int64_t groups, int64_t total_m, int64_t n, int64_t k, void* dw,
                      int dw_type, void* stream) {
  if (int s = gradient_shape(groups, total_m, n, k, dw_type)) return s;
  if (n == 0 || k == 0) return FP8_OK;
  if (total_m > 0) {
    if (int s = source_rows(x_rows, row_index, total_m, k, kMaxRows)) return s;
    if (!dy || !x) return FP8_ERR_INVALID_ARG;
  }
  if (!group_offsets || !dw) return FP8_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(row_index, 4) || !aligned(group_offsets, 4) || !aligned(dw, 16))
    return FP8_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if (int s = current_device(&dev)) return s;
  GroupedGrad a{dy, x, x_rows, row_index, nullptr, group_offsets, (int)groups, total_m, n, k, dw,
                dw_type == FP8_OUT_F32};
  return hip_status(launch_grouped_wgrad(a, dev->num_cu, as_stream(stream)));
}

}  // extern "C"
