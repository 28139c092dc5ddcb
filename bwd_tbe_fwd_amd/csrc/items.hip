// The entry points of include/tbe_items.h: what they refuse before anything is launched.
#include "items.h"

using namespace tbe;

namespace {

bool dtype_ok(int dt) { return dt == TBE_F32 || dt == TBE_F16 || dt == TBE_BF16; }
bool aligned_to(const void* p, int dt) { return !(reinterpret_cast<uintptr_t>(p) & (dt == TBE_F32 ? 3u : 1u)); }

tbe_status check_matrix(const char* what, const void* p, int dt, int64_t rows, int64_t width, int64_t stride) {
  if (!dtype_ok(dt)) {
    set_error("%s: unknown type %d", what, dt);
    return TBE_ERR_UNSUPPORTED;
  }
  if (rows > 0 && (!p || !aligned_to(p, dt))) {
    set_error("%s is NULL or not aligned to its element", what);
    return TBE_ERR_ARG;
  }
  if (rows > 1 && (stride < width || stride > (int64_t{1} << 31))) {
    set_error("%s: rows of %lld elements cannot be %lld apart", what, static_cast<long long>(width), static_cast<long long>(stride));
    return TBE_ERR_ARG;
  }
  return TBE_OK;
}
tbe_status check_ids(const char* what, const void* p, int type, int64_t n) {
  if (type != TBE_I32 && type != TBE_I64) {
    set_error("%s: unknown type %d", what, type);
    return TBE_ERR_ARG;
  }
  if (n > 0 && (!p || (reinterpret_cast<uintptr_t>(p) & (type == TBE_I32 ? 3u : 7u)))) {
    set_error("%s are NULL or not aligned to their element", what);
    return TBE_ERR_ARG;
  }
  return TBE_OK;
}
tbe_status check_workspace(const char* what, const void* workspace, size_t given, size_t need) {
  if (need && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || given < need)) {
    set_error("%s: workspace of %zu bytes, 256-byte aligned; %zu given", what, need, workspace ? given : 0);
    return TBE_ERR_WORKSPACE;
  }
  return TBE_OK;
}

constexpr int64_t kMaxItems = (int64_t{1} << 31) - 2;
bool lookup_sizes_ok(int64_t n, int64_t items, int64_t width) {
  return n >= 0 && n <= TBE_MAX_LOOKUPS && items >= 1 && items <= kMaxItems && width >= 1 && width <= TBE_ITEMS_MAX_WIDTH;
}
tbe_status check_lookup(int64_t n, int64_t items, int64_t width) {
  if (lookup_sizes_ok(n, items, width)) return TBE_OK;
  set_error("lookup: %lld ids, %lld items of width %lld (0 <= ids <= 2^31 - 4096, 1 <= items < 2^31 - 1, 1 <= width <= %d)",
            static_cast<long long>(n), static_cast<long long>(items), static_cast<long long>(width), TBE_ITEMS_MAX_WIDTH);
  return n < 0 || items < 1 || width < 1 ? TBE_ERR_ARG : TBE_ERR_UNSUPPORTED;
}

bool loss_sizes_ok(int64_t rows, int64_t items, int64_t width) {
  return rows >= 0 && rows <= TBE_CROSS_ENTROPY_MAX_ROWS && items >= 1 && items <= kMaxItems && width >= 1 &&
         width <= TBE_CROSS_ENTROPY_MAX_WIDTH;
}
// What both directions ask.
tbe_status check_loss(int64_t rows, int64_t items, int64_t width, const void* x, int64_t x_stride, const void* weight,
                      int64_t weight_stride, int dtype, const float* bias, const void* targets, int target_type, float scale) {
  if (!loss_sizes_ok(rows, items, width)) {
    set_error("cross entropy: %lld rows, %lld items of width %lld (0 <= rows <= %d, 1 <= items < 2^31 - 1, 1 <= width <= %d)",
              static_cast<long long>(rows), static_cast<long long>(items), static_cast<long long>(width), TBE_CROSS_ENTROPY_MAX_ROWS,
              TBE_CROSS_ENTROPY_MAX_WIDTH);
    return rows < 0 || items < 1 || width < 1 ? TBE_ERR_ARG : TBE_ERR_UNSUPPORTED;
  }
  if (dtype != TBE_F16 && dtype != TBE_BF16) {
    set_error("cross entropy: type %d (fp16 or bf16)", dtype);
    return TBE_ERR_UNSUPPORTED;
  }
  if (!(scale - scale == 0.0f)) {
    set_error("cross entropy: scale is not finite");
    return TBE_ERR_ARG;
  }
  const float size = scale < 0.0f ? -scale : scale;  // biases are divided by it
  if (size != 0.0f && (size < 0x1p-64f || size > 0x1p64f)) {
    set_error("cross entropy: scale %g (0, or from 2^-64 to 2^64)", static_cast<double>(scale));
    return TBE_ERR_UNSUPPORTED;
  }
  tbe_status st = check_matrix("x", x, dtype, rows, width, x_stride);
  if (st == TBE_OK) st = check_matrix("weight", weight, dtype, items, width, weight_stride);
  if (st == TBE_OK && bias) st = check_matrix("bias", bias, TBE_F32, 1, items, items);
  if (st == TBE_OK) st = check_ids("targets", targets, target_type, rows);
  return st;
}

}  // namespace

extern "C" size_t tbe_cross_entropy_forward_workspace_bytes(int64_t rows, int64_t items, int64_t width) {
  return loss_sizes_ok(rows, items, width) ? cross_entropy_forward_workspace(rows, items, width) : 0;
}
extern "C" size_t tbe_cross_entropy_backward_workspace_bytes(int64_t rows, int64_t items, int64_t width) {
  return loss_sizes_ok(rows, items, width) ? cross_entropy_backward_workspace(rows, items, width) : 0;
}

extern "C" tbe_status tbe_cross_entropy_forward(int64_t rows, int64_t items, int64_t width, const void* x, int64_t x_stride,
                                                const void* weight, int64_t weight_stride, int32_t dtype, const float* bias,
                                                const void* targets, int32_t target_type, float scale, float* loss, float* lse,
                                                void* workspace, size_t workspace_bytes, tbe_stream_t stream) {
  clear_error();
  tbe_status st = check_loss(rows, items, width, x, x_stride, weight, weight_stride, dtype, bias, targets, target_type, scale);
  if (st == TBE_OK) st = check_matrix("loss", loss, TBE_F32, rows, 1, 1);
  if (st == TBE_OK) st = check_matrix("lse", lse, TBE_F32, rows, 1, 1);
  if (st != TBE_OK || rows == 0) return st;
  st = check_workspace("cross entropy", workspace, workspace_bytes, cross_entropy_forward_workspace(rows, items, width));
  if (st != TBE_OK) return st;
  return launch_cross_entropy_forward(rows, items, width, x, x_stride, weight, weight_stride, dtype, bias, targets, target_type, scale,
                                      loss, lse, workspace, static_cast<hipStream_t>(stream));
}

extern "C" tbe_status tbe_cross_entropy_backward(int64_t rows, int64_t items, int64_t width, const void* x, int64_t x_stride,
                                                 const void* weight, int64_t weight_stride, int32_t dtype, const float* bias,
                                                 const void* targets, int32_t target_type, float scale, const float* lse,
                                                 const float* grad_loss, void* grad_x, int64_t grad_x_stride, void* grad_weight,
                                                 int64_t grad_weight_stride, float* grad_bias, void* workspace, size_t workspace_bytes,
                                                 tbe_stream_t stream) {
  clear_error();
  tbe_status st = check_loss(rows, items, width, x, x_stride, weight, weight_stride, dtype, bias, targets, target_type, scale);
  if (st == TBE_OK) st = check_matrix("lse", lse, TBE_F32, rows, 1, 1);
  if (st == TBE_OK) st = check_matrix("grad_loss", grad_loss, TBE_F32, rows, 1, 1);
  if (st == TBE_OK && grad_x) st = check_matrix("grad_x", grad_x, dtype, rows, width, grad_x_stride);
  if (st == TBE_OK && grad_weight) st = check_matrix("grad_weight", grad_weight, dtype, items, width, grad_weight_stride);
  if (st == TBE_OK && grad_bias) st = check_matrix("grad_bias", grad_bias, TBE_F32, 1, items, items);
  if (st == TBE_OK)
    st = check_workspace("cross entropy backward", workspace, workspace_bytes, cross_entropy_backward_workspace(rows, items, width));
  if (st != TBE_OK || (!grad_x && !grad_weight && !grad_bias)) return st;
  return launch_cross_entropy_backward(rows, items, width, x, x_stride, weight, weight_stride, dtype, bias, targets, target_type, scale,
                                       lse, grad_loss, grad_x, grad_x_stride, grad_weight, grad_weight_stride, grad_bias, workspace,
                                       static_cast<hipStream_t>(stream));
}

extern "C" tbe_status tbe_lookup_forward(int64_t num_ids, int64_t items, int64_t width, const void* table, int64_t table_stride,
                                         int32_t table_dtype, const void* ids, int32_t id_type, float scale, void* y,
                                         int64_t y_stride, int32_t y_dtype, tbe_stream_t stream) {
  clear_error();
  tbe_status st = check_lookup(num_ids, items, width);
  if (st == TBE_OK) st = check_matrix("table", table, table_dtype, items, width, table_stride);
  if (st == TBE_OK) st = check_ids("ids", ids, id_type, num_ids);
  if (st == TBE_OK) st = check_matrix("y", y, y_dtype, num_ids, width, y_stride);
  if (st != TBE_OK || num_ids == 0) return st;
  return launch_lookup_forward(num_ids, items, width, table, table_stride, table_dtype, ids, id_type, scale, y, y_stride, y_dtype,
                               static_cast<hipStream_t>(stream));
}

extern "C" size_t tbe_lookup_backward_workspace_bytes(int64_t num_ids, int64_t items, int64_t width) {
  return lookup_sizes_ok(num_ids, items, width) ? lookup_backward_workspace(num_ids, items, width) : 0;
}

extern "C" tbe_status tbe_lookup_backward(int64_t num_ids, int64_t items, int64_t width, const void* ids, int32_t id_type,
                                          const void* grad_y, int64_t grad_y_stride, int32_t y_dtype, float scale,
                                          void* grad_table, int64_t grad_table_stride, int32_t table_dtype, int32_t accumulate,
                                          void* workspace, size_t workspace_bytes, tbe_stream_t stream) {
  clear_error();
  tbe_status st = check_lookup(num_ids, items, width);
  if (st == TBE_OK) st = check_ids("ids", ids, id_type, num_ids);
  if (st == TBE_OK) st = check_matrix("grad_y", grad_y, y_dtype, num_ids, width, grad_y_stride);
  if (st == TBE_OK) st = check_matrix("grad_table", grad_table, table_dtype, items, width, grad_table_stride);
  if (st == TBE_OK)
    st = check_workspace("lookup backward", workspace, workspace_bytes, lookup_backward_workspace(num_ids, items, width));
  if (st != TBE_OK || (accumulate && num_ids == 0)) return st;
  return launch_lookup_backward(num_ids, items, width, ids, id_type, grad_y, grad_y_stride, y_dtype, scale, grad_table,
                                grad_table_stride, table_dtype, accumulate != 0, workspace, static_cast<hipStream_t>(stream));
}
