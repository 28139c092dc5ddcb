// Host-side internals of the operators of include/tbe_items.h.
#pragma once

#include <type_traits>

#include "../../include/tbe_items.h"
#include "tbe_internal.h"

namespace tbe {

// Whether every row starts on 16 bytes.
inline bool rows_on_16(const void* p, int64_t stride, int dt) {
  return !(reinterpret_cast<uintptr_t>(p) & 15) && stride * (dt == TBE_F32 ? 4 : 2) % 16 == 0;
}

tbe_status launch_lookup_forward(int64_t n, int64_t items, int64_t width, const void* table, int64_t table_stride, int table_dtype,
                                 const void* ids, int id_type, float scale, void* y, int64_t y_stride, int y_dtype, hipStream_t s);
size_t lookup_backward_workspace(int64_t n, int64_t items, int64_t width);
tbe_status launch_lookup_backward(int64_t n, int64_t items, int64_t width, const void* ids, int id_type, const void* gy,
                                  int64_t gy_stride, int y_dtype, float scale, void* grad, int64_t grad_stride, int table_dtype,
                                  bool add, void* workspace, hipStream_t s);


size_t cross_entropy_forward_workspace(int64_t rows, int64_t items, int64_t width);
size_t cross_entropy_backward_workspace(int64_t rows, int64_t items, int64_t width);
tbe_status launch_cross_entropy_forward(int64_t rows, int64_t items, int64_t width, const void* x, int64_t x_stride, const void* weight,
                                        int64_t weight_stride, int dtype, const float* bias, const void* targets, int target_type,
                                        float scale, float* loss, float* lse, void* workspace, hipStream_t s);
tbe_status launch_cross_entropy_backward(int64_t rows, int64_t items, int64_t width, const void* x, int64_t x_stride, const void* weight,
                                         int64_t weight_stride, int dtype, const float* bias, const void* targets, int target_type,
                                         float scale, const float* lse, const float* grad_loss, void* grad_x, int64_t grad_x_stride,
                                         void* grad_weight, int64_t grad_weight_stride, float* grad_bias, void* workspace, hipStream_t s);

}  // namespace tbe
