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

}  // namespace tbe
