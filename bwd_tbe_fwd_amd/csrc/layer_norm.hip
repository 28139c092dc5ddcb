// Layer norm: argument validation, workspace, dispatch and the final sum of the backward's
// partial rows.  Declarations and the meaning of every argument are in include/tbe_tower.h;
// the kernels are in layer_norm.h.
#include "layer_norm.h"

#include <initializer_list>

#include "../../include/tbe_tower.h"

namespace tbe {
namespace {

// Final sum of the partial rows [P][2][width], in a fixed order: a workgroup takes 16 columns, its 64
// groups of 16 lanes the rows g, g + 64, ..., 4 of them in flight, then 16 lanes add the 64 sums.  64
// columns and 16 groups left 1024 rows of 1001 columns to 32 workgroups that waited for one row
// after the other.
constexpr int kSumCols = 16, kSumGroups = 64;
__global__ __launch_bounds__(kSumCols * kSumGroups) void norm_partials_kernel(const float* __restrict__ partial, int P,
                                                                             int64_t width, void* gw, void* gb, int dt) {
  __shared__ float s[kSumGroups][kSumCols + 1];
  const int g = threadIdx.x / kSumCols, l = threadIdx.x % kSumCols;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kSumCols + l;
  float sum = 0.0f;
  if (c < 2 * width) {
    const float* p = partial + c;
#pragma unroll 4
    for (int r = g; r < P; r += kSumGroups) sum += p[static_cast<int64_t>(r) * 2 * width];
  }
  s[g][l] = sum;
  __syncthreads();
  if (g || c >= 2 * width) return;
  sum = 0.0f;
#pragma unroll 8
  for (int k = 0; k < kSumGroups; ++k) sum += s[k][l];
  if (c < width) {
    if (gw) store_any(gw, dt, c, sum);
  } else if (gb) {
    store_any(gb, dt, c - width, sum);
  }
}

bool dtype_ok(int dt) { return dt == TBE_F32 || dt == TBE_F16 || dt == TBE_BF16; }
bool aligned_to(const void* p, int dt) { return !(reinterpret_cast<uintptr_t>(p) & (dt == TBE_F32 ? 3u : 1u)); }

// Whether every row starts on 16 bytes.
bool rows_on_16(const void* p, int64_t stride, int dt) {
  return !(reinterpret_cast<uintptr_t>(p) & 15) && stride * (dt == TBE_F32 ? 4 : 2) % 16 == 0;
}

// What both directions ask of a row matrix.
tbe_status check_rows(const char* what, const void* p, int64_t stride, int dt, int64_t rows, int64_t width) {
  if (!dtype_ok(dt)) {
    set_error("%s: unknown type %d", what, dt);
    return TBE_ERR_UNSUPPORTED;
  }
  if (rows > 0 && (!p || !aligned_to(p, dt))) {
    set_error("%s is NULL or not aligned to its element", what);
    return TBE_ERR_ARG;
  }
  // the last element's index stays within 64 bits
  if (rows > 1 && (stride < width || stride > (int64_t{1} << 31))) {
    set_error("%s: rows of %lld elements cannot be %lld apart", what, static_cast<long long>(width),
              static_cast<long long>(stride));
    return TBE_ERR_ARG;
  }
  return TBE_OK;
}

tbe_status check_sizes(int64_t rows, int64_t width) {
  if (rows < 0 || rows > 0x7fffffffll || width < 1 || width > TBE_LAYER_NORM_MAX_WIDTH) {
    set_error("layer norm: %lld rows of %lld elements (0 <= rows < 2^31, 1 <= width <= %d)", static_cast<long long>(rows),
              static_cast<long long>(width), TBE_LAYER_NORM_MAX_WIDTH);
    return rows < 0 || width < 1 ? TBE_ERR_ARG : TBE_ERR_UNSUPPORTED;
  }
  return TBE_OK;
}

tbe_status check_vectors(std::initializer_list<const void*> ps, int dt) {
  for (const void* p : ps) {
    if (!p) continue;
    if (!dtype_ok(dt)) {
      set_error("layer norm: unknown type %d of weight and bias", dt);
      return TBE_ERR_UNSUPPORTED;
    }
    if (!aligned_to(p, dt)) {
      set_error("layer norm: weight, bias and their gradients are aligned to their element");
      return TBE_ERR_ARG;
    }
  }
  return TBE_OK;
}

}  // namespace
}  // namespace tbe

using namespace tbe;

extern "C" tbe_status tbe_layer_norm_forward(int64_t rows, int64_t width, const void* x, int64_t x_stride, int32_t x_dtype,
                                             const void* weight, const void* bias, int32_t w_dtype, float eps, void* y,
                                             int64_t y_stride, int32_t y_dtype, float* mean, float* rstd,
                                             tbe_stream_t stream) {
  clear_error();
  tbe_status st = check_sizes(rows, width);
  if (st == TBE_OK) st = check_rows("x", x, x_stride, x_dtype, rows, width);
  if (st == TBE_OK) st = check_rows("y", y, y_stride, y_dtype, rows, width);
  if (st == TBE_OK) st = check_vectors({weight, bias}, w_dtype);
  if (st != TBE_OK) return st;
  if (!(eps >= 0.0f)) {
    set_error("layer norm: eps is %g, it is at least 0", static_cast<double>(eps));
    return TBE_ERR_ARG;
  }
  if (!aligned_to(mean, TBE_F32) || !aligned_to(rstd, TBE_F32)) {
    set_error("layer norm: mean and rstd are aligned to their element");
    return TBE_ERR_ARG;
  }
  if (rows == 0) return TBE_OK;
  NormArgs a = {};
  a.rows = rows; a.width = width; a.x = x; a.x_stride = x_stride;
  a.w = weight; a.b = bias; a.w_dt = w_dtype; a.eps = eps;
  a.y = y; a.y_stride = y_stride; a.mean = mean; a.rstd = rstd;
  a.stream = rows_on_16(y, rows > 1 ? y_stride : 0, y_dtype);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return x_dtype == TBE_F32 ? norm_forward_x<0>(a, y_dtype, s)
                            : x_dtype == TBE_F16 ? norm_forward_x<1>(a, y_dtype, s) : norm_forward_x<2>(a, y_dtype, s);
}

extern "C" size_t tbe_layer_norm_backward_workspace_bytes(int64_t rows, int64_t width) {
  if (rows < 0 || width < 1 || width > TBE_LAYER_NORM_MAX_WIDTH) return 0;
  return static_cast<size_t>(hmax(1, hmin(rows, norm_partials(width))) * 2 * width * 4);
}

extern "C" tbe_status tbe_layer_norm_backward(int64_t rows, int64_t width, const void* x, int64_t x_stride, int32_t x_dtype,
                                              const void* grad_y, int64_t grad_y_stride, int32_t y_dtype, const float* mean,
                                              const float* rstd, const void* weight, int32_t w_dtype, void* grad_x,
                                              int64_t grad_x_stride, void* grad_weight, void* grad_bias, void* workspace,
                                              size_t workspace_bytes, tbe_stream_t stream) {
  clear_error();
  tbe_status st = check_sizes(rows, width);
  if (st == TBE_OK) st = check_rows("x", x, x_stride, x_dtype, rows, width);
  if (st == TBE_OK) st = check_rows("grad_y", grad_y, grad_y_stride, y_dtype, rows, width);
  if (st == TBE_OK && grad_x) st = check_rows("grad_x", grad_x, grad_x_stride, x_dtype, rows, width);
  if (st == TBE_OK) st = check_vectors({weight, grad_weight, grad_bias}, w_dtype);
  if (st != TBE_OK) return st;
  if (rows > 0 && (!mean || !rstd || !aligned_to(mean, TBE_F32) || !aligned_to(rstd, TBE_F32))) {
    set_error("layer norm: the backward reads the forward's mean and rstd");
    return TBE_ERR_ARG;
  }
  const bool sums = grad_weight || grad_bias;
  if (sums && rows > 0 &&
      (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) ||
       workspace_bytes < tbe_layer_norm_backward_workspace_bytes(rows, width))) {
    set_error("layer norm backward: workspace of %zu bytes, 256-byte aligned; %zu given",
              tbe_layer_norm_backward_workspace_bytes(rows, width), workspace ? workspace_bytes : 0);
    return TBE_ERR_WORKSPACE;
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  NormArgs a = {};
  a.rows = rows; a.width = width; a.x = x; a.x_stride = x_stride;
  a.w = weight; a.w_dt = w_dtype;
  a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
  a.gy = grad_y; a.gy_stride = grad_y_stride; a.gx = grad_x; a.gx_stride = grad_x_stride;
  a.stream = rows_on_16(grad_x, rows > 1 ? grad_x_stride : 0, x_dtype);
  a.partial = sums ? static_cast<float*>(workspace) : nullptr;
  int grid = 0;  // partial rows
  if (rows > 0 && (sums || grad_x)) {
    st = x_dtype == TBE_F32 ? norm_backward_x<0>(a, y_dtype, s, &grid)
                            : x_dtype == TBE_F16 ? norm_backward_x<1>(a, y_dtype, s, &grid)
                                                 : norm_backward_x<2>(a, y_dtype, s, &grid);
    if (st != TBE_OK) return st;
  }
  if (!sums) return TBE_OK;
  ProfScope ps("norm_partials", s);
  hipLaunchKernelGGL(norm_partials_kernel, dim3((2 * width + kSumCols - 1) / kSumCols), dim3(kSumCols * kSumGroups), 0, s, a.partial, grid,
                     width, grad_weight, grad_bias, w_dtype);
  return check_launch("norm_partials");
}
