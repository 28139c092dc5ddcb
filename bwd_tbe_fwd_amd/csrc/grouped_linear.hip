// Linear layers of E experts on rows grouped by expert: argument validation, the weight gradient's
// shares and their sum.  The products are in grouped_tile.h, a translation unit each.
#include "grouped_linear.h"

#include "../../include/tbe_tower.h"

namespace tbe {
namespace {

// Sum of the units' partial weight gradients of the experts that have more than one, in the order of
// their rows; zeros for the experts without rows, which have no unit.
__global__ __launch_bounds__(kBlock) void grouped_reduce_kernel(GroupedArgs a) {
  const int e = blockIdx.y;
  const int64_t io = static_cast<int64_t>(a.inner) * a.outer, each = io + a.outer;
  auto units_of = [&](int k) {
    const RowRange r = rows_of(a, k);
    return (r.hi - r.lo + a.split - 1) / a.split;
  };
  int64_t n = units_of(e);
  if (n == 1) return;
  int64_t first = 0;  // units of the experts before that have several
  for (int k = lane_id(); k < e; k += kWave) {
    const int64_t u = units_of(k);
    first += u > 1 ? u : 0;
  }
  for (int d = 1; d < kWave; d <<= 1) first += __shfl_xor(first, d);
  n = min(n, max(a.slots - first, static_cast<int64_t>(0)));  // offsets that are not in order: inside the workspace
  const float* p = static_cast<const float*>(a.workspace) + first * each;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x) * 4; i < each; i += static_cast<int64_t>(gridDim.x) * kBlock * 4) {
    Vec<float, 4> sum = {};
    for (int64_t u = 0; u < n; ++u) {
      Vec<float, 4> v;
      load_vec_part<float, 4>(p + u * each + i, each - i, v);
#pragma unroll
      for (int k = 0; k < 4; ++k) sum.e[k] += v.e[k];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i + k < io) store_any(a.out, a.out_dt, e * io + i + k, sum.e[k]);
      else if (i + k < each && a.grad_bias) store_any(a.grad_bias, a.out_dt, static_cast<int64_t>(e) * a.outer + i + k - io, sum.e[k]);
    }
  }
}

// The weight gradient's tile and the rows of a unit.  With few tiles for the 256 CUs, an expert's rows
// are shared among workgroups, and a second kernel adds their partial sums: units of 512, 1024, ...
// rows (0: an expert's rows are one).  The least of the expected times: rounds of tiles, the last of
// them by an expert of twice the average rows where rows are not shared, and 4 TB/s for the partial
// sums' way to memory and back.  A step of 64 rows takes longer the more workgroups read their rows
// from memory at once.  Measured with tile and unit as given: 16384 rows, 1 expert, 4096 x 1024: 256, 4096
// rows 139 us; 256, all 398; 128, all 207; 64, all 227.  65536 rows, 16 experts, 1024 x 1024: 256, all 130
// us (the experts' rows unequal, 370); 256, 4096 rows 257 (205); 128, all 186 (238); 64, all 279 (263).  The
// plan sees sizes only, not the offsets: where rows are not shared, one expert with far more rows than twice
// the average decides (popularity 1 / rank^1.2, the largest 5.8 times the average, 538 us).
//
// Partial sums are kept for the units of experts that have several: an expert of n rows has at most n / split + 1,
// and at most rows / split experts have more than split rows.  A split that would need more bytes of them than
// 1 GiB, or an eighth of the operands' where that is more, is not taken: this changes no plan of up to 64 K rows
// with sides up to 4096, and of 20000 random sizes up to 2 M rows and 8192 it changes 36, by at most 9% of their
// expected time.  (824148 rows, 5204 x 4045, took 4.4 GB for a gradient of 84 MB: now 1.1 GB.)
int64_t most_partials(int64_t rows, int64_t inner, int64_t outer) { return hmax(int64_t{1} << 30, rows * (inner + outer) / 4); }
constexpr int64_t kLeastSplit = 512;
int64_t weight_slots(int64_t rows, int64_t experts, int64_t split) { return rows / split + hmin(experts, rows / split); }
int64_t slot_bytes(int64_t inner, int64_t outer) { return (inner + 1) * outer * 4; }

struct WeightPlan {
  int tile, split;
};
WeightPlan weight_plan(int64_t rows, int64_t experts, int64_t inner, int64_t outer) {
  WeightPlan p = {0, 0};
  double best = -1.0;
  const double used = static_cast<double>(hmax(1, hmin(experts, rows))), average = static_cast<double>(rows) / used;
  for (int t = 0; t < 3; ++t) {
    const TileCost& c = kWeightTiles[t];
    const int64_t tiles = ((outer + c.bm - 1) / c.bm) * ((inner + c.bn - 1) / c.bn);
    const double each = static_cast<double>(tiles);
    double us = tiles_us(c, used * each, average, experts > 1 ? 2.0 * average : average);
    if (best < 0.0 || (us < best && launch_takes(experts * tiles, c.threads))) {
      best = us;
      p = WeightPlan{t, 0};
    }
    for (int64_t split = kLeastSplit; split < rows && split <= (1 << 20); split *= 2) {
      if (!launch_takes(row_tiles_bound(rows, experts, split) * tiles, c.threads)) continue;
      if (weight_slots(rows, experts, split) > most_partials(rows, inner, outer) / slot_bytes(inner, outer)) continue;
      const double units = row_tiles_expected(rows, experts, static_cast<int>(split)), k = static_cast<double>(split);
      const double bytes = 4.0 * static_cast<double>(rows / split) * static_cast<double>(inner + 1) * static_cast<double>(outer);
      us = tiles_us(c, units * each, k, k) + 5.0 + 2.0 * bytes / 4e6;
      if (us < best) {
        best = us;
        p = WeightPlan{t, static_cast<int>(split)};
      }
    }
  }
  return p;
}

template <int OP>
tbe_status launch(const GroupedArgs& a, int dtype, hipStream_t s) {
  const tbe_status st = dtype == TBE_F16 ? grouped_launch<1, OP>(a, s) : grouped_launch<2, OP>(a, s);
  if (st != TBE_OK || OP != kBackwardWeight || !a.split) return st;
  const int64_t each = static_cast<int64_t>(a.inner + 1) * a.outer;
  ProfScope ps("grouped_reduce", s);
  hipLaunchKernelGGL(grouped_reduce_kernel, dim3(static_cast<unsigned>(hmin(1024, (each + 4 * kBlock - 1) / (4 * kBlock))), a.experts),
                     dim3(kBlock), 0, s, a);
  return check_launch("grouped_reduce");
}

bool aligned_to(const void* p, int dt) { return !(reinterpret_cast<uintptr_t>(p) & (dt == TBE_F32 ? 3u : 1u)); }

constexpr int64_t kMaxRows = int64_t{1} << 29;  // a launch has fewer than 2^32 threads
constexpr int64_t kMaxSide = int64_t{1} << 20;
constexpr int kMaxExperts = 65535;

tbe_status check_sizes(int64_t rows, int32_t experts, int64_t inner, int64_t outer, int dtype, int out_dtype,
                       const void* offsets, int offset_type) {
  if (rows < 0 || experts < 1 || inner < 1 || outer < 1) {
    set_error("grouped linear: %lld rows, %d experts, inner %lld, outer %lld", static_cast<long long>(rows), experts,
              static_cast<long long>(inner), static_cast<long long>(outer));
    return TBE_ERR_ARG;
  }
  if (rows > kMaxRows || experts > kMaxExperts || inner > kMaxSide || outer > kMaxSide) {
    set_error("grouped linear: %lld rows, %d experts, inner %lld, outer %lld are more than supported",
              static_cast<long long>(rows), experts, static_cast<long long>(inner), static_cast<long long>(outer));
    return TBE_ERR_UNSUPPORTED;
  }
  if ((dtype != TBE_F16 && dtype != TBE_BF16) || (out_dtype != dtype && out_dtype != TBE_F32)) {
    set_error("grouped linear: types %d -> %d (fp16 or bf16, to itself or fp32)", dtype, out_dtype);
    return TBE_ERR_UNSUPPORTED;
  }
  if (offset_type != TBE_I32 && offset_type != TBE_I64) {
    set_error("grouped linear: unknown offset type %d", offset_type);
    return TBE_ERR_ARG;
  }
  if (!offsets || (reinterpret_cast<uintptr_t>(offsets) & (offset_type == TBE_I32 ? 3u : 7u))) {
    set_error("grouped linear: offsets are NULL or not aligned to their element");
    return TBE_ERR_ARG;
  }
  return TBE_OK;
}
tbe_status check_matrix(const char* what, const void* p, int dt, int64_t rows, int64_t width, int64_t stride) {
  if (rows > 0 && (!p || !aligned_to(p, dt))) {
    set_error("grouped linear: %s is NULL or not aligned to its element", what);
    return TBE_ERR_ARG;
  }
  if (rows > 1 && (stride < width || stride > (int64_t{1} << 31))) {
    set_error("grouped linear: %s: rows of %lld elements cannot be %lld apart", what, static_cast<long long>(width),
              static_cast<long long>(stride));
    return TBE_ERR_ARG;
  }
  return TBE_OK;
}

}  // namespace
}  // namespace tbe

using namespace tbe;

extern "C" tbe_status tbe_grouped_linear_forward(int64_t rows, int32_t experts, int64_t inner, int64_t outer, const void* x,
                                                 int64_t x_stride, const void* weight, const void* bias, int32_t dtype,
                                                 const void* offsets, int32_t offset_type, void* y, int64_t y_stride,
                                                 int32_t out_dtype, tbe_stream_t stream) {
  clear_error();
  tbe_status st = check_sizes(rows, experts, inner, outer, dtype, out_dtype, offsets, offset_type);
  if (st == TBE_OK) st = check_matrix("x", x, dtype, rows, inner, x_stride);
  if (st == TBE_OK) st = check_matrix("weight", weight, dtype, 1, inner, inner);
  if (st == TBE_OK && bias) st = check_matrix("bias", bias, dtype, 1, outer, outer);
  if (st == TBE_OK) st = check_matrix("y", y, out_dtype, rows, outer, y_stride);
  if (st != TBE_OK || rows == 0) return st;
  GroupedArgs a = {};
  a.rows = rows; a.experts = experts; a.inner = static_cast<int>(inner); a.outer = static_cast<int>(outer);
  a.x = x; a.x_stride = x_stride; a.w = weight; a.bias = bias;
  a.offsets = offsets; a.offset64 = offset_type == TBE_I64;
  a.out = y; a.out_stride = y_stride; a.out_dt = out_dtype;
  return launch<kForward>(a, dtype, static_cast<hipStream_t>(stream));
}

extern "C" tbe_status tbe_grouped_linear_backward_input(int64_t rows, int32_t experts, int64_t inner, int64_t outer,
                                                        const void* grad_y, int64_t grad_y_stride, const void* weight,
                                                        int32_t dtype, const void* offsets, int32_t offset_type,
                                                        void* grad_x, int64_t grad_x_stride, int32_t out_dtype,
                                                        tbe_stream_t stream) {
  clear_error();
  tbe_status st = check_sizes(rows, experts, inner, outer, dtype, out_dtype, offsets, offset_type);
  if (st == TBE_OK) st = check_matrix("grad_y", grad_y, dtype, rows, outer, grad_y_stride);
  if (st == TBE_OK) st = check_matrix("weight", weight, dtype, 1, inner, inner);
  if (st == TBE_OK) st = check_matrix("grad_x", grad_x, out_dtype, rows, inner, grad_x_stride);
  if (st != TBE_OK || rows == 0) return st;
  GroupedArgs a = {};
  a.rows = rows; a.experts = experts; a.inner = static_cast<int>(inner); a.outer = static_cast<int>(outer);
  a.gy = grad_y; a.gy_stride = grad_y_stride; a.w = weight;
  a.offsets = offsets; a.offset64 = offset_type == TBE_I64;
  a.out = grad_x; a.out_stride = grad_x_stride; a.out_dt = out_dtype;
  return launch<kBackwardInput>(a, dtype, static_cast<hipStream_t>(stream));
}

extern "C" size_t tbe_grouped_linear_backward_weight_workspace_bytes(int64_t rows, int32_t experts, int64_t inner,
                                                                     int64_t outer) {
  if (rows < 0 || rows > kMaxRows || experts < 1 || experts > kMaxExperts || inner < 1 || inner > kMaxSide || outer < 1 ||
      outer > kMaxSide)
    return 0;
  // What any plan for up to so many rows may need, the one for these rows or not: a workspace sized for the
  // largest batch serves every smaller one.  Both terms grow with the rows.
  const int64_t each = slot_bytes(inner, outer);
  return static_cast<size_t>(hmin(weight_slots(rows, experts, kLeastSplit), most_partials(rows, inner, outer) / each) * each);
}

extern "C" tbe_status tbe_grouped_linear_backward_weight(int64_t rows, int32_t experts, int64_t inner, int64_t outer,
                                                         const void* x, int64_t x_stride, const void* grad_y,
                                                         int64_t grad_y_stride, int32_t dtype, const void* offsets,
                                                         int32_t offset_type, void* grad_weight, void* grad_bias,
                                                         int32_t out_dtype, void* workspace, size_t workspace_bytes,
                                                         tbe_stream_t stream) {
  clear_error();
  tbe_status st = check_sizes(rows, experts, inner, outer, dtype, out_dtype, offsets, offset_type);
  if (st == TBE_OK) st = check_matrix("x", x, dtype, rows, inner, x_stride);
  if (st == TBE_OK) st = check_matrix("grad_y", grad_y, dtype, rows, outer, grad_y_stride);
  if (st == TBE_OK) st = check_matrix("grad_weight", grad_weight, out_dtype, 1, inner, inner);
  if (st == TBE_OK && grad_bias) st = check_matrix("grad_bias", grad_bias, out_dtype, 1, outer, outer);
  if (st != TBE_OK) return st;
  const size_t need = tbe_grouped_linear_backward_weight_workspace_bytes(rows, experts, inner, outer);
  if (need && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < need)) {
    set_error("grouped linear backward by weight: workspace of %zu bytes, 256-byte aligned; %zu given", need,
              workspace ? workspace_bytes : 0);
    return TBE_ERR_WORKSPACE;
  }
  GroupedArgs a = {};
  a.rows = rows; a.experts = experts; a.inner = static_cast<int>(inner); a.outer = static_cast<int>(outer);
  a.x = x; a.x_stride = x_stride; a.gy = grad_y; a.gy_stride = grad_y_stride;
  a.offsets = offsets; a.offset64 = offset_type == TBE_I64;
  a.out = grad_weight; a.out_dt = out_dtype; a.grad_bias = grad_bias; a.workspace = workspace;
  const WeightPlan plan = weight_plan(rows, experts, inner, outer);
  a.split = plan.split;
  a.units = plan.split ? static_cast<int>(row_tiles_bound(rows, experts, plan.split)) : 0;
  a.slots = plan.split ? static_cast<int>(weight_slots(rows, experts, plan.split)) : 0;
  a.tile = plan.tile;
  return launch<kBackwardWeight>(a, dtype, static_cast<hipStream_t>(stream));
}
