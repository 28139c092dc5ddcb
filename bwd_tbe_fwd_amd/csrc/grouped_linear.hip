// Linear layers of E experts on rows grouped by expert: argument validation, dispatch and the
// kernel.
#include "grouped_linear.h"
#include "grouped_tile.h"

#include "../../include/tbe_tower.h"

namespace tbe {
namespace {

// The kernel for any size, stride and alignment: a workgroup of 4 waves takes 64 x 64 of C, 32 of k
// at a time through LDS, each wave 32 x 32 as 2 x 2 products of 16 x 16 x 32.
constexpr int kTile = 64, kTileK = 32, kPad = 8;

// 64 x 32 of an operand into LDS as [m][k]; what lies past `ms` or `ks` is zero.
template <bool ALONG>
__device__ __forceinline__ void stage_any(const uint16_t* p, int64_t ld, int64_t ms, int64_t ks, uint16_t (*s)[kTileK + kPad]) {
#pragma unroll
  for (int i = 0; i < kTile * kTileK / kBlock; ++i) {
    const int at = i * kBlock + threadIdx.x;
    const int m = ALONG ? at / kTileK : at % kTile, k = ALONG ? at % kTileK : at / kTile;
    s[m][k] = m < ms && k < ks ? p[ALONG ? m * ld + k : k * ld + m] : uint16_t(0);
  }
}

template <int DT, int OP>
__global__ __launch_bounds__(kBlock) void grouped_any_kernel(GroupedArgs a) {
  __shared__ uint16_t sa[kTile][kTileK + kPad], sb[kTile][kTileK + kPad];
  const uint16_t *pa, *pb;
  int64_t lda, ldb, ms, ns, ks;
  int expert;
  int64_t row = 0;
  const int64_t n0 = static_cast<int64_t>(blockIdx.y) * kTile;
  const int64_t io = static_cast<int64_t>(a.inner) * a.outer;
  int64_t m0 = 0;
  if constexpr (OP == kBackwardWeight) {
    expert = blockIdx.z;
    const RowRange r = rows_of(a, expert);
    m0 = static_cast<int64_t>(blockIdx.x) * kTile;
    ms = a.outer - m0;
    ns = a.inner - n0;
    ks = r.hi - r.lo;
    lda = a.gy_stride;
    ldb = a.x_stride;
    pa = static_cast<const uint16_t*>(a.gy) + r.lo * lda + m0;
    pb = static_cast<const uint16_t*>(a.x) + r.lo * ldb + n0;
  } else {
    RowTiles tiles;
    RowTile t;
    if (!tiles.find(a, kTile, blockIdx.x, false, t)) return;
    expert = t.expert;
    row = t.row;
    ms = t.hi - t.row;
    const bool fwd = OP == kForward;
    lda = fwd ? a.x_stride : a.gy_stride;
    pa = static_cast<const uint16_t*>(fwd ? a.x : a.gy) + row * lda;
    ks = expert < a.experts ? (fwd ? a.inner : a.outer) : 0;
    ns = (fwd ? a.outer : a.inner) - n0;
    ldb = a.inner;
    pb = static_cast<const uint16_t*>(a.w) + expert * io + (fwd ? n0 * ldb : n0);
  }
  const int w = threadIdx.x >> 6, l = lane_id(), wm = (w >> 1) * 32, wn = (w & 1) * 32;
  f32x4 acc[2][2] = {};
  f32x4 ones_acc[2] = {};
  u16x8_t ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = DT == 2 ? 0x3f80 : 0x3c00;
  for (int64_t k0 = 0; k0 < ks; k0 += kTileK) {
    constexpr bool A_ALONG = OP != kBackwardWeight, B_ALONG = OP == kForward;
    __syncthreads();
    stage_any<A_ALONG>(pa + k0 * (A_ALONG ? 1 : lda), lda, ms, ks - k0, sa);
    stage_any<B_ALONG>(pb + k0 * (B_ALONG ? 1 : ldb), ldb, ns, ks - k0, sb);
    __syncthreads();
    u16x8_t fa[2], fb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fa[i] = *reinterpret_cast<const u16x8_t*>(&sa[wm + 16 * i + (l & 15)][8 * (l >> 4)]);
      fb[i] = *reinterpret_cast<const u16x8_t*>(&sb[wn + 16 * i + (l & 15)][8 * (l >> 4)]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma16<DT>(fa[i], fb[j], acc[i][j]);
      if (OP == kBackwardWeight) ones_acc[i] = mfma16<DT>(fa[i], ones, ones_acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int m = wm + 16 * i + 4 * (l >> 4) + r, n = wn + 16 * j + (l & 15);
        if (m >= ms || n >= ns) continue;
        float v = acc[i][j][r];
        if constexpr (OP == kBackwardWeight) {
          store_any(a.out, a.out_dt, expert * io + (m0 + m) * a.inner + n0 + n, v);
        } else {
          if (OP == kForward && a.bias && expert < a.experts)
            v += Fmt<DT>::to_f(static_cast<const uint16_t*>(a.bias)[static_cast<int64_t>(expert) * a.outer + n0 + n]);
          store_any(a.out, a.out_dt, (row + m) * a.out_stride + n0 + n, v);
        }
      }
  if constexpr (OP == kBackwardWeight) {
    if (a.grad_bias && blockIdx.y == 0 && wn == 0 && (l & 15) == 0)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int m = wm + 16 * i + 4 * (l >> 4) + r;
          if (m < ms) store_any(a.grad_bias, a.out_dt, static_cast<int64_t>(expert) * a.outer + m0 + m, ones_acc[i][r]);
        }
  }
}

template <int DT, int OP>
tbe_status launch_any(const GroupedArgs& a, hipStream_t s) {
  const int n = OP == kForward ? a.outer : a.inner;
  const unsigned ny = static_cast<unsigned>((n + kTile - 1) / kTile);
  const dim3 grid = OP == kBackwardWeight ? dim3((a.outer + kTile - 1) / kTile, ny, a.experts)
                                          : dim3(static_cast<unsigned>(row_tiles_bound(a, kTile)), ny, 1);
  const char* what = OP == kForward ? "grouped_forward" : OP == kBackwardInput ? "grouped_input" : "grouped_weight";
  ProfScope ps(what, s);
  hipLaunchKernelGGL((grouped_any_kernel<DT, OP>), grid, dim3(kBlock), 0, s, a);
  return check_launch(what);
}

constexpr int64_t kMaxGroups = int64_t{1} << 22;  // a launch has fewer than 2^32 threads
const char* name_of(int op) { return op == kForward ? "grouped_forward" : op == kBackwardInput ? "grouped_input" : "grouped_weight"; }

template <int DT, int OP, int BM, int BN, int WM, int WN, bool DIRECT>
tbe_status launch_tile(const GroupedArgs& a, hipStream_t s) {
  auto kernel = grouped_tile_kernel<DT, OP, BM, BN, WM, WN, DIRECT>;
  constexpr int kThreads = WM * WN * kWave;
  const int n = OP == kForward ? a.outer : a.inner;
  const int n_tiles = (n + BN - 1) / BN;
  const int64_t units = OP != kBackwardWeight ? row_tiles_bound(a, BM) : a.split ? row_tiles_bound(a, a.split) : a.experts;
  // rows: a multiple of 8, for the chiplets' shares
  const int64_t groups = OP == kBackwardWeight ? units * ((a.outer + BM - 1) / BM) * n_tiles : (units * n_tiles + 7) / 8 * 8;
  if (groups > kMaxGroups) {
    set_error("grouped linear: %lld tiles are more than a launch takes", static_cast<long long>(groups));
    return TBE_ERR_UNSUPPORTED;
  }
  ProfScope ps(name_of(OP), s);
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(groups)), dim3(kThreads), 0, s, a, n_tiles);
  return check_launch(name_of(OP));
}

// Sum of the units' partial weight gradients of the experts that have more than one, in the order of
// their rows; zeros for the experts without rows, which have no unit.
__global__ __launch_bounds__(kBlock) void grouped_reduce_kernel(GroupedArgs a) {
  const int e = blockIdx.y;
  const int64_t io = static_cast<int64_t>(a.inner) * a.outer, each = io + a.outer;
  auto units_of = [&](int k) {
    const RowRange r = rows_of(a, k);
    return (r.hi - r.lo + a.split - 1) / a.split;
  };
  const int64_t n = units_of(e);
  if (n == 1) return;
  int64_t first = 0;  // units of the experts before
  for (int k = lane_id(); k < e; k += kWave) first += units_of(k);
  for (int d = 1; d < kWave; d <<= 1) first += __shfl_xor(first, d);
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

// Rows of a unit of the weight gradient.  With few tiles for the 256 CUs, or experts of unequal rows,
// an expert's rows are shared among workgroups whose partial sums a second kernel adds: units of at
// least 512 rows (the partial sums of shorter ones cost more than the products), as many as give
// two workgroups a CU.  0: the tiles of the experts are enough.
int split_rows(int64_t rows, int64_t experts, int64_t inner, int64_t outer) {
  const int64_t tiles = ((outer + 255) / 256) * ((inner + 255) / 256);
  if (experts * tiles >= 512 || rows <= 512) return 0;
  const int64_t c = (rows * tiles / 512 + 63) / 64 * 64;
  return static_cast<int>(hmax(512, c));
}

// Whether every 16-byte chunk of the operands is whole and starts on 16 bytes, and a tile's offsets
// stay below 2^31.
bool chunked(const GroupedArgs& a, int op) {
  auto whole = [](const void* p, int64_t ld, int64_t contiguous) {
    return !(reinterpret_cast<uintptr_t>(p) & 15) && ld % 8 == 0 && contiguous % 8 == 0 && ld < (int64_t{1} << 21);
  };
  const int64_t xs = a.rows > 1 ? a.x_stride : a.inner, gs = a.rows > 1 ? a.gy_stride : a.outer;
  if (op == kForward) return whole(a.x, xs, a.inner) && whole(a.w, a.inner, a.inner);
  if (op == kBackwardInput) return whole(a.gy, gs, a.outer) && whole(a.w, a.inner, a.inner);
  return whole(a.gy, gs, a.outer) && whole(a.x, xs, a.inner);
}

template <int DT, int OP>
tbe_status launch_type(const GroupedArgs& a, hipStream_t s) {
  return chunked(a, OP) ? launch_tile<DT, OP, 256, 256, 2, 4, true>(a, s) : launch_tile<DT, OP, 256, 128, 2, 4, false>(a, s);
}

template <int OP>
tbe_status launch(const GroupedArgs& a, int dtype, hipStream_t s) {
  const tbe_status st = dtype == TBE_F16 ? launch_type<1, OP>(a, s) : launch_type<2, OP>(a, s);
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
  const int64_t split = split_rows(rows, experts, inner, outer);
  return split ? static_cast<size_t>((rows / split + experts + 1) * (inner + 1) * outer) * 4 : 0;
}

extern "C" tbe_status tbe_grouped_linear_backward_weight(int64_t rows, int32_t experts, int64_t inner, int64_t outer,
                                                         const void* x, int64_t x_stride, const void* grad_y,
                                                         int64_t grad_y_stride, int32_t dtype, const void* offsets,
                                                         int32_t offset_type, void* grad_weight, void* grad_bias,
                                                         int32_t out_dtype, void* workspace, size_t workspace_bytes,
                                                         tbe_stream_t stream) {
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
  a.split = split_rows(rows, experts, inner, outer);
  return launch<kBackwardWeight>(a, dtype, static_cast<hipStream_t>(stream));
}
