// Linear layers of E experts on rows grouped by expert: the three products and their kernels'
// common parts.  Declarations and the meaning of every argument are in include/tbe_tower.h.
//
// Each product is C(m, n) = sum_k A(m, k) B(n, k) for every expert e:
//   forward          m = row, n = output, k = input:   A = x,      B = W_e
//   backward, input  m = row, n = input,  k = output:  A = grad_y, B = W_e read across
//   backward, weight m = output, n = input, k = row:   A = grad_y and B = x, both read across
// An operand is "along" where its k are adjacent in memory and "across" where its m or n are.
#pragma once

#include "tbe_internal.h"
#include "tower_device.h"

namespace tbe {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef uint16_t u16x8_t __attribute__((ext_vector_type(8)));

// D = A B + C, 16 x 16 x 32: lane l holds A(l % 16, 8 (l / 16) + i), B(l % 16, 8 (l / 16) + i) for
// i < 8, and C(4 (l / 16) + i, l % 16) for i < 4.
template <int DT>
__device__ __forceinline__ f32x4 mfma16(u16x8_t a, u16x8_t b, f32x4 c) {
  if constexpr (DT == 2)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

struct GroupedArgs {
  int64_t rows;
  int32_t experts;
  int32_t inner, outer;
  const void* x;        // forward, backward by weight
  int64_t x_stride;
  const void* gy;       // backward
  int64_t gy_stride;
  const void* w;
  const void* bias;     // forward; NULL: none
  const void* offsets;
  int32_t offset64;
  void* out;            // y, grad_x, grad_weight
  int64_t out_stride;   // rows of y or grad_x
  int32_t out_dt;
  void* grad_bias;      // backward by weight; NULL: none
  void* workspace;
};

// Rows [lo, hi) of expert e < experts, inside [0, rows]; e = experts: the rows of no expert.
struct RowRange {
  int64_t lo, hi;
};
__device__ __forceinline__ int64_t offset_at(const GroupedArgs& a, int e) {
  const int64_t o = a.offset64 ? static_cast<const int64_t*>(a.offsets)[e] : static_cast<const int32_t*>(a.offsets)[e];
  return min(max(o, static_cast<int64_t>(0)), a.rows);
}
__device__ __forceinline__ RowRange rows_of(const GroupedArgs& a, int e) {
  RowRange r;
  r.lo = offset_at(a, e);
  r.hi = e < a.experts ? max(offset_at(a, e + 1), r.lo) : a.rows;
  return r;
}

// Row tile `tile` of tiles of BM rows counted over the experts in order and then the rows of no
// expert: its expert and first row; false past the last tile.  Every wave finds it by itself: 64
// experts a step, their tile counts summed over the lanes.
struct RowTile {
  int expert;
  int64_t row, hi;
};
__device__ __forceinline__ bool find_row_tile(const GroupedArgs& a, int BM, int64_t tile, RowTile& t) {
  const int l = lane_id();
  int64_t before = 0;
  for (int base = 0; base <= a.experts; base += kWave) {
    const int e = base + l;
    RowRange r = {0, 0};
    if (e <= a.experts) r = rows_of(a, e);
    const int32_t n = static_cast<int32_t>((r.hi - r.lo + BM - 1) / BM);
    int32_t upto = n;  // tiles of lanes 0 .. l
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int32_t up = __shfl_up(upto, d);
      if (l >= d) upto += up;
    }
    const int32_t total = read_lane(upto, kWave - 1);
    if (tile < before + total) {
      // the first lane whose tiles reach past this one
      const int src = __ffsll(static_cast<unsigned long long>(__ballot(before + upto > tile))) - 1;
      const int64_t first = read_lane64(r.lo + (tile - before - (upto - n)) * BM, src);
      t.expert = base + src;
      t.row = first;
      t.hi = read_lane64(r.hi, src);
      return true;
    }
    before += total;
  }
  return false;
}

// Row tiles at most: a partly filled one for every expert and the rows of no expert.
inline int64_t row_tiles_bound(const GroupedArgs& a, int BM) { return a.rows / BM + a.experts + 1; }

enum { kForward = 0, kBackwardInput = 1, kBackwardWeight = 2 };

}  // namespace tbe
