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
  int32_t split;        // backward by weight: rows of a unit, 0: an expert's rows are one
  int32_t units;        // units at most: partial sums that the workspace holds
  int32_t tile;         // backward by weight: which of kTileSide, host only
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

// Tiles of BM rows are counted over the experts in order and then the rows of no expert.  Every wave
// counts them by itself, 64 experts a step, a lane each.  Offsets that are not in order may count some
// rows twice, but a tile's rows lie inside [0, rows] whatever they are.
struct RowTile {
  int expert;
  int64_t row, hi;   // first row, and where its expert's end
};
struct RowTiles {
  RowRange r;        // of this lane's expert, and its tiles: how many, and with those of the lanes before
  int32_t n, upto;
  __device__ __forceinline__ int32_t count(const GroupedArgs& a, int BM, int base) {
    const int l = lane_id(), e = base + l;
    r = RowRange{0, 0};
    if (e <= a.experts) r = rows_of(a, e);
    n = static_cast<int32_t>((r.hi - r.lo + BM - 1) / BM);
    upto = n;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int32_t up = __shfl_up(upto, d);
      if (l >= d) upto += up;
    }
    return read_lane(upto, kWave - 1);
  }
  // Tile `tile` (>= 0); false past the last one.  counted: count(a, BM, 0) was called, and all experts are
  // in it.
  __device__ __forceinline__ bool find(const GroupedArgs& a, int BM, int tile, bool counted, RowTile& t) {
    for (int base = 0; base <= a.experts; base += kWave) {
      const int here = counted ? read_lane(upto, kWave - 1) : count(a, BM, base);
      if (tile < here) {
        const int src = __ffsll(static_cast<unsigned long long>(__ballot(upto > tile))) - 1;
        t.expert = base + src;
        t.row = read_lane64(r.lo + static_cast<int64_t>(tile - (upto - n)) * BM, src);
        t.hi = read_lane64(r.hi, src);
        return true;
      }
      tile -= here;
    }
    return false;
  }
};

// The expert with the k-th most rows (the lower one first among equals); with more than 64 experts,
// expert k.
__device__ __forceinline__ int expert_by_rows(const GroupedArgs& a, int k) {
  if (a.experts > kWave) return k;
  const int l = lane_id();
  int64_t n = -1;
  if (l < a.experts) {
    const RowRange r = rows_of(a, l);
    n = r.hi - r.lo;
  }
  int rank = 0;
  for (int e = 0; e < a.experts; ++e) {
    const int64_t m = read_lane64(n, e);
    rank += m > n || (m == n && e < l) ? 1 : 0;
  }
  return __ffsll(static_cast<unsigned long long>(__ballot(l < a.experts && rank == k))) - 1;
}

// Row tiles at most: a partly filled one for every expert and the rows of no expert.
inline int64_t row_tiles_bound(const GroupedArgs& a, int BM) { return a.rows / BM + a.experts + 1; }

// ---------------------------------------------------------------------------
// the tile, on the host
// ---------------------------------------------------------------------------
// Three tiles of C: 256 x 256 by 8 waves, 128 x 128 and 64 x 64 by 4; as many run at once as
// kTileSlots on 256 CUs.  Time of a round of them in us: a fixed part and one for each 64 of k, fitted
// to 65536 rows, 16 experts, 1024 x 1024 (139 / 148 / 218 us) and to 1024 and 4096 rows (27 / 18 /
// 14 and 27 / 21 / 27 us).  The larger tile moves fewer operand bytes for each product, the smaller one
// leaves fewer CUs idle: 8192 rows, 8 experts, 2048 x 2048 take 93 / 88 / 122 us, 400 rows, 8 experts,
// 1024 x 512 take 24 / 13 / 10 us.
constexpr int kTileSide[3] = {256, 128, 64};
constexpr double kTileSlots[3] = {256, 512, 1024}, kTileFixed[3] = {6.0, 4.0, 3.0}, kTileStep[3] = {1.37, 0.78, 0.61};
inline double round_us(int tile, double k) { return kTileFixed[tile] + (k + 63) / 64 * kTileStep[tile]; }
// Row tiles of `bm` rows that are expected of rows spread over experts.
inline double row_tiles_expected(int64_t rows, int64_t experts, int bm) {
  if (experts == 1) return static_cast<double>((rows + bm - 1) / bm);
  return static_cast<double>(rows) / bm + 0.5 * static_cast<double>(hmin(experts, rows));
}
inline double rounds_of(double tiles, double slots) {
  const double r = tiles / slots;
  const int64_t whole = static_cast<int64_t>(r);
  return r > static_cast<double>(whole) ? static_cast<double>(whole + 1) : static_cast<double>(hmax(1, whole));
}

enum { kForward = 0, kBackwardInput = 1, kBackwardWeight = 2 };

// Defined in grouped_launch.h, in a translation unit for each product and type.
template <int DT, int OP>
tbe_status grouped_launch(const GroupedArgs& a, hipStream_t s);

}  // namespace tbe
