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
  int32_t units;        // units at most
  int32_t slots;        // partial sums that the workspace holds
  int32_t tile;         // backward by weight: which of the three, host only
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
  int singles;       // experts before it that have one tile
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
    t.singles = 0;
    for (int base = 0; base <= a.experts; base += kWave) {
      const int here = counted ? read_lane(upto, kWave - 1) : count(a, BM, base);
      const unsigned long long singles = __ballot(n == 1);
      if (tile < here) {
        const int src = __ffsll(static_cast<unsigned long long>(__ballot(upto > tile))) - 1;
        t.expert = base + src;
        t.singles += __popcll(singles & ((1ull << src) - 1));
        t.row = read_lane64(r.lo + static_cast<int64_t>(tile - (upto - n)) * BM, src);
        t.hi = read_lane64(r.hi, src);
        return true;
      }
      tile -= here;
      t.singles += __popcll(singles);
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

// Row tiles at most: a partly filled one for every expert that has rows and for the rows of no expert.
inline int64_t row_tiles_bound(int64_t rows, int64_t experts, int64_t bm) { return rows / bm + hmin(experts, rows) + 1; }
// A launch has fewer than 2^32 threads.
inline bool launch_takes(int64_t groups, int threads) { return groups * threads < (int64_t{1} << 32); }

// ---------------------------------------------------------------------------
// the tile, on the host
// ---------------------------------------------------------------------------
inline double rounds_of(double tiles, double slots) {
  const double r = tiles / slots;
  const int64_t whole = static_cast<int64_t>(r);
  return r > static_cast<double>(whole) ? static_cast<double>(whole + 1) : static_cast<double>(hmax(1, whole));
}
// Three tiles of C for a product: the larger one moves fewer operand bytes for each product, the smaller
// one leaves fewer CUs idle.  As many run at once as `slots` on 256 CUs; a round of them takes a fixed
// time and one for each 64 of k, `alone` where few of the slots are taken and `full` where all are (us,
// fitted to times with the tile as given).
struct TileCost {
  int bm, bn, threads;
  double slots, fixed, alone, full;
};
// Operands straight to LDS, forward, the three tiles in turn: 65536 rows, 16 experts, 1024 x 1024: 137 / 143 /
// 213 us; 8192 rows, 8 experts, 2048 x 2048: 91 / 84 / 119; 4096 rows, 4 experts, 1024 x 1024: 26 / 21 /
// 26; 400 rows, 8 experts, 1024 x 512: 24 / 12 / 10.
constexpr TileCost kDirectTiles[3] = {{256, 256, 512, 256, 6.0, 1.37, 1.37}, {128, 128, 256, 512, 4.0, 0.78, 0.78}, {64, 64, 256, 1024, 3.0, 0.61, 0.61}};
// Operands through registers: 60000 rows, 8 experts, 1777 x 1201, forward: 334 / 419 / 746 us; 3000 rows, 4
// experts, 2047 x 901, by input: 37 / 30 / 40; 1000 rows, 1 expert, 2047 x 901, by input: 34 / 23 / 18.
constexpr TileCost kRegisterTiles[3] = {{256, 256, 512, 256, 6.0, 1.3, 2.05}, {256, 128, 512, 256, 6.0, 1.0, 1.3}, {64, 64, 256, 1024, 3.0, 0.55, 1.35}};
// The weight gradient, both ways; times of the direct loads are at its plan (grouped_linear.hip).  Through
// registers: 60000 rows, 8 experts, 1777 x 1201: 365 / 465 / 862 us; 3000 rows, 4 experts, 2047 x 901: 39 /
// 29 / 44; 5003 rows, 13 experts, 1000 x 515: 33 / 33 / 30.
constexpr TileCost kWeightTiles[3] = {{256, 256, 512, 256, 6.0, 1.5, 1.85}, {128, 128, 256, 512, 4.0, 0.75, 1.36}, {64, 64, 256, 1024, 3.0, 0.6, 0.95}};
// Tiles of k each, those of the last round of `last`.
inline double tiles_us(const TileCost& c, double tiles, double k, double last) {
  const double r = rounds_of(tiles, c.slots);
  return r * c.fixed + ((r - 1.0) * k + last) / 64 * (c.alone + (c.full - c.alone) * tiles / (r * c.slots));
}
// Row tiles of `bm` rows that are expected of rows spread over experts.
inline double row_tiles_expected(int64_t rows, int64_t experts, int bm) {
  if (experts == 1) return static_cast<double>((rows + bm - 1) / bm);
  return static_cast<double>(rows) / bm + 0.5 * static_cast<double>(hmin(experts, rows));
}

enum { kForward = 0, kBackwardInput = 1, kBackwardWeight = 2 };

// Defined in grouped_launch.h, in a translation unit for each product and type.
template <int DT, int OP>
tbe_status grouped_launch(const GroupedArgs& a, hipStream_t s);

}  // namespace tbe
