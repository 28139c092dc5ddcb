// Launch of one grouped product: which tile, and the grid.  One translation unit for each product and
// type (grouped_forward_f16.hip and its siblings).
#pragma once

#include "grouped_tile.h"

namespace tbe {


template <int DT, int OP, int BM, int BN, int WM, int WN, bool DIRECT>
tbe_status launch_tile(const GroupedArgs& a, hipStream_t s) {
  auto kernel = grouped_tile_kernel<DT, OP, BM, BN, WM, WN, DIRECT>;
  constexpr int kThreads = WM * WN * kWave;
  const char* what = OP == kForward ? "grouped_forward" : OP == kBackwardInput ? "grouped_input" : "grouped_weight";
  const int n = OP == kForward ? a.outer : a.inner;
  const int n_tiles = (n + BN - 1) / BN;
  const int64_t units = OP != kBackwardWeight ? row_tiles_bound(a.rows, a.experts, BM) : a.split ? a.units : a.experts;
  // rows: a multiple of 8, for the chiplets' shares
  const int64_t groups = OP == kBackwardWeight ? units * ((a.outer + BM - 1) / BM) * n_tiles : (units * n_tiles + 7) / 8 * 8;
  if (!launch_takes(groups, kThreads)) {
    set_error("grouped linear: %lld tiles are more than a launch takes", static_cast<long long>(groups));
    return TBE_ERR_UNSUPPORTED;
  }
  ProfScope ps(what, s);
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(groups)), dim3(kThreads), 0, s, a, n_tiles);
  return check_launch(what);
}

// Whether every 16-byte chunk of the operands is whole and starts on 16 bytes, and a tile's offsets
// stay below 2^31.
inline bool chunked(const GroupedArgs& a, int op) {
  auto whole = [](const void* p, int64_t ld, int64_t contiguous) {
    return !(reinterpret_cast<uintptr_t>(p) & 15) && ld % 8 == 0 && contiguous % 8 == 0 && ld < (int64_t{1} << 21);
  };
  const int64_t xs = a.rows > 1 ? a.x_stride : a.inner, gs = a.rows > 1 ? a.gy_stride : a.outer;
  if (op == kForward) return whole(a.x, xs, a.inner) && whole(a.w, a.inner, a.inner);
  if (op == kBackwardInput) return whole(a.gy, gs, a.outer) && whole(a.w, a.inner, a.inner);
  return whole(a.gy, gs, a.outer) && whole(a.x, xs, a.inner);
}

// The tile of least expected time among those that a launch takes.  (The weight gradient's comes with its plan.)
inline int row_tile(const GroupedArgs& a, const TileCost (&tiles)[3], int64_t n, int64_t k) {
  int tile = 0;
  double best = 0.0;
  for (int t = 0; t < 3; ++t) {
    const TileCost& c = tiles[t];
    const int64_t n_tiles = (n + c.bn - 1) / c.bn;
    if (t > 0 && !launch_takes(row_tiles_bound(a.rows, a.experts, c.bm) * n_tiles + 7, c.threads)) continue;
    const double us = tiles_us(c, row_tiles_expected(a.rows, a.experts, c.bm) * static_cast<double>(n_tiles),
                               static_cast<double>((k + 63) / 64 * 64), static_cast<double>((k + 63) / 64 * 64));
    if (t == 0 || us < best) {
      best = us;
      tile = t;
    }
  }
  return tile;
}

template <int DT, int OP>
tbe_status grouped_launch(const GroupedArgs& a, hipStream_t s) {
  const int64_t n = OP == kForward ? a.outer : a.inner, k = OP == kForward ? a.inner : a.outer;
  if (chunked(a, OP)) {
    const int tile = OP == kBackwardWeight ? a.tile : row_tile(a, kDirectTiles, n, k);
    return tile == 0 ? launch_tile<DT, OP, 256, 256, 2, 4, true>(a, s)
                     : tile == 1 ? launch_tile<DT, OP, 128, 128, 2, 2, true>(a, s) : launch_tile<DT, OP, 64, 64, 2, 2, true>(a, s);
  }
  const int tile = OP == kBackwardWeight ? a.tile : row_tile(a, kRegisterTiles, n, k);
  if (tile == 0) return launch_tile<DT, OP, 256, 256, 2, 4, false>(a, s);
  if (tile == 2) return launch_tile<DT, OP, 64, 64, 2, 2, false>(a, s);
  if constexpr (OP == kBackwardWeight) return launch_tile<DT, OP, 128, 128, 2, 2, false>(a, s);
  else return launch_tile<DT, OP, 256, 128, 4, 2, false>(a, s);
}

#define TBE_GROUPED(DT, OP)                                                                  \
  namespace tbe {                                                                            \
  template tbe_status grouped_launch<DT, OP>(const GroupedArgs& a, hipStream_t s);           \
  }

}  // namespace tbe
