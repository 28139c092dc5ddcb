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
  const int64_t units = OP != kBackwardWeight ? row_tiles_bound(a, BM) : a.split ? a.units : a.experts;
  // rows: a multiple of 8, for the chiplets' shares
  const int64_t groups = OP == kBackwardWeight ? units * ((a.outer + BM - 1) / BM) * n_tiles : (units * n_tiles + 7) / 8 * 8;
  if (groups * kThreads >= (int64_t{1} << 32)) {
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

template <int DT, int OP>
tbe_status grouped_launch(const GroupedArgs& a, hipStream_t s) {
  const int64_t n = OP == kForward ? a.outer : a.inner, k = OP == kForward ? a.inner : a.outer;
  if (chunked(a, OP)) {
    int tile = a.tile;
    if (OP != kBackwardWeight) {
      double best = 0.0;
      for (int t = 0; t < 3; ++t) {
        const int side = kTileSide[t];
        const double tiles = row_tiles_expected(a.rows, a.experts, side) * static_cast<double>((n + side - 1) / side);
        const double us = rounds_of(tiles, kTileSlots[t]) * round_us(t, static_cast<double>(k));
        if (t == 0 || us < best) {
          best = us;
          tile = t;
        }
      }
    }
    return tile == 0 ? launch_tile<DT, OP, 256, 256, 2, 4, true>(a, s)
                     : tile == 1 ? launch_tile<DT, OP, 128, 128, 2, 2, true>(a, s) : launch_tile<DT, OP, 64, 64, 2, 2, true>(a, s);
  }
  // Through registers: 256 x 128 (the registers of 256 x 256 do not suffice) or 64 x 64; 128 x 128 was
  // never the fastest.  20000 rows, 8 experts, 1001 x 515: 68 / 80 / 78 us; 2000 rows: 36 / 45 / 26 us.
  bool large;
  if (OP == kBackwardWeight) {
    large = a.tile == 0;
  } else {
    const double steps = static_cast<double>((k + 63) / 64);
    const double l = rounds_of(row_tiles_expected(a.rows, a.experts, 256) * static_cast<double>((n + 127) / 128), 256) * (6.0 + steps * 1.75);
    const double t = rounds_of(row_tiles_expected(a.rows, a.experts, 64) * static_cast<double>((n + 63) / 64), 1024) * (3.0 + steps * 1.44);
    large = l <= t;
  }
  return large ? launch_tile<DT, OP, 256, 128, 4, 2, false>(a, s) : launch_tile<DT, OP, 64, 64, 2, 2, false>(a, s);
}

#define TBE_GROUPED(DT, OP)                                                                  \
  namespace tbe {                                                                            \
  template tbe_status grouped_launch<DT, OP>(const GroupedArgs& a, hipStream_t s);           \
  }

}  // namespace tbe
