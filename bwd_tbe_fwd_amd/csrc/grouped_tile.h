// The tiled kernel of the grouped products: a workgroup's expert, rows and place, the products (tile_products.h) and the
// results.  grouped_linear.h says what m, n, k, "along" and "across" are.
#pragma once

#include "grouped_linear.h"
#include "tile_products.h"

namespace tbe {

template <int DT, int OP, int BM, int BN, int WM, int WN, bool DIRECT>
__global__ __launch_bounds__(WM * WN * kWave, BM * BN <= 64 * 64 ? 4 : 2) void grouped_tile_kernel(GroupedArgs a, int n_tiles) {
  constexpr int T = WM * WN * kWave;
  constexpr int MF = BM / WM / 16, NF = BN / WN / 16;  // products of 16 x 16 a wave
  constexpr bool A_ALONG = OP != kBackwardWeight, B_ALONG = OP == kForward;
  constexpr int K = kStepK, GA = 4, GB = 4 * NF;
  using OA = Operand<A_ALONG, BM, GA, T, DIRECT>;
  using OB = Operand<B_ALONG, BN, GB, T, DIRECT>;
  constexpr int kBytes = 2 * 2 * (OA::kElems + OB::kElems);
  __shared__ __align__(16) char lds[kBytes];
  OA A;
  OB B;
  const int64_t io = static_cast<int64_t>(a.inner) * a.outer;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane_id();
  const int wm = (w / WN) * (MF * 16), wn = (w % WN) * (NF * 16);

  // the tile: its expert, rows, place in C and what of it lies inside, steps of k
  int expert, row, m0 = 0, n0, m_left, n_left, steps;
  float* part = nullptr;  // backward by weight: the unit's partial sums
  if constexpr (OP == kBackwardWeight) {
    // one tile of one expert's rows, or with a.split of one unit of at most a.split of them; the
    // experts with the most rows come first, so that the workgroups still to come are the short ones
    const int m_tiles = (a.outer + BM - 1) / BM, each = n_tiles * m_tiles;
    const int unit = blockIdx.x / each;
    // experts differ in their rows: each one's tiles are shared among the chiplets
    const int k = chiplet_order(blockIdx.x % each, each);
    m0 = (k % m_tiles) * BM;
    n0 = (k / m_tiles) * BN;
    m_left = a.outer - m0;
    n_left = a.inner - n0;
    int rows;
    if (a.split) {
      RowTiles tiles;
      RowTile t;
      if (!tiles.find(a, a.split, unit, false, t) || t.expert >= a.experts) return;
      expert = t.expert;
      row = static_cast<int>(t.row);
      rows = static_cast<int>(min(t.hi - t.row, static_cast<int64_t>(a.split)));
      const RowRange all = rows_of(a, expert);
      if (all.hi - all.lo > a.split) {
        const int slot = unit - t.singles;  // units of experts that have several, in order
        if (slot >= a.slots) return;        // offsets that are not in order: inside the workspace
        part = static_cast<float*>(a.workspace) + slot * (io + a.outer);
      }
    } else {
      expert = expert_by_rows(a, unit);
      const RowRange r = rows_of(a, expert);
      row = static_cast<int>(r.lo);
      rows = static_cast<int>(r.hi - r.lo);
    }
    steps = (rows + K - 1) / K;
    A.init(static_cast<const uint16_t*>(a.gy) + row * a.gy_stride + m0, a.gy_stride, m_left, rows, a.outer);
    B.init(static_cast<const uint16_t*>(a.x) + row * a.x_stride + n0, a.x_stride, n_left, rows, a.inner);
  } else {
    // a chiplet's tiles are neighbours: a contiguous share of all, of which there are fewer than
    // workgroups where experts' last tiles are not all there; with 64 experts and more, whose counting
    // takes several steps, the tiles are taken as they come
    constexpr bool fwd = OP == kForward;
    RowTiles tiles;
    RowTile t;
    const bool counted = a.experts < kWave;
    int id = blockIdx.x;
    if (counted) {
      const int64_t total = min(static_cast<int64_t>(tiles.count(a, BM, 0)) * n_tiles, static_cast<int64_t>(gridDim.x));
      const unsigned x = blockIdx.x % 8;
      id = static_cast<int>(total * x / 8 + blockIdx.x / 8);
      if (id >= total * (x + 1) / 8) return;
    }
    if (!tiles.find(a, BM, id / n_tiles, counted, t)) return;
    expert = t.expert;
    row = static_cast<int>(t.row);
    n0 = (id % n_tiles) * BN;
    m_left = static_cast<int>(t.hi - t.row);
    n_left = (fwd ? a.outer : a.inner) - n0;
    const int64_t lda = fwd ? a.x_stride : a.gy_stride;
    const int ks = fwd ? a.inner : a.outer;
    steps = expert < a.experts ? (ks + K - 1) / K : 0;
    A.init(static_cast<const uint16_t*>(fwd ? a.x : a.gy) + row * lda, lda, m_left, ks, ks);
    B.init(static_cast<const uint16_t*>(a.w) + expert * io + (fwd ? static_cast<int64_t>(n0) * a.inner : n0), a.inner, n_left, ks, a.inner);
  }

  const bool sums = OP == kBackwardWeight && a.grad_bias && n0 == 0 && wn == 0;
  f32x4 acc[MF][NF];
  float sum[OP == kBackwardWeight ? MF : 1];  // of this lane's values of A
#pragma unroll
  for (int i = 0; i < MF; ++i) {
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    if constexpr (OP == kBackwardWeight) sum[i] = 0.0f;
  }

  auto add_up = [&](int i, u16x8_t v) {
    if constexpr (OP == kBackwardWeight) {
      if (sums) {
        float u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = Fmt<DT>::to_f(v[e]);
        sum[i] += ((u[0] + u[1]) + (u[2] + u[3])) + ((u[4] + u[5]) + (u[6] + u[7]));
      }
    }
  };
  tile_products<DT, A_ALONG, B_ALONG, DIRECT>(A, B, lds, wm, wn, steps, acc, add_up);

  constexpr int LEN = B_ALONG ? 4 * NF : 4;  // adjacent n of a lane
  float bias[OP == kForward ? LEN : 1];
  if constexpr (OP == kForward) {
    const int n = wn + (l >> 4) * LEN;
    const uint16_t* p = static_cast<const uint16_t*>(a.bias) + static_cast<int64_t>(expert) * a.outer + n0 + n;
    const bool with = a.bias && expert < a.experts;
#pragma unroll
    for (int i = 0; i < LEN; ++i) bias[i] = with && i < n_left - n ? Fmt<DT>::to_f(p[i]) : 0.0f;
  }
  auto value = [&](int i, int j, int e) { return OP == kForward ? acc[i][j][e] + bias[4 * j + e] : acc[i][j][e]; };
  constexpr int kWaveBytes = kBytes / (WM * WN) / 16 * 16;
  char* s = lds + w * kWaveBytes;
  const int64_t pitch = OP == kBackwardWeight ? a.inner : a.out_stride;
  const int64_t at = OP == kBackwardWeight ? (part ? 0 : expert * io) + (m0 + wm) * pitch + n0 + wn : (row + wm) * pitch + n0 + wn;
  const int ml = m_left - wm, nl = n_left - wn;
  if (OP == kBackwardWeight && part)  // read back soon
    store_tile<float, false, MF, NF, LEN, kWaveBytes>(part + at, pitch, ml, nl, s, value);
  else if (a.out_dt == 0)
    store_tile<float, true, MF, NF, LEN, kWaveBytes>(static_cast<float*>(a.out) + at, pitch, ml, nl, s, value);
  else
    store_tile<uint16_t, true, MF, NF, LEN, kWaveBytes>(static_cast<uint16_t*>(a.out) + at, pitch, ml, nl, s,
                                                        [&](int i, int j, int e) { return tower_from_f<DT>(value(i, j, e)); });
  if constexpr (OP == kBackwardWeight) {
    if (sums) {  // the 4 lanes of an m have its rows 8 at a time
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        float u = sum[i] + __shfl_xor(sum[i], 16);
        u += __shfl_xor(u, 32);
        const int m = wm + 16 * i + (l & 15);
        if (l < 16 && m < m_left) {
          if (part) part[io + m0 + m] = u;
          else store_any(a.grad_bias, a.out_dt, static_cast<int64_t>(expert) * a.outer + m0 + m, u);
        }
      }
    }
  }
}

}  // namespace tbe
