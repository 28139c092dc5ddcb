// Logits of rows of up to 256 columns (cross_entropy.h says what becomes of them).
//
// So few columns leave 2 width operations of the matrix instructions for each logit, as long as the exponential and what
// stands around it take on the vector unit: at 128 columns 16 cycles a product of 16 x 16 x 32 against 4 cycles an
// instruction and 16 an exponential, 256 logits a wave.  So the rows stay in registers, the items pass through LDS, and the
// two waves of a SIMD, of different workgroups, overlap: while one takes products the other takes exponentials.
//  * A workgroup takes kRows<WM> rows and a range of the items.  WM = 4: 64 rows a wave, all waves the same items; WM = 1,
//    for few rows: 64 rows in all, a quarter of the items a wave.
//  * A ring of three tiles of 64 items in LDS, loaded two ahead, one barrier a tile.  What a wave stores leaves before the
//    loads of its step start: the loads' counter then needs no look at the stores.
//  * Forward a lane keeps a maximum and a sum for its 4 rows over all its items; lanes, waves and workgroups are joined at
//    the end.  The logits' factor goes into the exponential's argument and the biases, divided by it beforehand, are where
//    the products' sums begin: a logit then costs a multiply-add, an exponential, a half of a maximum and an addition.
#pragma once

#include "cross_entropy_tile.h"

namespace tbe {

constexpr int kNarrowItems = 64;  // of a tile
constexpr int kRing = 3;
template <int WM> constexpr int kNarrowRows = 64 * WM;

// One dword a lane from offset `o` of the buffer to LDS, lane l's at lds + 4 l (load_to_lds of tile_products.h is its like).
__device__ __forceinline__ void load_dword_to_lds(u32x4 r, uint32_t o, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(o), "s"(r) : "memory", "m0");
}

template <int DT, bool BACK, bool BIAS, int KS, int WM>
__global__ __launch_bounds__(256, 2) void ce_narrow_kernel(CeArgs a) {
  constexpr int T = 256, MF = 4, WN = 4 / WM, NF = 4 / WN, LEN = 4 * NF, KT = KS / 2;
  using OB = Operand<true, kNarrowItems, 4 * NF, T, true>;
  constexpr int kTile = KT * OB::kElems;
  constexpr int kLoads = KT * OB::kEach + (BIAS ? 1 : 0);  // a wave's, of a tile
  __shared__ __align__(16) uint16_t lds[kRing * kTile];
  __shared__ __align__(16) float s_bias[BIAS ? kRing * 4 * kNarrowItems : 1];  // a copy for each wave
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane_id(), g = l >> 4;
  const int wm = w / WN * 64, wn = w % WN * (16 * NF);
  const int count = *a.r.count, row_tiles = (count + kNarrowRows<WM> - 1) / kNarrowRows<WM>;
  // this workgroup's rows and tiles of items: a chiplet's workgroups share ranges of items
  const int64_t total = static_cast<int64_t>(row_tiles) * a.splits, x = blockIdx.x % 8;
  const int64_t id = total * x / 8 + blockIdx.x / 8;
  if (id >= total * (x + 1) / 8) return;
  const int split = static_cast<int>(id / row_tiles), m0 = static_cast<int>(id % row_tiles) * kNarrowRows<WM>;
  const int tiles = (a.items + kNarrowItems - 1) / kNarrowItems;
  const int t0 = static_cast<int>(static_cast<int64_t>(tiles) * split / a.splits), t1 = static_cast<int>(static_cast<int64_t>(tiles) * (split + 1) / a.splits);
  const int steps = (a.width + kStepK - 1) / kStepK;

  // the rows: lane l holds row l % 16 of each 16, 8 columns from 8 (l / 16) on of each 32
  u16x8_t fa[MF][KS];
  int target[MF];
  float lse[MF], grad[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int m = m0 + wm + 16 * i + (l & 15);
    const bool in = m < count;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int c = 32 * k + 8 * g;
      fa[i][k] = u16x8_t{};
      if (in && c < a.x_stride) fa[i][k] = *reinterpret_cast<const u16x8_t*>(static_cast<const uint16_t*>(a.x) + m * a.x_stride + c);
    }
    if constexpr (BACK) {
      target[i] = in ? a.r.target[m] - a.first - wn - g * LEN : -1;
      const float e = in ? a.r.lse[m] : 0.0f;
      lse[i] = e < -1e38f ? -kInfinity : fmaf(e, -kLog2e, DT == 1 ? 15.0f : 0.0f);  // every item masked: no probability
      grad[i] = in ? a.r.grad[m] / kUnit<DT> : 0.0f;
    }
  }
  // what the exponential of base 2 takes: the sum of products times `unit`, less the row's reference
  const float unit = a.scale * kLog2e;

  OB B;
  auto stage = [&](int t) {
    const int n0 = t * kNarrowItems, slot = (t - t0) % kRing;
    const int n_left = t < t1 ? a.items - n0 : 0;
    B.init(static_cast<const uint16_t*>(a.w) + (t < t1 ? n0 * a.w_stride : 0), a.w_stride, n_left, a.width, a.width);
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      // steps past the width: with nothing in range, so that there are equally many
#pragma unroll
      for (int i = 0; i < OB::kEach; ++i) B.template load<false>(i, k < steps ? k * kStepK : a.width, lds + slot * kTile + k * OB::kElems);
    }
    if constexpr (BIAS) {
      const uint64_t u = reinterpret_cast<uint64_t>(a.bias + (t < t1 ? n0 : 0));
      const u32x4 r = {static_cast<uint32_t>(u), static_cast<uint32_t>(u >> 32) & 0xffffu, 0x7fffffffu, 0x00027000u};
      load_dword_to_lds(r, l < n_left ? 4 * l : kOutside,
                        static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void*)(s_bias + (slot * 4 + w) * kNarrowItems))));
    }
  };

  float top[MF], sum[MF];  // forward
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    top[i] = -kInfinity;
    sum[i] = 0.0f;
  }
  u32x2 z[BACK ? MF : 1][BACK ? NF : 1];  // backward: the last tile's, and its columns' sums
  float column = 0.0f;
  auto store_z = [&](int t) {
    if constexpr (BACK) {
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        const int m = m0 + wm + 16 * i + (l & 15);
        if (m < count) {
          uint16_t* p = a.z + t * a.panel + static_cast<int64_t>(m) * 64 + wn + g * LEN;
#pragma unroll
          for (int j = 0; j + 1 < NF; j += 2) *reinterpret_cast<u32x4*>(p + 4 * j) = u32x4{z[i][j].x, z[i][j].y, z[i][j + 1].x, z[i][j + 1].y};
          if constexpr (NF == 1) *reinterpret_cast<u32x2*>(p) = z[i][0];
        }
      }
      // lane l has the sum of item g LEN + l % 16; with 4 items a lane group the first 4 lanes do
      const int n = t * kNarrowItems + wn + g * LEN + (l & 15);
      if (a.bias_part && (l & 15) < LEN && n < a.items && m0 + wm < count) a.bias_part[(m0 + wm) / 64 * a.bias_stride + n] = column;
    }
  };

  const int b_place = OB::read_place(wn + ((l & 15) >> 2) * LEN + (l & 3));
  const int b_half[2] = {b_place, OB::second_half(b_place)};
  stage(t0);
  stage(t0 + 1);
  for (int t = t0; t < t1; ++t) {
    wait_loads<kLoads>();  // this tile's: those of the next one may be on their way
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (BACK && t > t0) store_z(t - 1);
    stage(t + 2);          // where the tile before this one was: every wave has read it
    const int slot = (t - t0) % kRing;
    f32x4 acc[MF][NF];
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      f32x4 from = {0, 0, 0, 0};
      if constexpr (BIAS) from = *reinterpret_cast<const f32x4*>(s_bias + (slot * 4 + w) * kNarrowItems + wn + g * LEN + 4 * j);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const u16x8_t fb = OB::read(lds + slot * kTile + k / 2 * OB::kElems + b_half[k % 2], 4 * j);
#pragma unroll
        for (int i = 0; i < MF; ++i) acc[i][j] = mfma16<DT>(fb, fa[i][k], k == 0 ? from : acc[i][j]);
      }
    }
    const int n0 = t * kNarrowItems;
    const int left = a.items - n0 - wn - g * LEN;  // of this lane's items
    const bool edge = a.items - n0 < kNarrowItems;
    if constexpr (!BACK) {
      if (edge) {
#pragma unroll
        for (int c = 0; c < LEN; ++c)
          if (c >= left)
#pragma unroll
            for (int i = 0; i < MF; ++i) acc[i][c / 4][c % 4] = -kInfinity;
      }
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        float most = acc[i][0][0];
#pragma unroll
        for (int c = 1; c < LEN; ++c) most = fmaxf(most, acc[i][c / 4][c % 4]);
        const float old = fmaxf(top[i], -1e38f);  // a reference that stays finite
        top[i] = fmaxf(top[i], most);
        const float from = fmaxf(top[i], -1e38f), base = -from * unit;
        if (__any(from > old)) sum[i] *= __builtin_amdgcn_exp2f((old - from) * unit);
        float part[4] = {};
#pragma unroll
        for (int c = 0; c < LEN; ++c) part[c % 4] += __builtin_amdgcn_exp2f(fmaf(acc[i][c / 4][c % 4], unit, base));
        sum[i] += (part[0] + part[1]) + (part[2] + part[3]);
      }
    } else {
      float columns[LEN];
#pragma unroll
      for (int c = 0; c < LEN; ++c) columns[c] = 0.0f;
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        float p[LEN];
#pragma unroll
        for (int c = 0; c < LEN; ++c) p[c] = __builtin_amdgcn_exp2f(fmaf(acc[i][c / 4][c % 4], unit, lse[i]));
        const unsigned at = static_cast<unsigned>(target[i] - n0);
        if (__any(at < LEN)) {
#pragma unroll
          for (int c = 0; c < LEN; ++c) p[c] -= c == static_cast<int>(at) ? kUnit<DT> : 0.0f;
        }
        if (edge) {
#pragma unroll
          for (int c = 0; c < LEN; ++c)
            if (c >= left) p[c] = 0.0f;
        }
        if (a.bias_part && m0 + wm + 16 * i + (l & 15) < count) {
#pragma unroll
          for (int c = 0; c < LEN; ++c) columns[c] = fmaf(p[c], grad[i], columns[c]);
        }
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          Vec<uint16_t, 4> v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v.e[e] = tower_from_f<DT>(p[4 * j + e]);
          z[i][j] = __builtin_bit_cast(u32x2, v);
        }
      }
      if (a.bias_part) {
#pragma unroll
        for (int c = 0; c < LEN; ++c) {
          const float s = lanes_sum<16>(columns[c]);
          if (c == (l & 15)) column = s;
        }
      }
    }
  }
  wait_loads<0>();  // nothing is on its way into LDS when the workgroup ends
  if constexpr (BACK) {
    if (t1 > t0) store_z(t1 - 1);
  } else {
    float2* stat = reinterpret_cast<float2*>(lds);  // [WN][rows]
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const float from = fmaxf(top[i], -1e38f);
      float all = fmaxf(top[i], __shfl_xor(top[i], 16));
      all = fmaxf(all, __shfl_xor(all, 32));
      float s = sum[i] * __builtin_amdgcn_exp2f((from - fmaxf(all, -1e38f)) * unit);
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      if (l < 16) stat[w % WN * kNarrowRows<WM> + wm + 16 * i + l] = make_float2(all == -kInfinity ? all : all * a.scale, s);
    }
    __syncthreads();
    if (threadIdx.x < kNarrowRows<WM> && m0 + static_cast<int>(threadIdx.x) < count) {
      float2 all = stat[threadIdx.x];
      for (int k = 1; k < WN; ++k) all = ce_join(all, stat[k * kNarrowRows<WM> + threadIdx.x]);
      a.part[split * a.rows + m0 + threadIdx.x] = all;
    }
  }
}

template <int DT, bool BACK, int KS, int WM>
tbe_status ce_narrow_go(CeArgs a, hipStream_t s) {
  const int64_t groups = ((a.rows + kNarrowRows<WM> - 1) / kNarrowRows<WM>) * a.splits;
  const char* what = BACK ? "ce_z" : "ce_logits";
  return a.bias ? ce_launch(ce_narrow_kernel<DT, BACK, true, KS, WM>, what, 256, groups, 1, a, s)
                : ce_launch(ce_narrow_kernel<DT, BACK, false, KS, WM>, what, 256, groups, 1, a, s);
}
template <int DT, bool BACK>
tbe_status ce_narrow(const CeArgs& a, bool few, hipStream_t s) {
  if (few)
    return a.width <= 64 ? ce_narrow_go<DT, BACK, 2, 1>(a, s) : a.width <= 128 ? ce_narrow_go<DT, BACK, 4, 1>(a, s) : ce_narrow_go<DT, BACK, 8, 1>(a, s);
  return a.width <= 64 ? ce_narrow_go<DT, BACK, 2, 4>(a, s) : a.width <= 128 ? ce_narrow_go<DT, BACK, 4, 4>(a, s) : ce_narrow_go<DT, BACK, 8, 4>(a, s);
}

}  // namespace tbe
