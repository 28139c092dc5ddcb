// Forward, rows of up to 128 columns (cross_entropy.h).
//
// So few columns leave the matrix instructions no more to do for a logit than the exponential and what stands around it
// leave the vector unit: at 128 columns 64 cycles of products for the 64 logits that a wave holds in a register, and 8 for
// their exponential and 4 for each other instruction.  So the rows stay in registers, the items pass through LDS, and a
// wave's products of 32 items stand beside the exponentials of the 32 items before, which they do not wait for: the matrix unit
// works on the ones while the vector unit takes the others, of this wave or of the other one of its SIMD.
//  * A workgroup takes 64 MF rows, 16 MF a wave, and a range of the items.  MF = 4; MF = 1 for few rows, where the items'
//    way from memory bounds it.
//  * A ring of three tiles of 64 items in LDS, loaded two ahead, one barrier a tile.
//  * Each item has a bias, divided by the logits' factor beforehand, where the products' sums begin: 0 without biases,
//    -infinity behind the last item, so that no tile looks at the edge.
//  * A lane keeps a sum for each of its rows over all its items, less a reference that moves only when a logit is kSlack
//    powers of two above it: most tiles change nothing but the sums.  A logit costs a multiply-add, an exponential, an
//    addition and less than one instruction more.
// 2048 rows, 2 M items of 128 columns: 1.05 to 1.1 ms, 0.98 PFLOP/s (2.49 ms by tiles of 256 x 256 without rows that
// stay).  Matrix instructions are busy 46% of the cycles.  An order of single products between the exponentials, asked of the
// compiler, was not followed in this kernel (1104 us with the request, 1095 without), and where it was it cost 1 to 6% (2048 rows, 1 M
// items of 64: 375 and 370; 64 rows, 1 M items of 128: 62 and 59).
#pragma once

#include "cross_entropy_tile.h"

namespace tbe {

constexpr int kNarrowItems = 64;  // of a tile
constexpr int kRing = 3;
constexpr float kSlack = 16.0f;

template <int DT, int KS, int MF>
__global__ __launch_bounds__(256, 2) void ce_narrow_kernel(CeArgs a) {
  constexpr int T = 256, NF = 2, LEN = 4 * NF, KT = KS / 2, kRows = 64 * MF;
  using OB = Operand<true, kNarrowItems, LEN, T, true>;
  constexpr int kTile = KT * OB::kElems;
  constexpr int kLoads = KT * OB::kEach + 1;  // a wave's, of a tile
  __shared__ __align__(16) uint16_t lds[kRing * kTile];
  __shared__ __align__(16) float s_bias[kRing * 4 * kNarrowItems];  // a copy for each wave
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane_id(), g = l >> 4;
  const int count = *a.r.count, row_tiles = (count + kRows - 1) / kRows;
  // this workgroup's rows and tiles of items: a chiplet's workgroups share ranges of items
  const int64_t total = static_cast<int64_t>(row_tiles) * a.splits, x = blockIdx.x % 8;
  const int64_t id = total * x / 8 + blockIdx.x / 8;
  if (id >= total * (x + 1) / 8) return;
  const int split = static_cast<int>(id / row_tiles), m0 = static_cast<int>(id % row_tiles) * kRows + w * (16 * MF);  // the wave's first row
  const int tiles = a.items / kNarrowItems + (a.items % kNarrowItems != 0);
  const int t0 = static_cast<int>(static_cast<int64_t>(tiles) * split / a.splits), t1 = static_cast<int>(static_cast<int64_t>(tiles) * (split + 1) / a.splits);
  const int steps = (a.width + kStepK - 1) / kStepK;

  OB B;
  auto stage = [&](int t) {
    const bool in = t < t1;
    const int n0 = in ? t * kNarrowItems : 0, slot = (t - t0) % kRing;
    B.init(static_cast<const uint16_t*>(a.w) + n0 * a.w_stride, a.w_stride, in ? a.items - n0 : 0, a.width, a.width);
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      // steps past the width: with nothing in range, so that there are equally many
#pragma unroll
      for (int i = 0; i < OB::kEach; ++i) B.template load<false>(i, k < steps ? k * kStepK : a.width, lds + slot * kTile + k * OB::kElems);
    }
    const uint64_t u = reinterpret_cast<uint64_t>(a.bias + n0);
    const u32x4 r = {static_cast<uint32_t>(u), static_cast<uint32_t>(u >> 32) & 0xffffu, 0x7fffffffu, 0x00027000u};
    load_dword_to_lds(r, 4 * l, static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void*)(s_bias + (slot * 4 + w) * kNarrowItems))));
  };
  stage(t0);
  stage(t0 + 1);

  // what the exponential of base 2 takes: the sum of products times `unit`, less the row's reference
  const float unit = a.scale * kLog2e;
  // the lowest reference, before a lane has seen a logit that is not masked: times unit it stays finite, so that a masked one's
  // exponential is 0 beside it.  Lower logits count as masked
  const float floor = kFloor / fmaxf(a.scale, 1.0f);

  // the rows: lane l holds row l % 16 of each 16, 8 columns from 8 (l / 16) on of each 32
  u16x8_t fa[MF][KS];
  float ref[MF], top[MF], sum[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int m = m0 + 16 * i + (l & 15);
    const bool in = m < count;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int c = 32 * k + 8 * g;
      fa[i][k] = u16x8_t{};
      if (in && c < a.x_stride) fa[i][k] = *reinterpret_cast<const u16x8_t*>(static_cast<const uint16_t*>(a.x) + m * a.x_stride + c);
    }
    top[i] = -kInfinity;
    sum[i] = 0.0f;
    ref[i] = floor;
  }

  const int b_place = OB::read_place(((l & 15) >> 2) * LEN + (l & 3));
  // 32 items from `half` * 32 on of the tile in `slot`
  auto products = [&](f32x4 (&acc)[MF][NF], int slot, int half) {
    const uint16_t* s = lds + slot * kTile + half * 32 * kStepK;
    const int place[2] = {b_place, OB::second_half(b_place)};
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      const f32x4 from = *reinterpret_cast<const f32x4*>(s_bias + (slot * 4 + w) * kNarrowItems + half * 32 + g * LEN + 4 * j);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const u16x8_t fb = OB::read(s + k / 2 * OB::kElems + place[k % 2], 4 * j);
#pragma unroll
        for (int i = 0; i < MF; ++i) acc[i][j] = mfma16<DT>(fb, fa[i][k], k == 0 ? from : acc[i][j]);
      }
    }
  };
  // What an exponential's argument has a reference as.  Far out its rounding is worth powers of two, but a lane's exponentials of a
  // row all have the same, so it is taken out again where the reference moves and at the end.
  auto rounded = [&](float of) {
#pragma clang fp contract(off)
    return of * unit;
  };
  // Ahead of 32 items' exponentials: whether a logit asks for another reference.
  auto look = [&](const f32x4 (&acc)[MF][NF]) {
    float over = -kInfinity;
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      float most = acc[i][0][0];  // NaN stays NaN: no instruction to make sure that it is a quiet one
#pragma unroll
      for (int c = 1; c < LEN; ++c) most = __builtin_elementwise_maximum(most, acc[i][c / 4][c % 4]);
      top[i] = __builtin_elementwise_maximum(top[i], most);
      over = fmaxf(over, (most - ref[i]) * unit);  // drops NaN: such a row asks for nothing, the lane's others for themselves
    }
    if (__any(over > kSlack)) {
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        float now = fmaxf(top[i], floor);
        asm volatile("" : "+v"(now));  // keeps what follows from being worked out where it is not needed
        sum[i] *= __builtin_amdgcn_exp2f(rounded(ref[i]) - rounded(now));
        ref[i] = now;
      }
    }
  };
  auto exponentials = [&](const f32x4 (&acc)[MF][NF]) {
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const float base = -rounded(ref[i]);
      float p[LEN];
#pragma unroll
      for (int c = 0; c < LEN; ++c) p[c] = __builtin_amdgcn_exp2f(fmaf(acc[i][c / 4][c % 4], unit, base));
      sum[i] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
    }
  };

  f32x4 first[MF][NF], second[MF][NF];  // of a tile's two halves
  for (int t = t0; t < t1; ++t) {
    wait_loads<kLoads>();  // this tile's: those of the next one may be on their way
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    stage(t + 2);  // where the tile before this one was: every wave has read it
    const int slot = (t - t0) % kRing;
    if (t > t0) {
      look(second);
      products(first, slot, 0);
      exponentials(second);
    } else {
      products(first, slot, 0);
    }
    look(first);
    products(second, slot, 1);
    exponentials(first);
  }
  if (t1 > t0) {
    look(second);
    exponentials(second);
  }
  wait_loads<0>();  // nothing is on its way into LDS when the workgroup ends
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    // the lanes that share a row, each sum less the lane's largest logit; where no logit was above the floor the sum is 0 and the
    // maximum tells what there was.  Past 2^28 powers of two the sum may have overflowed, but its logarithm, of the number of items
    // at most, is no more than half a unit of lse there
    const int m = m0 + 16 * i + (l & 15);
    float most = fmaxf(top[i], __shfl_xor(top[i], 16)), s = sum[i] * __builtin_amdgcn_exp2f(-fmaf(top[i], unit, -rounded(ref[i])));
    most = fmaxf(most, __shfl_xor(most, 32));
    if (fabsf(top[i]) * unit > 0x1p28f) s = 1.0f;
    s = top[i] <= floor ? 0.0f : s * __builtin_amdgcn_exp2f((top[i] - most) * unit);
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (l < 16 && m < count) {
      // the largest and the lowest bias, over the scale and times the scale, may round to infinity
      a.part[split * a.rows + m] = make_float2(ce_times(most, a.scale), s);
    }
  }
}

template <int DT, int KS, int MF>
tbe_status ce_narrow_go(const CeArgs& a, hipStream_t s) {
  return ce_launch(ce_narrow_kernel<DT, KS, MF>, "ce_logits", 256, (a.rows + 64 * MF - 1) / (64 * MF) * a.splits, s, a);
}
template <int DT>
tbe_status ce_narrow(const CeArgs& a, bool few, hipStream_t s) {
  if (few) return a.width <= 64 ? ce_narrow_go<DT, 2, 1>(a, s) : ce_narrow_go<DT, 4, 1>(a, s);
  return a.width <= 64 ? ce_narrow_go<DT, 2, 4>(a, s) : ce_narrow_go<DT, 4, 4>(a, s);
}

}  // namespace tbe
