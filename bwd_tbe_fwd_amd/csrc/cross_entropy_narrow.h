// Logits of rows of up to 256 columns (cross_entropy.h says what becomes of them).
//
// So few columns leave the matrix instructions no more to do for a logit than the exponential and what stands around it
// leave the vector unit: at 128 columns 16 cycles a product of 16 x 16 x 32, four for each 64 x 32 logits of a lane group's 32,
// against 16 an exponential and 4 an instruction.  So the rows stay in registers, the items pass through LDS, and a wave's
// products of 32 items are taken between the exponentials of the 32 items before.
//  * A workgroup takes 64 MF rows, 16 MF a wave, and a range of the items.  MF = 4; MF = 1 for few rows, where the items'
//    way from memory bounds it.
//  * A ring of three tiles of 64 items in LDS, loaded two ahead, one barrier a tile.  z is stored by equally many stores in
//    every wave (what lies outside goes past the buffer's range), so that the wait for a tile's loads leaves the stores and
//    loads of the last step on their way.
//  * Each item has a bias, divided by the logits' factor beforehand, where the products' sums begin: 0 without biases,
//    -infinity behind the last item, so that no tile looks at the edge.
//  * Forward a lane keeps a sum for each of its rows over all its items, less a reference that moves only when a logit is
//    2^kSlack above it, as powers of two go: most tiles change nothing but the sums.  A logit costs a multiply-add, an
//    exponential, an addition and less than one instruction more.
#pragma once

#include "cross_entropy_tile.h"

namespace tbe {

constexpr int kNarrowItems = 64;  // of a tile
constexpr int kRing = 3;
constexpr float kSlack = 16.0f;
constexpr float kFloor = -1e38f;  // a reference is no lower, so that it stays finite

// One dword a lane from offset `o` of the buffer to LDS, lane l's at lds + 4 l (load_to_lds of tile_products.h is its like).
__device__ __forceinline__ void load_dword_to_lds(u32x4 r, uint32_t o, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(o), "s"(r) : "memory", "m0");
}

// Sums over the 16 lanes of a row of v[c], c < 8: lane l gets that of c = l % 8.  Lanes exchange halves: 7 additions, not 32.
__device__ __forceinline__ float columns_sum(const float (&v)[8]) {
  const int l = lane_id();
  float a[4], b[2];
  const bool h2 = l & 4, h1 = l & 2, h0 = l & 1;
  // lanes l and 7 - l of 8: the lower keeps c < 4 and hands over the others
#pragma unroll
  for (int c = 0; c < 4; ++c) a[c] = (h2 ? v[c + 4] : v[c]) + dpp_f<kDppHalfMirror>(h2 ? v[c] : v[c + 4]);
  // then l xor 2, then l xor 1
#pragma unroll
  for (int c = 0; c < 2; ++c) b[c] = (h1 ? a[c + 2] : a[c]) + dpp_f<kDppXor2>(h1 ? a[c] : a[c + 2]);
  const float s = (h0 ? b[1] : b[0]) + dpp_f<kDppXor1>(h0 ? b[0] : b[1]);
  return s + dpp_f<0x128>(s);  // row_ror:8, the other 8 lanes of the row
}

template <int DT, bool BACK, int KS, int MF>
__global__ __launch_bounds__(256, 2) void ce_narrow_kernel(CeArgs a) {
  constexpr int T = 256, NF = 2, LEN = 4 * NF, KT = KS / 2, kRows = 64 * MF;
  using OB = Operand<true, kNarrowItems, LEN, T, true>;
  constexpr int kTile = KT * OB::kElems;
  constexpr int kLoads = KT * OB::kEach + 1;  // a wave's, of a tile
  constexpr int kStores = MF;                 // of 32 items of z, and one for their columns' sums
  __shared__ __align__(16) uint16_t lds[kRing * kTile];
  __shared__ __align__(16) float s_bias[kRing * 4 * kNarrowItems];  // a copy for each wave
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane_id(), g = l >> 4;
  const int count = *a.r.count, row_tiles = (count + kRows - 1) / kRows;
  // this workgroup's rows and tiles of items: a chiplet's workgroups share ranges of items
  const int64_t total = static_cast<int64_t>(row_tiles) * a.splits, x = blockIdx.x % 8;
  const int64_t id = total * x / 8 + blockIdx.x / 8;
  if (id >= total * (x + 1) / 8) return;
  const int split = static_cast<int>(id / row_tiles), m0 = static_cast<int>(id % row_tiles) * kRows + w * (16 * MF);  // the wave's first row
  const int tiles = (a.items + kNarrowItems - 1) / kNarrowItems;
  const int t0 = static_cast<int>(static_cast<int64_t>(tiles) * split / a.splits), t1 = static_cast<int>(static_cast<int64_t>(tiles) * (split + 1) / a.splits);
  const int steps = (a.width + kStepK - 1) / kStepK;

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
    const uint64_t u = reinterpret_cast<uint64_t>(a.bias + (t < t1 ? n0 : 0));
    const u32x4 r = {static_cast<uint32_t>(u), static_cast<uint32_t>(u >> 32) & 0xffffu, 0x7fffffffu, 0x00027000u};
    load_dword_to_lds(r, 4 * l, static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void*)(s_bias + (slot * 4 + w) * kNarrowItems))));
  };
  stage(t0);
  stage(t0 + 1);

  // the rows: lane l holds row l % 16 of each 16, 8 columns from 8 (l / 16) on of each 32
  u16x8_t fa[MF][KS];
  int target[MF];
  float ref[MF], grad[MF];      // backward: -lse in powers of two
  float top[MF], sum[MF];       // forward
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
    ref[i] = kFloor;
    if constexpr (BACK) {
      target[i] = in ? a.r.target[m] - a.first : -1;
      const float e = in ? a.r.lse[m] : 0.0f;
      ref[i] = e < kFloor ? -kInfinity : fmaf(e, -kLog2e, DT == 1 ? 15.0f : 0.0f);  // every item masked: no probability
      grad[i] = in && a.bias_part ? a.r.grad[m] / kUnit<DT> : 0.0f;
    }
  }
  // what the exponential of base 2 takes: the sum of products times `unit`, less the row's reference
  const float unit = a.scale * kLog2e;

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
  // Products between the exponentials' instructions, an equal share each.
  auto interleave = [&] {
    constexpr int kProducts = MF * NF * KS, kVector = MF * (BACK ? LEN : 2 * LEN + 2);
#pragma unroll
    for (int q = 0; q < kProducts; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, (kVector + kProducts - 1) / kProducts, 0);
      __builtin_amdgcn_sched_group_barrier(0x400, (MF * LEN + kProducts - 1) / kProducts, 0);
    }
  };
  // Forward, ahead of their exponentials: whether a logit asks for another reference.
  auto look = [&](const f32x4 (&acc)[MF][NF]) {
    if constexpr (!BACK) {
      float over = kFloor;
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        float most = acc[i][0][0];  // NaN stays NaN: no instruction to make sure that it is a quiet one
#pragma unroll
        for (int c = 1; c < LEN; ++c) most = __builtin_elementwise_maximum(most, acc[i][c / 4][c % 4]);
        top[i] = __builtin_elementwise_maximum(top[i], most);
        over = __builtin_elementwise_maximum(over, (most - ref[i]) * unit);
      }
      if (__any(over > kSlack)) {
#pragma unroll
        for (int i = 0; i < MF; ++i) {
          float now = fmaxf(top[i], kFloor);
          asm volatile("" : "+v"(now));  // keeps what follows from being worked out where it is not needed
          sum[i] *= __builtin_amdgcn_exp2f((ref[i] - now) * unit);
          ref[i] = now;
        }
      }
    }
  };
  // The logits of 32 items from n0 on, and what becomes of them.
  auto consume = [&](f32x4 (&acc)[MF][NF], int n0) {
    if constexpr (!BACK) {
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        const float base = -ref[i] * unit;
        float p[LEN];
#pragma unroll
        for (int c = 0; c < LEN; ++c) p[c] = __builtin_amdgcn_exp2f(fmaf(acc[i][c / 4][c % 4], unit, base));
        sum[i] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
      }
    } else {
      bool here = false;
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        here |= static_cast<unsigned>(target[i] - n0) < 32u;
#pragma unroll
        for (int c = 0; c < LEN; ++c) acc[i][c / 4][c % 4] = __builtin_amdgcn_exp2f(fmaf(acc[i][c / 4][c % 4], unit, ref[i]));
      }
      if (__any(here)) {
#pragma unroll
        for (int i = 0; i < MF; ++i) {
          int at = target[i] - n0 - g * LEN;
          asm volatile("" : "+v"(at));  // keeps what follows from being worked out where it is not needed
#pragma unroll
          for (int c = 0; c < LEN; ++c) acc[i][c / 4][c % 4] -= c == at ? kUnit<DT> : 0.0f;
        }
      }
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(a.z + n0 / 64 * a.panel + n0 % 64, 0, 0x7fffffff, 0x00027000);
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        const int m = m0 + 16 * i + (l & 15);
        Vec<uint16_t, LEN> v;
#pragma unroll
        for (int c = 0; c < LEN; ++c) v.e[c] = tower_from_f<DT>(acc[i][c / 4][c % 4]);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, m < count ? static_cast<uint32_t>(m) * 128 + g * LEN * 2 : kOutside, 0, 0);
      }
      if (a.bias_part) {
        float columns[LEN];
#pragma unroll
        for (int c = 0; c < LEN; ++c) {
          columns[c] = 0.0f;
#pragma unroll
          for (int i = 0; i < MF; ++i)
            if (m0 + 16 * i + (l & 15) < count) columns[c] = fmaf(acc[i][c / 4][c % 4], grad[i], columns[c]);
        }
        const float column = columns_sum(columns);
        const int n = n0 + g * LEN + (l & 7);
        const __amdgpu_buffer_rsrc_t q = __builtin_amdgcn_make_buffer_rsrc(a.bias_part + m0 / (16 * MF) * a.bias_stride, 0, 0x7fffffff, 0x00027000);
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(column), q, (l & 8) == 0 && n < a.items && m0 < count ? 4 * n : kOutside, 0, 0);
      }
    }
  };

  f32x4 first[MF][NF], second[MF][NF];  // of a tile's two halves
  for (int t = t0; t < t1; ++t) {
    // this tile's loads: the next one's may be on their way, and the stores of the last step
    if (BACK && t > t0 + 1) {
      if (a.bias_part) wait_loads<kLoads + 2 * (kStores + 1)>();
      else wait_loads<kLoads + 2 * kStores>();
    } else if (BACK && t > t0) {
      if (a.bias_part) wait_loads<kLoads + kStores + 1>();
      else wait_loads<kLoads + kStores>();
    } else {
      wait_loads<kLoads>();
    }
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    stage(t + 2);  // where the tile before this one was: every wave has read it
    const int slot = (t - t0) % kRing;
    if (t > t0) {
      look(second);
      products(first, slot, 0);
      consume(second, (t - 1) * kNarrowItems + 32);
      interleave();
    } else {
      products(first, slot, 0);
    }
    look(first);
    products(second, slot, 1);
    consume(first, t * kNarrowItems);
    interleave();
  }
  if (t1 > t0) {
    look(second);
    consume(second, (t1 - 1) * kNarrowItems + 32);
  }
  wait_loads<0>();  // nothing is on its way into LDS when the workgroup ends
  if constexpr (!BACK) {
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      // the lanes that share a row; where no logit was above kFloor the sum is 0 and the maximum tells what there was
      const int m = m0 + 16 * i + (l & 15);
      float all = fmaxf(ref[i], __shfl_xor(ref[i], 16)), most = fmaxf(top[i], __shfl_xor(top[i], 16));
      all = fmaxf(all, __shfl_xor(all, 32));
      most = fmaxf(most, __shfl_xor(most, 32));
      float s = sum[i] * __builtin_amdgcn_exp2f((ref[i] - all) * unit);
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      if (l < 16 && m < count) a.part[split * a.rows + m] = make_float2(most <= kFloor ? (most == -kInfinity ? most : most * a.scale) : all * a.scale, s);
    }
  }
}

template <int DT, bool BACK, int KS, int MF>
tbe_status ce_narrow_go(const CeArgs& a, hipStream_t s) {
  return ce_launch(ce_narrow_kernel<DT, BACK, KS, MF>, BACK ? "ce_z" : "ce_logits", 256, (a.rows + 64 * MF - 1) / (64 * MF) * a.splits, 1, a, s);
}
template <int DT, bool BACK>
tbe_status ce_narrow(const CeArgs& a, bool few, hipStream_t s) {
  if (few) return a.width <= 64 ? ce_narrow_go<DT, BACK, 2, 1>(a, s) : a.width <= 128 ? ce_narrow_go<DT, BACK, 4, 1>(a, s) : ce_narrow_go<DT, BACK, 8, 1>(a, s);
  return a.width <= 64 ? ce_narrow_go<DT, BACK, 2, 4>(a, s) : a.width <= 128 ? ce_narrow_go<DT, BACK, 4, 4>(a, s) : ce_narrow_go<DT, BACK, 8, 4>(a, s);
}

}  // namespace tbe
