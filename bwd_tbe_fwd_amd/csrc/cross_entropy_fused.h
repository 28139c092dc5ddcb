// The gradients of rows of up to 128 columns without z in memory (cross_entropy.h).
//
// Writing z and reading it twice takes three times as long as its products do at 128 columns (2048 rows, 500000 items: 2 GB
// of z), so here each gradient takes the logits again and z goes from the registers of one product into those of the next:
//   X      rows stay, items pass:  grad_x(row, column)  = sum over items of z weight
//   not X  items stay, rows pass:  grad_w(item, column) = sum over rows of z grad_loss x, and the biases' gradient
// What stays is called s (64 lanes hold 16 s MF times, as the second operand of the logits' product), what passes t.
//  * Logits of 16 t and 16 s: lane l gets those of s = l % 16 and four t.  Two such are a second operand, s = l % 16 and 8 t a
//    lane, as they are: the order of the t in a product is free, if only the other operand has it too.
//  * The passing matrix is therefore read from LDS in two ways: along, 16 t and 32 columns, for the logits, and turned, 4 t
//    and 16 columns, for the gradient.  t = q + 4 r (q, r < 4) is row 4 q + r of the logits' first operand, and the 16-byte
//    columns of row t are exchanged by 2 ((t / 4) % 4): both reads then find their banks free.
//  * A row's factor goes into the exponent, ahead of the rounding of z; its sign is looked at where there is a negative one (a
//    product each instead: 1 to 3.5% more).
//  * Rows whose lse is past kFar have it taken off the logits ahead of the exponentials, behind a branch that other tiles jump over
//    (0.3%).
//  * A ring of three tiles of 64 t, loaded two ahead, one barrier a tile; two workgroups a CU, so that one's exponentials
//    are taken while the other's products are.  192 s a workgroup at 128 columns, 256 at 64: what the registers hold.
// Bound by the matrix instructions and the vector unit together (2048 rows, 500000 items of 128, all three gradients 0.93 ms, 1.12
// PFLOP/s of products, the logits' counted twice as they are taken; matrix instructions busy 50% of the cycles; a call 0.95 to
// 0.99 ms, with z in memory 1.99).
#pragma once

#include "cross_entropy_tile.h"

namespace tbe {

constexpr int kPassing = 64;  // t of a tile

constexpr int kRing = 3;

// `block`: the workgroup among this gradient's.  s_more: X: the items' biases; else the rows' references, factors, targets and far
// lse; each 64 t in the order of the lanes that ask for them.
template <int DT, bool X, int KS, int MF, bool BIAS>
__device__ __forceinline__ void ce_fused_part(const CeArgs& a, unsigned block, uint16_t* lds, uint32_t (*s_more)[4][kPassing]) {
  constexpr int T = 256, KT = KS / 2, CG = 2 * KS, kStay = 64 * MF;
  using OT = Operand<true, kPassing, 0, T, true>;
  constexpr int kTile = KT * OT::kElems;
  constexpr int kLoads = KT * OT::kEach + 1;  // a wave's, of a tile
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane_id(), g = l >> 4;
  const int count = *a.r.count, stay = X ? count : a.items, pass = X ? a.items : count;
  // 0 of them too, and as many as an int holds
  const int stay_tiles = stay / kStay + (stay % kStay != 0), pass_tiles = pass / kPassing + (pass % kPassing != 0);
  // this workgroup's s and tiles of t: a chiplet's workgroups share ranges of t
  const int64_t total = static_cast<int64_t>(stay_tiles) * a.splits, x = block % 8;
  const int64_t id = total * x / 8 + block / 8;
  if (id >= total * (x + 1) / 8) return;
  const int split = static_cast<int>(id / stay_tiles), s0 = static_cast<int>(id % stay_tiles) * kStay + w * (16 * MF);  // the wave's first s
  const int t0 = static_cast<int>(static_cast<int64_t>(pass_tiles) * split / a.splits), t1 = static_cast<int>(static_cast<int64_t>(pass_tiles) * (split + 1) / a.splits);
  const int steps = (a.width + kStepK - 1) / kStepK;
  const uint16_t* const stay_from = static_cast<const uint16_t*>(X ? a.x : a.w);
  const uint16_t* const pass_from = static_cast<const uint16_t*>(X ? a.w : a.x);
  const int64_t stay_pitch = X ? a.x_stride : a.w_stride, pass_pitch = X ? a.w_stride : a.x_stride;
  // wave w brings one of the arrays of s_more
  const void* const more_from = X ? static_cast<const void*>(a.bias) : w == 0 ? static_cast<const void*>(a.r.ref) : w == 1 ? static_cast<const void*>(a.r.part) : w == 2 ? static_cast<const void*>(a.r.target) : static_cast<const void*>(a.r.far);
  const bool more = !X || w == 0;
  // place l of a tile's 64: t = 16 (l / 16) + (l / 4) % 4 + 4 (l % 4); targets in their own order
  const int more_at = !X && w == 2 ? l : (l & 48) + ((l >> 2) & 3) + 4 * (l & 3);

  OT P;
  auto stage = [&](int t) {
    const bool in = t < t1;
    const int n0 = in ? t * kPassing : 0, slot = (t - t0) % kRing;
    P.init(pass_from + n0 * pass_pitch, pass_pitch, in ? pass - n0 : 0, a.width, a.width);
#pragma unroll
    for (int k = 0; k < KT; ++k) {
#pragma unroll
      for (int i = 0; i < OT::kEach; ++i) P.template load<false>(i, k < steps ? k * kStepK : a.width, lds + slot * kTile + k * OT::kElems);
    }
    const uint64_t u = reinterpret_cast<uint64_t>(more_from) + 4ull * n0;
    const u32x4 r = {static_cast<uint32_t>(u), static_cast<uint32_t>(u >> 32) & 0xffffu, 0x7fffffffu, 0x00027000u};
    load_dword_to_lds(r, more ? 4 * more_at : kOutside, static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void*)&s_more[slot][w][0])));
  };
  stage(t0);
  stage(t0 + 1);

  // what stays: lane l holds s = l % 16 of each 16, 8 columns from 8 (l / 16) on of each 32
  u16x8_t fs[MF][KS];
  float ref[MF], sum[MF], far[MF];
  f32x4 from[MF];  // not X: the items' biases, where the sums begin
  int target[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int s = s0 + 16 * i + (l & 15);
    const bool in = s < stay;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int c = 32 * k + 8 * g;
      fs[i][k] = u16x8_t{};
      if (in && c < a.width) fs[i][k] = *reinterpret_cast<const u16x8_t*>(stay_from + s * stay_pitch + c);
    }
    sum[i] = 0.0f;
    if constexpr (X) {
      ref[i] = in ? a.r.ref[s] : -kInfinity;
      target[i] = in ? a.r.target[s] - a.first : -1;
      far[i] = in ? a.r.far[s] : 0.0f;
    } else {
      const float b = in ? a.bias[s] : -kInfinity;
      from[i] = f32x4{b, b, b, b};
    }
  }
  const float unit = a.scale * kLog2e;
  bool away = false;  // the wave has rows whose lse is past kFar
  if constexpr (X) {
#pragma unroll
    for (int i = 0; i < MF; ++i) away |= far[i] != 0.0f;
    away = __any(away);
  }
  f32x4 out[MF][CG];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int c = 0; c < CG; ++c) out[i][c] = f32x4{0, 0, 0, 0};

  // this lane's places in LDS, in elements: along, t = q + 4 r with 4 q + r = l % 16; turned, t = g + 4 q and 4 columns
  const int q = (l & 15) >> 2, r = l & 3;
  const int along = (q + 4 * r) * kStepK + ((g ^ (2 * r)) << 3);  // the second 32 columns: exchanged with 4
  int turned[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) turned[c] = (g + 4 * q) * kStepK + (((2 * c + (r >> 1)) ^ (2 * q)) << 3) + (r & 1) * 4;

  for (int t = t0; t < t1; ++t) {
    wait_loads<kLoads>();  // this tile's: those of the next one may be on their way
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    stage(t + 2);  // where the tile before this one was: every wave has read it
    const int slot = (t - t0) % kRing, n0 = t * kPassing;
    const uint16_t* const tile = lds + slot * kTile;
    uint64_t hits = 0;  // not X: rows whose target is one of this wave's items
    bool minus = false;
    if constexpr (!X) {
      minus = __any(__uint_as_float(s_more[slot][1][l]) < 0.0f);
      away = __any(s_more[slot][3][l] != 0);
      hits = __ballot(s_more[slot][2][l] - static_cast<unsigned>(a.first + s0) < 16u * MF);
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      f32x4 acc[MF][2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        f32x4 begin = {0, 0, 0, 0};
        if constexpr (X) begin = *reinterpret_cast<const f32x4*>(&s_more[slot][0][half * 32 + 16 * j + 4 * g]);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const u16x8_t ft = *reinterpret_cast<const u16x8_t*>(tile + k / 2 * OT::kElems + ((k & 1) ? along ^ 32 : along) + (half * 32 + 16 * j) * kStepK);
#pragma unroll
          for (int i = 0; i < MF; ++i) acc[i][j] = mfma16<DT>(ft, fs[i][k], k > 0 ? acc[i][j] : X ? begin : from[i]);
        }
      }
      if (__builtin_expect(away, 0)) {
#pragma unroll
        for (int i = 0; i < MF; ++i) {
          float lse = 0.0f;
          if constexpr (X) lse = s0 + 16 * i + (l & 15) < stay ? a.r.far[s0 + 16 * i + (l & 15)] : 0.0f;
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (!X) lse = __uint_as_float(s_more[slot][3][half * 32 + 16 * j + 4 * g + e]);
              if (lse != 0.0f) acc[i][j][e] = ce_near(acc[i][j][e], a.scale, a.over, lse);
            }
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        f32x4 less = {};
        if constexpr (!X) less = *reinterpret_cast<const f32x4*>(&s_more[slot][0][half * 32 + 16 * j + 4 * g]);
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_amdgcn_exp2f(fmaf(acc[i][j][e], unit, X ? ref[i] : less[e]));
      }
      if constexpr (X) {
        bool here = false;
#pragma unroll
        for (int i = 0; i < MF; ++i) here |= static_cast<unsigned>(target[i] - n0 - half * 32) < 32u;
        if (__any(here)) {
#pragma unroll
          for (int i = 0; i < MF; ++i) {
            int at = target[i] - n0 - half * 32 - g;
            asm volatile("" : "+v"(at));  // keeps what follows from being worked out where it is not needed
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[i][j][e] -= at == 16 * j + 4 * e ? kUnit<DT> : 0.0f;
          }
        }
      } else {
        // all rows of the half at once: with few items every row's target is here (353 rows, 42 items of 80: 20 us, and 118 with one
        // row after the other)
        if ((hits >> (32 * half)) & 0xffffffffu) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              unsigned at = s_more[slot][2][half * 32 + 16 * j + 4 * e + g] - static_cast<unsigned>(a.first + s0 + (l & 15));
              asm volatile("" : "+v"(at));  // keeps what follows from being worked out where it is not needed
              const float one = fabsf(__uint_as_float(s_more[slot][1][half * 32 + 16 * j + 4 * g + e])) * kUnit<DT>;
#pragma unroll
              for (int i = 0; i < MF; ++i) acc[i][j][e] -= at == 16u * i ? one : 0.0f;
            }
        }
        if (minus) {  // rows with a negative factor: its size is in the reference
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const f32x4 part = *reinterpret_cast<const f32x4*>(&s_more[slot][1][half * 32 + 16 * j + 4 * g]);
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[i][j][e] = part[e] < 0.0f ? -acc[i][j][e] : acc[i][j][e];
          }
        }
        if constexpr (BIAS) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) sum[i] += acc[i][j][e];
        }
      }
      u16x8_t z[MF];
#pragma unroll
      for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) z[i][e] = tower_from_f<DT>(acc[i][e / 4][e % 4]);
#pragma unroll
      for (int c = 0; c < CG; ++c) {
        u16x8_t fy;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const s16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(tile + c / 4 * OT::kElems + turned[c % 4] + (half * 32 + 16 * h) * kStepK));
#pragma unroll
          for (int e = 0; e < 4; ++e) fy[4 * h + e] = static_cast<uint16_t>(v[e]);
        }
#pragma unroll
        for (int i = 0; i < MF; ++i) out[i][c] = mfma16<DT>(fy, z[i], out[i][c]);
      }
    }
  }
  wait_loads<0>();  // nothing is on its way into LDS when the workgroup ends

  // lane l has s = l % 16 and columns 16 c + 4 (l / 16) .. + 4
  const bool whole = !X && a.splits == 1;
  const float factor = whole ? a.factor * *a.r.largest : 1.0f;
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int s = s0 + 16 * i + (l & 15);
    if (s < stay && (a.out || !whole)) {
#pragma unroll
      for (int c = 0; c < CG; ++c) {
        const int n = 16 * c + 4 * g;
        if (n >= a.out_width) continue;
        if (whole) {
          Vec<uint16_t, 4> v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v.e[e] = tower_from_f<DT>(out[i][c][e] * factor);
          store_vec_part<uint16_t, 4>(static_cast<uint16_t*>(a.out) + s * a.out_stride + n, a.out_width - n, v);
        } else {
          float* p = a.sum + (static_cast<int64_t>(split) * (X ? a.rows : a.items) + s) * a.sum_pitch + n;
          if (X && a.add) out[i][c] += load_f4(p);
          store_f4(p, out[i][c]);
        }
      }
    }
    if constexpr (BIAS) {
      float b = sum[i] + __shfl_xor(sum[i], 16);
      b += __shfl_xor(b, 32);
      if (g == 0 && s < stay) a.bias_part[split * a.bias_stride + s] = b;
    }
  }
}

// Both gradients in one launch, the rows' workgroups first: the one's last workgroups run beside the other's first.
template <int DT, int KS, int MF, bool BIAS>
__global__ __launch_bounds__(256, 2) void ce_fused_kernel(CeArgs ax, CeArgs aw, unsigned x_groups) {
  __shared__ __align__(16) uint16_t lds[kRing * (KS / 2) * kPassing * kStepK];
  __shared__ __align__(16) uint32_t s_more[kRing][4][kPassing];
  if (blockIdx.x < x_groups) ce_fused_part<DT, true, KS, MF, false>(ax, blockIdx.x, lds, s_more);
  else ce_fused_part<DT, false, KS, MF, BIAS>(aw, blockIdx.x - x_groups, lds, s_more);
}

template <int DT, int KS, int MF>
tbe_status ce_fused(const CeArgs& x, const CeArgs& w, hipStream_t s) {
  constexpr int kStay = 64 * MF;
  const int64_t xg = ce_groups((x.rows + kStay - 1) / kStay * x.splits), wg = ce_groups((w.items + int64_t{kStay} - 1) / kStay * w.splits);
  const unsigned x_groups = static_cast<unsigned>(xg);
  if (w.bias_part) return ce_launch(ce_fused_kernel<DT, KS, MF, true>, "ce_grads", 256, xg + wg, s, x, w, x_groups);
  return ce_launch(ce_fused_kernel<DT, KS, MF, false>, "ce_grads", 256, xg + wg, s, x, w, x_groups);
}

}  // namespace tbe
