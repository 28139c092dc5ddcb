// The tiled kernels of the cross entropy (cross_entropy.h says what m, n and k are).
#pragma once

#include "cross_entropy.h"
#include "tile_products.h"

namespace tbe {

// Workgroup `block`'s place among m_tiles x n_tiles of each share of k: a contiguous part for each chiplet, and in it bands
// of 8 tiles of m walked along n, so that the 32 workgroups that a chiplet runs at once read 8 + 4 tiles of operands and not
// 1 + 32.  False: none.
struct TilePlace {
  int m, n, share;
};
__device__ __forceinline__ bool tile_place(int64_t m_tiles, int64_t n_tiles, int shares, unsigned block, TilePlace& t) {
  const int64_t tiles = m_tiles * n_tiles, total = tiles * shares, x = block % 8;
  int64_t id = total * x / 8 + block / 8;
  if (id >= total * (x + 1) / 8) return false;
  t.share = static_cast<int>(id / tiles);
  id -= t.share * tiles;
  const int64_t band = id / (8 * n_tiles);
  const int r = static_cast<int>(id - band * 8 * n_tiles);
  const int high = static_cast<int>(m_tiles - band * 8 < 8 ? m_tiles - band * 8 : 8);
  t.m = static_cast<int>(band) * 8 + r % high;
  t.n = r / high;
  return true;
}

// Logits of BM rows and BN items, and what becomes of them.  The logits leave the matrix instructions 16 or 32 a lane and are
// used up there: forward, a maximum and a sum of 16 bytes for every BN items leave the workgroup; backward, z.  Bound by the
// matrix instructions, which wait while a tile's exponentials are taken, since 256 x 256 leave room for one workgroup a CU.
// 8192 rows (0.9 of them with a target), 65536 items of 1024, bf16: forward 857 us, 1.15 PFLOP/s (busy 56% of the cycles; the
// library's product alone, logits stored, all rows, takes 920); backward 16384 items 276 us (0.90, 40%): 0.24 GB of z are stored
// in each.  8 rows, 131072 items: 51 us, 5.2 TB/s (41 where the last pass left half of the weights in the Infinity Cache).  Rows
// with a far lse are looked for once a wave, behind all loads (right behind each row's: 16384 items 6 us more).
template <int DT, bool BACK, int BM, int BN, int WM, int WN, bool DIRECT>
__global__ __launch_bounds__(WM * WN * kWave, BM * BN <= 64 * 64 ? 4 : 2) void ce_logits_kernel(CeArgs a) {
  constexpr int T = WM * WN * kWave;
  constexpr int MF = BM / WM / 16, NF = BN / WN / 16, LEN = 4 * NF;  // LEN adjacent items of a lane
  using OA = Operand<true, BM, 4, T, DIRECT>;
  using OB = Operand<true, BN, 4 * NF, T, DIRECT>;
  constexpr int kBytes = 2 * 2 * (OA::kElems + OB::kElems);
  __shared__ __align__(16) char lds[kBytes];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane_id();
  const int wm = (w / WN) * (MF * 16), wn = (w % WN) * (NF * 16);
  const int count = *a.r.count;
  TilePlace t;
  if (!tile_place((count + BM - 1) / BM, (a.items + BN - 1) / BN, 1, blockIdx.x, t)) return;
  const int m0 = t.m * BM, n0 = t.n * BN;
  const int m_left = count - m0, n_left = a.items - n0;
  OA A;
  OB B;
  A.init(static_cast<const uint16_t*>(a.x) + m0 * a.x_stride, a.x_stride, m_left, a.width, a.width);
  B.init(static_cast<const uint16_t*>(a.w) + n0 * a.w_stride, a.w_stride, n_left, a.width, a.width);
  f32x4 acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  tile_products<DT, true, true, DIRECT>(A, B, lds, wm, wn, (a.width + kStepK - 1) / kStepK, acc, [](int, u16x8_t) {});

  // this lane's items: n .. n + LEN of the tile
  const int n = wn + (l >> 4) * LEN;
  float bias[LEN];
#pragma unroll
  for (int c = 0; c < LEN; ++c) bias[c] = a.bias && n + c < n_left ? a.bias[n0 + n + c] : 0.0f;
  // behind the other loads, so that nothing waits between them
  auto as_counted = [&] {
#pragma unroll
    for (int c = 0; c < LEN; ++c) bias[c] = ce_bias(bias[c], a.most);
  };
  auto logit = [&](int i, int c) { return fmaf(acc[i][c / 4][c % 4], a.scale, bias[c]); };
  if constexpr (!BACK) {
    float2* stat = reinterpret_cast<float2*>(lds);  // [WN][BM]
    as_counted();
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int m = wm + 16 * i + (l & 15);
      float v[LEN], top = -kInfinity;
#pragma unroll
      for (int c = 0; c < LEN; ++c) {
        v[c] = n + c < n_left ? logit(i, c) : -kInfinity;
        top = fmaxf(top, v[c]);
      }
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float from = top == -kInfinity ? 0.0f : top;  // no item that is not masked: the sum is 0
      float sum = 0.0f;
#pragma unroll
      for (int c = 0; c < LEN; ++c) sum += __builtin_amdgcn_exp2f((v[c] - from) * kLog2e);
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (l < 16) stat[(w % WN) * BM + m] = make_float2(top, sum);
    }
    __syncthreads();
    for (int m = threadIdx.x; m < BM; m += T) {
      float2 all = stat[m];
      for (int k = 1; k < WN; ++k) all = ce_join(all, stat[k * BM + m]);
      if (m < m_left) a.part[t.n * a.rows + m0 + m] = all;
    }
  } else {
    // z in place of the logits, times its unit
    constexpr float kOne = kUnit<DT>;
    const float shift = DT == 1 ? 15.0f : 0.0f;
    float columns[LEN];
#pragma unroll
    for (int c = 0; c < LEN; ++c) columns[c] = 0.0f;
    // the rows' loads under way together
    float lses[MF], grads[MF];
    int targets[MF];
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int m = wm + 16 * i + (l & 15);
      lses[i] = 0.0f;
      grads[i] = 0.0f;
      targets[i] = -1;
      if (m < m_left) {
        lses[i] = a.r.lse[m0 + m];
        targets[i] = a.r.target[m0 + m];
        if (a.bias_part) grads[i] = a.r.grad[m0 + m];
      }
    }
    as_counted();
    bool far = false;
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      far |= fabsf(lses[i]) > kFar;
#pragma unroll
      for (int c = 0; c < LEN; ++c) acc[i][c / 4][c % 4] = logit(i, c);
    }
    if (__builtin_expect(__any(far), 0)) {
      // lse is taken off before anything is rounded to powers of two: it is at least the row's largest logit, to the bit, so that
      // no probability passes 1 however large they are
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        float less = lses[i] == -kInfinity ? kInfinity : lses[i];  // every item is masked: no probability
        asm volatile("" : "+v"(less));  // keeps what follows from being worked out where it is not needed
#pragma unroll
        for (int c = 0; c < LEN; ++c) acc[i][c / 4][c % 4] -= less;
        lses[i] = 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int m = wm + 16 * i + (l & 15);
      const bool in = m < m_left;
      const unsigned at = in ? static_cast<unsigned>(targets[i] - a.first - n0 - n) : ~0u;
      const float base = fmaf(lses[i], -kLog2e, shift);
#pragma unroll
      for (int c = 0; c < LEN; ++c) acc[i][c / 4][c % 4] = __builtin_amdgcn_exp2f(fmaf(acc[i][c / 4][c % 4], kLog2e, base));
      if (__any(at < LEN)) {
        int here = static_cast<int>(at);
        asm volatile("" : "+v"(here));  // keeps what follows from being worked out where it is not needed
#pragma unroll
        for (int c = 0; c < LEN; ++c) acc[i][c / 4][c % 4] -= c == here ? kOne : 0.0f;
      }
      if (n_left < BN) {  // z's columns up to a whole 16 bytes are read
#pragma unroll
        for (int c = 0; c < LEN; ++c)
          if (n + c >= n_left) acc[i][c / 4][c % 4] = 0.0f;
      }
      if (a.bias_part) {
        const float g = grads[i] / kOne;
#pragma unroll
        for (int c = 0; c < LEN; ++c) columns[c] = in ? fmaf(acc[i][c / 4][c % 4], g, columns[c]) : columns[c];
      }
    }
    if (a.bias_part) {
      float* sums = reinterpret_cast<float*>(lds);  // [WM][BN]
#pragma unroll
      for (int c = 0; c < LEN; ++c) {
        const float s = lanes_sum<16>(columns[c]);
        if ((l & 15) == 0) sums[(w / WN) * BN + n + c] = s;
      }
      __syncthreads();
      for (int k = threadIdx.x; k < BN; k += T) {
        float s = sums[k];
        for (int q = 1; q < WM; ++q) s += sums[q * BN + k];
        if (k < n_left) a.bias_part[t.m * a.bias_stride + n0 + k] = s;
      }
      __syncthreads();
    }
    constexpr int kWaveBytes = kBytes / (WM * WN) / 16 * 16;
    static_assert(NF * 16 <= 64, "a wave's items lie in one panel");
    uint16_t* out = a.z + (n0 + wn) / 64 * a.panel + static_cast<int64_t>(m0 + wm) * 64 + (n0 + wn) % 64;
    store_tile<uint16_t, false, MF, NF, LEN, kWaveBytes>(out, 64, m_left - wm, (n_left + 7) / 8 * 8 - wn, lds + w * kWaveBytes,
                                                         [&](int i, int j, int e) { return tower_from_f<DT>(acc[i][j][e]); });
  }
}

// The two products of z.  X: the gradient of x, else of the weights; `block`: the workgroup among this gradient's.  A chiplet
// takes whole shares of k where there are many: few rows' weights are then read by one (64 rows, 131072 items of 1000: 61 us,
// and 85 with each share's tiles dealt to all eight).  Bound by the matrix instructions: 16384 items and 8192 rows (0.9 with a
// target) of 1024, both 371 us, 1.33 PFLOP/s, busy 64% of the cycles.
template <bool X, int BM, int BN, int WM, int WN>
struct GradTile {
  static constexpr int T = WM * WN * kWave, MF = BM / WM / 16, NF = BN / WN / 16;
  using OA = PanelOperand<X, BM, 4, T, true>;
  using OB = Operand<false, BN, 4 * NF, T, true>;
  static constexpr int kBytes = 2 * 2 * (OA::kElems + OB::kElems);
};
template <int DT, bool X, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void ce_grad_part(const CeArgs& a, unsigned block, char* lds) {
  using G = GradTile<X, BM, BN, WM, WN>;
  constexpr int MF = G::MF, NF = G::NF, kBytes = G::kBytes;
  using OA = typename G::OA;
  using OB = typename G::OB;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane_id();
  const int wm = (w / WN) * (MF * 16), wn = (w % WN) * (NF * 16);
  const int count = *a.r.count, ms = X ? count : a.items, ks = X ? a.items : count;
  TilePlace t;
  if (!tile_place((ms + BM - 1) / BM, (a.out_width + BN - 1) / BN, a.splits, block, t)) return;
  const int m0 = t.m * BM, n0 = t.n * BN;
  const int m_left = ms - m0, n_left = a.out_width - n0;
  // parts of whole steps
  const int each = ((ks + a.splits - 1) / a.splits + kStepK - 1) / kStepK * kStepK;
  const int64_t k0 = min(static_cast<int64_t>(t.share) * each, static_cast<int64_t>(ks));
  const int k = min(each, static_cast<int>(ks - k0));
  OA A;
  OB B;
  if constexpr (X) {
    A.init(a.z, a.panel, m0, k0, m_left, k);
    B.init(static_cast<const uint16_t*>(a.w) + k0 * a.w_stride + n0, a.w_stride, n_left, k, a.width);
  } else {
    A.init(a.z, a.panel, m0, k0, m_left, k);
    B.init(static_cast<const uint16_t*>(a.xg) + k0 * a.x_stride + n0, a.x_stride, n_left, k, a.width);
  }
  const int64_t pitch = a.sum_pitch;
  float* const sum = a.sum + (static_cast<int64_t>(t.share) * (X ? a.rows : a.items) + m0 + wm) * pitch + n0 + wn;
  f32x4 acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int m = 16 * i + (l & 15);
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      const int n = 16 * j + 4 * (l >> 4);
      acc[i][j] = f32x4{0, 0, 0, 0};
      if (X && a.add && m < m_left - wm) {
        Vec<float, 4> v;
        load_vec_part<float, 4>(sum + m * pitch + n, n_left - wn - n, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = v.e[e];
      }
    }
  }
  tile_products<DT, X, false, true>(A, B, lds, wm, wn, (k + kStepK - 1) / kStepK, acc, [](int, u16x8_t) {});
  constexpr int kWaveBytes = kBytes / (WM * WN) / 16 * 16;
  char* s = lds + w * kWaveBytes;
  if (!X && a.splits == 1) {
    const float factor = a.factor * *a.r.largest;
    store_tile<uint16_t, true, MF, NF, 4, kWaveBytes>(static_cast<uint16_t*>(a.out) + (m0 + wm) * a.out_stride + n0 + wn, a.out_stride,
                                                      m_left - wm, n_left - wn, s,
                                                      [&](int i, int j, int e) { return tower_from_f<DT>(acc[i][j][e] * factor); });
  } else {
    store_tile<float, false, MF, NF, 4, kWaveBytes>(sum, pitch, m_left - wm, n_left - wn, s,
                                                    [&](int i, int j, int e) { return acc[i][j][e]; });
  }
}

// Both in one launch, the rows' workgroups first, where their tiles are alike; X: the gradient of x alone, of a tile that the
// weights' has not.
template <int DT, bool X, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * kWave, BM * BN <= 64 * 64 ? 4 : 2) void ce_grad_kernel(CeArgs ax, CeArgs aw, unsigned x_groups) {
  constexpr int kX = GradTile<true, BM, BN, WM, WN>::kBytes, kW = GradTile<false, BM, BN, WM, WN>::kBytes;
  __shared__ __align__(16) char lds[X || kX > kW ? kX : kW];
  if (X || blockIdx.x < x_groups) {
    ce_grad_part<DT, true, BM, BN, WM, WN>(ax, blockIdx.x, lds);
    return;
  }
  if constexpr (!X) ce_grad_part<DT, false, BM, BN, WM, WN>(aw, blockIdx.x - x_groups, lds);
}

inline int64_t ce_groups(int64_t tiles) { return (tiles + 7) / 8 * 8; }  // for the chiplets' shares
template <typename K, typename... A>
tbe_status ce_launch(K* kernel, const char* what, int threads, int64_t groups, hipStream_t s, const A&... args) {
  groups = ce_groups(groups);
  if (groups * threads >= (int64_t{1} << 32)) {
    set_error("cross entropy: %lld tiles are more than a launch takes", static_cast<long long>(groups));
    return TBE_ERR_UNSUPPORTED;
  }
  ProfScope ps(what, s);
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(groups)), dim3(threads), 0, s, args...);
  return check_launch(what);
}
inline int64_t ce_tiles(int64_t m, int bm, int64_t n, int bn) { return ((m + bm - 1) / bm) * ((n + bn - 1) / bn); }

template <int DT, bool BACK>
tbe_status ce_logits(const CeArgs& a, int tile, hipStream_t s) {
  const char* what = BACK ? "ce_z" : "ce_logits";
  if (tile == kTile256) return ce_launch(ce_logits_kernel<DT, BACK, 256, 256, 2, 4, true>, what, 512, ce_tiles(a.rows, 256, a.items, 256), s, a);
  if (tile == kTile128) return ce_launch(ce_logits_kernel<DT, BACK, 128, 128, 2, 2, true>, what, 256, ce_tiles(a.rows, 128, a.items, 128), s, a);
  if (tile == kTile64x256)
    return ce_launch(ce_logits_kernel<DT, BACK, 64, 256, 1, 4, true>, what, 256, ce_tiles(a.rows, 64, a.items, 256), s, a);
  return ce_launch(ce_logits_kernel<DT, BACK, 64, 64, 2, 2, true>, what, 256, ce_tiles(a.rows, 64, a.items, 64), s, a);
}
// One of them where the other has no shares.
template <int DT, int BM, int BN, int WM, int WN>
tbe_status ce_grad(const CeArgs& x, const CeArgs& w, hipStream_t s) {
  const int64_t xg = ce_groups(ce_tiles(x.rows, BM, x.out_width, BN) * x.splits), wg = ce_groups(ce_tiles(w.items, BM, w.out_width, BN) * w.splits);
  return ce_launch(ce_grad_kernel<DT, false, BM, BN, WM, WN>, "ce_grads", WM * WN * kWave, xg + wg, s, x, w, static_cast<unsigned>(xg));
}
template <int DT>
tbe_status ce_grads(const CeArgs& x, int x_tile, const CeArgs& w, int w_tile, hipStream_t s) {
  if (x.splits && w.splits && x_tile != w_tile) {
    CeArgs none = w;
    none.splits = 0;
    const tbe_status st = ce_grads<DT>(x, x_tile, none, x_tile, s);
    if (st != TBE_OK) return st;
    none = x;
    none.splits = 0;
    return ce_grads<DT>(none, w_tile, w, w_tile, s);
  }
  const int tile = x.splits ? x_tile : w_tile;
  if (tile == kTile256) return ce_grad<DT, 256, 256, 2, 4>(x, w, s);
  if (tile == kTile128) return ce_grad<DT, 128, 128, 2, 2>(x, w, s);
  if (tile == kTile64) return ce_grad<DT, 64, 64, 2, 2>(x, w, s);
  return ce_launch(ce_grad_kernel<DT, true, 256, 128, 4, 2>, "ce_grads", 512, ce_tiles(x.rows, 256, x.out_width, 128) * x.splits, s, x, w, 0u);
}

}  // namespace tbe
