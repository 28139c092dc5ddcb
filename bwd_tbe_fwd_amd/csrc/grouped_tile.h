// The tiled kernel of the grouped products (grouped_linear.h says what m, n, k, "along" and
// "across" are): a workgroup takes BM x BN of C and walks k in steps of 64 through two LDS buffers.
//
// Bound by the matrix instructions where the sides are large, so everything else has to stay out of
// their way:
//  * Operands go from memory to LDS without registers (buffer loads with an LDS destination, 16
//    bytes a lane), one step ahead of the products, with one barrier a step.  Lanes past the
//    matrix's edge get an offset past the buffer's range and so write zeros: the edges of the
//    groups cost no branch in the loop.  Rows that do not start on 16 bytes (or k or n that are not
//    whole 16 bytes) go through registers instead, with the same LDS layout.
//  * LDS holds an operand as it lies in memory, along: [m][64 k], across: [64 k][m].  The 16-byte
//    columns of a row are exchanged by a pattern of the row (along) or the 32-byte columns by one of
//    k (across), so that the 16 rows that a read takes lie in different banks.
//  * An across operand is turned on the way from LDS to the registers (ds_read_b64_tr_b16: 16 lanes
//    read 4 k x 16 m and each gets 4 k of one m).
//  * The products are taken as C^T: a lane then holds adjacent n of one m, 4 of each product.  Where B
//    lies along, the 16 n of one product are 4 at a time from 4 blocks of 4 NF, so that a lane's NF
//    products give 4 NF adjacent n (an across read of such n would meet in the same banks).
#pragma once

#include "grouped_linear.h"

namespace tbe {

constexpr uint32_t kOutside = 0x80000000u;  // a buffer offset past any range

typedef uint16_t u16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

// Exchange of an along row's K / 8 columns of 16 bytes.  A 16-byte LDS read is served 16 lanes at a
// time, lanes 0-3, 12-15 and 20-27, then 4-11, 16-19 and 28-31: of rows q = row / 4 (or the 4 blocks of
// 16 that a read of B takes), 0 and 3 at one column with 1 and 2 at the next.  With these patterns
// they differ in their place within 256 bytes, all banks (conflict counter: 0).
template <int K>
__device__ __forceinline__ int along_pattern(int r) {
  const int h = ((r >> 2) ^ (r >> 4)) & 3;
  return K == 64 ? ((r >> 1) & 1) | h << 1 : h ^ (h & 1) << 1;
}
// Exchange of an across row's columns of 32 bytes: k of the 4 x 4 rows that a read takes differ.
template <int SIDE>
__device__ __forceinline__ int across_pattern(int k) {
  const int f = (k & 3) | ((k >> 3) & 1) << 2;
  return SIDE >= 128 ? f : f & 3;
}

// 16 bytes a lane from offset `o` of the buffer to LDS, lane l's at lds + 16 l.  Written as an
// instruction because the compiler, which cannot tell the LDS buffers apart, would wait for every
// load under way before each LDS read; it writes no register but m0, which the compiler uses for
// nothing here, and wait_loads is its wait.
__device__ __forceinline__ void load_to_lds(u32x4 r, uint32_t o, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(o), "s"(r) : "memory");
}

// One operand's tile of SIDE m by K k, THREADS threads.
template <bool ALONG, int SIDE, int K, int THREADS, bool DIRECT>
struct Operand {
  static constexpr int kChunks = SIDE * K / 8;     // of 16 bytes
  static constexpr int kEach = kChunks / THREADS;
  static constexpr int kRowChunks = ALONG ? K / 8 : SIDE / 8;
  static_assert(kChunks % THREADS == 0, "whole chunks a thread");

  const uint16_t* base;  // (m0, k = 0)
  int64_t ld;
  int64_t ms, ks;
  uint32_t at[kEach];    // DIRECT: byte offset of a chunk, or kOutside
  u16x8_t reg[DIRECT ? 1 : kEach];

  // row of LDS (m or k) and the chunk of the matrix's row that a thread's i-th chunk holds
  __device__ __forceinline__ static void place(int i, int& row, int& chunk) {
    const int q = i * THREADS + threadIdx.x;
    row = q / kRowChunks;
    const int slot = q % kRowChunks;
    chunk = ALONG ? slot ^ along_pattern<K>(row) : slot ^ (across_pattern<SIDE>(row) << 1);
  }
  __device__ __forceinline__ void init(const uint16_t* p, int64_t stride, int64_t m_left, int64_t k_left) {
    base = p;
    ld = stride;
    ms = m_left;
    ks = k_left;
    if constexpr (DIRECT) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        int row, chunk;
        place(i, row, chunk);
        const bool in = ALONG ? row < ms : chunk * 8 < ms;
        at[i] = in ? static_cast<uint32_t>(row * ld * 2 + chunk * 16) : kOutside;
      }
    }
  }
  // Starts the loads of step k0.
  __device__ __forceinline__ void load(int64_t k0, uint16_t* __restrict s) {
    const uint16_t* p = base + (ALONG ? k0 : k0 * ld);
    const int64_t left = ks - k0;
    if constexpr (DIRECT) {
      const uint64_t u = reinterpret_cast<uint64_t>(p);
      const u32x4 r = {static_cast<uint32_t>(u), static_cast<uint32_t>(u >> 32) & 0xffffu, 0x7fffffffu, 0x00027000u};
      const uint32_t lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void*)s)) +
                           __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * (kWave * 16);
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        uint32_t o = at[i];
        if (left < K) {
          int row, chunk;
          place(i, row, chunk);
          if ((ALONG ? chunk * 8 : row) >= left) o = kOutside;
        }
        load_to_lds(r, o, lds + i * THREADS * 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        int row, chunk;
        place(i, row, chunk);
        Vec<uint16_t, 8> v;
        const int64_t n = (ALONG ? row < ms : row < left) ? (ALONG ? left : ms) - chunk * 8 : 0;
        load_vec_part<uint16_t, 8>(p + row * ld + chunk * 8, n, v);
        __builtin_memcpy(&reg[i], v.e, 16);
      }
    }
  }
  // Registers to LDS, where the loads went there.
  __device__ __forceinline__ void store(uint16_t* s) {
    if constexpr (!DIRECT) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) *reinterpret_cast<u16x8_t*>(s + (i * THREADS + threadIdx.x) * 8) = reg[i];
    }
  }
};

// The 8 k from 32 step + 8 (lane / 16) on of one m: along: m = `m` of this lane; across: `m` is the
// first of the 4 adjacent m that this lane reads for its group of 16, and the lane gets the group's
// (lane % 16)-th.
template <bool ALONG, int SIDE, int K>
__device__ __forceinline__ u16x8_t fragment(const uint16_t* s, int m, int step) {
  const int l = lane_id(), g = l >> 4;
  if constexpr (ALONG) {
    return *reinterpret_cast<const u16x8_t*>(s + m * K + (((4 * step + g) ^ along_pattern<K>(m)) << 3));
  } else {
    u16x8_t r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = 32 * step + 8 * g + 4 * h + ((l & 15) >> 2);
      const uint16_t* p = s + k * SIDE + (((m >> 4) ^ across_pattern<SIDE>(k)) << 4) + (m & 15);
      const s16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
#pragma unroll
      for (int i = 0; i < 4; ++i) r[4 * h + i] = static_cast<uint16_t>(v[i]);
    }
    return r;
  }
}

// N floats of row `p` of out from column n on, `left` of them inside.
template <int N>
__device__ __forceinline__ void store_out(void* out, int dt, int64_t at, int64_t left, const float (&v)[N]) {
  if (dt == 0) {
    Vec<float, N> o;
#pragma unroll
    for (int i = 0; i < N; ++i) o.e[i] = v[i];
    store_vec_part<float, N>(static_cast<float*>(out) + at, left, o);
  } else {
    Vec<uint16_t, N> o;
#pragma unroll
    for (int i = 0; i < N; ++i) o.e[i] = dt == 1 ? tower_from_f<1>(v[i]) : tower_from_f<2>(v[i]);
    store_vec_part<uint16_t, N>(static_cast<uint16_t*>(out) + at, left, o);
  }
}

// Waits until at most N of this wave's loads are on their way and its LDS reads are done.  (Fields of
// the counter word: loads in bits 0-3 and 14-15, LDS in 8-11, exports in 4-6, left alone.)
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "a 6-bit counter");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x70);
  asm volatile("" ::: "memory");
}

// Workgroup `id` of `n` as the id-th of the chiplets' contiguous shares: consecutive workgroups go to
// the 8 chiplets in turn, so each chiplet's L2 then sees neighbouring tiles.
__device__ __forceinline__ unsigned chiplet_order(unsigned id, unsigned n) {
  const unsigned x = id % 8, q = n / 8, r = n % 8;
  return x * q + min(x, r) + id / 8;
}

// K: k of a step; S: LDS buffers, S - 1 steps are on their way while one is read.
template <int DT, int OP, int BM, int BN, int WM, int WN, int K, int S, bool DIRECT>
__global__ __launch_bounds__(WM * WN * kWave, 2) void grouped_tile_kernel(GroupedArgs a, int n_tiles) {
  constexpr int T = WM * WN * kWave;
  constexpr int MF = BM / WM / 16, NF = BN / WN / 16;  // products of 16 x 16 a wave
  constexpr bool A_ALONG = OP != kBackwardWeight, B_ALONG = OP == kForward;
  static_assert(DIRECT || S == 2, "through registers: one step ahead");
  __shared__ __align__(16) uint16_t sa[S][BM * K], sb[S][BN * K];
  using OA = Operand<A_ALONG, BM, K, T, DIRECT>;
  using OB = Operand<B_ALONG, BN, K, T, DIRECT>;
  OA A;
  OB B;
  const int64_t io = static_cast<int64_t>(a.inner) * a.outer;
  int expert;
  int64_t row = 0, m0 = 0, n0;
  if constexpr (OP == kBackwardWeight) {
    const int m_tiles = (a.outer + BM - 1) / BM, tiles = n_tiles * m_tiles;
    expert = blockIdx.x / tiles;
    // experts differ in their rows: each one's tiles are shared among the chiplets
    const int t = chiplet_order(blockIdx.x % tiles, tiles);
    m0 = static_cast<int64_t>(t % m_tiles) * BM;
    n0 = static_cast<int64_t>(t / m_tiles) * BN;
    const RowRange r = rows_of(a, expert);
    A.init(static_cast<const uint16_t*>(a.gy) + r.lo * a.gy_stride + m0, a.gy_stride, a.outer - m0, r.hi - r.lo);
    B.init(static_cast<const uint16_t*>(a.x) + r.lo * a.x_stride + n0, a.x_stride, a.inner - n0, r.hi - r.lo);
  } else {
    constexpr bool fwd = OP == kForward;
    const unsigned id = chiplet_order(blockIdx.x, gridDim.x);
    RowTile t;
    if (!find_row_tile(a, BM, id / n_tiles, t)) return;
    expert = t.expert;
    row = t.row;
    n0 = static_cast<int64_t>(id % n_tiles) * BN;
    const int64_t lda = fwd ? a.x_stride : a.gy_stride;
    const int64_t ks = expert < a.experts ? (fwd ? a.inner : a.outer) : 0;
    A.init(static_cast<const uint16_t*>(fwd ? a.x : a.gy) + row * lda, lda, t.hi - t.row, ks);
    B.init(static_cast<const uint16_t*>(a.w) + expert * io + (fwd ? n0 * a.inner : n0), a.inner, (fwd ? a.outer : a.inner) - n0, ks);
  }
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane_id();
  const int wm = (w / WN) * (MF * 16), wn = (w % WN) * (NF * 16);
  // this lane's place in a product's 16 m and 16 n
  const int am = wm + (A_ALONG ? l & 15 : 4 * (l & 3));
  const int bn = wn + (B_ALONG ? ((l & 15) >> 2) * (4 * NF) + (l & 3) : 4 * (l & 3));
  constexpr int kNext = B_ALONG ? 4 : 16;  // n from one product to the next
  const bool sums = OP == kBackwardWeight && a.grad_bias && n0 == 0 && wn == 0;
  f32x4 acc[MF][NF], acc1[OP == kBackwardWeight ? MF : 1];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    if constexpr (OP == kBackwardWeight) acc1[i] = f32x4{0, 0, 0, 0};
  }

  const int steps = static_cast<int>((A.ks + K - 1) / K);
  u16x8_t ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = DT == 2 ? 0x3f80 : 0x3c00;
#pragma unroll
  for (int k = 0; k < S - 1; ++k) {
    A.load(static_cast<int64_t>(k) * K, sa[k]);
    B.load(static_cast<int64_t>(k) * K, sb[k]);
    A.store(sa[k]);
    B.store(sb[k]);
  }
  // A step's loads are always started, past the end with nothing in range, so that the number under
  // way is the same at every wait.  At `it`, steps it + 1 .. it + S - 2 may still be under way; the
  // buffer read at it - 1 takes step it + S - 1.
  int cur = 0, nxt = S - 1;
  for (int it = 0; it < steps; ++it) {
    wait_loads<DIRECT ? (S - 2) * (OA::kEach + OB::kEach) : 63>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    A.load(static_cast<int64_t>(it + S - 1) * K, sa[nxt]);
    B.load(static_cast<int64_t>(it + S - 1) * K, sb[nxt]);
#pragma unroll
    for (int k = 0; k < K / 32; ++k) {
      u16x8_t fa[MF], fb[NF];
#pragma unroll
      for (int j = 0; j < NF; ++j) fb[j] = fragment<B_ALONG, BN, K>(sb[cur], bn + kNext * j, k);
#pragma unroll
      for (int i = 0; i < MF; ++i) fa[i] = fragment<A_ALONG, BM, K>(sa[cur], am + 16 * i, k);
#pragma unroll
      for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[i][j] = mfma16<DT>(fb[j], fa[i], acc[i][j]);
      if constexpr (OP == kBackwardWeight) {
        if (sums) {
#pragma unroll
          for (int i = 0; i < MF; ++i) acc1[i] = mfma16<DT>(ones, fa[i], acc1[i]);
        }
      }
    }
    A.store(sa[nxt]);
    B.store(sb[nxt]);
    cur = cur + 1 == S ? 0 : cur + 1;
    nxt = nxt + 1 == S ? 0 : nxt + 1;
  }
  wait_loads<0>();  // LDS stays this workgroup's until the last load is done

  // this lane: m = wm + 16 i + l % 16; RUNS runs of LEN adjacent n from wn + LEN (l / 16) on
  constexpr int LEN = B_ALONG ? 4 * NF : 4, RUNS = 4 * NF / LEN;
  const int n = wn + (l >> 4) * LEN;
  float bias[OP == kForward ? LEN : 1];
  if constexpr (OP == kForward) {
    static_assert(RUNS == 1, "one run");
    const uint16_t* p = static_cast<const uint16_t*>(a.bias) + static_cast<int64_t>(expert) * a.outer + n0 + n;
    const bool with = a.bias && expert < a.experts;
#pragma unroll
    for (int i = 0; i < LEN; ++i) bias[i] = with && i < B.ms - n ? Fmt<DT>::to_f(p[i]) : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int m = wm + 16 * i + (l & 15);
    if (m >= A.ms) continue;
    const int64_t at = (OP == kBackwardWeight ? expert * io + (m0 + m) * a.inner : (row + m) * a.out_stride) + n0 + n;
#pragma unroll
    for (int u = 0; u < RUNS; ++u) {
      float v[LEN];
#pragma unroll
      for (int e = 0; e < LEN; ++e) {
        v[e] = acc[i][u * (LEN / 4) + e / 4][e % 4];
        if constexpr (OP == kForward) v[e] += bias[e];
      }
      store_out<LEN>(a.out, a.out_dt, at + 16 * u, B.ms - n - 16 * u, v);
    }
    if constexpr (OP == kBackwardWeight) {
      if (sums && l < 16) store_any(a.grad_bias, a.out_dt, static_cast<int64_t>(expert) * a.outer + m0 + m, acc1[i][0]);
    }
  }
}

}  // namespace tbe
