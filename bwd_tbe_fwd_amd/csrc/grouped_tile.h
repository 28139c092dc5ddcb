// The tiled kernel of the grouped products (grouped_linear.h says what m, n, k, "along" and
// "across" are): a workgroup takes BM x BN of C and walks k through two LDS buffers of 64 k.
//
// Bound by the matrix instructions where the sides are large, so everything else has to stay out of
// their way:
//  * Operands go from memory to LDS without registers (buffer loads with an LDS destination, 16
//    bytes a lane), one step ahead of the products, with one barrier a step.  Lanes past the
//    matrix's edge get an offset past the buffer's range and so write zeros: the edges of the
//    groups cost no branch in the loop.  Rows that do not start on 16 bytes (or k or n that are not
//    whole 16 bytes) go through registers instead, with the same LDS layout: 60000 rows, 8 experts, 1777 x
//    1201 forward take 340 us where 1776 x 1200 take 242.
//  * LDS holds an operand as it lies in memory, along: [m][64 k], across: [64 k][m].  The 16-byte
//    columns of an along row are exchanged by a pattern of the row, and the across rows are put in an
//    order with gaps, so that what a read takes lies in different banks.  A lane's place in a read
//    is a base that never changes plus a constant: no address arithmetic between the products.
//  * An across operand is turned on the way from LDS to the registers (ds_read_b64_tr_b16: 16 lanes
//    read 4 k x 16 m and each gets 4 k of one m).
//  * Only the last steps look at the matrix's end: the others' loads have no compare and no branch
//    (131072 rows, 16 experts, 4096 x 1024: forward 978 -> 955 us).
//  * The products are taken as C^T: a lane then holds adjacent n of one m, 4 of each product.  Where B
//    lies along, the 16 n of one product are 4 at a time from 4 blocks of 4 NF, so that a lane's NF
//    products give 4 NF adjacent n (an across read of such n would meet in the same banks).
#pragma once

#include <type_traits>

#include "grouped_linear.h"

namespace tbe {

constexpr int kStepK = 64;                  // k of an LDS buffer: two products'
constexpr uint32_t kOutside = 0x80000000u;  // a buffer offset past any range

typedef uint16_t u16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

// Exchange of an along row's 8 columns of 16 bytes.  A 16-byte LDS read is served 16 lanes at a time,
// lanes 0-3, 12-15 and 20-27, then 4-11, 16-19 and 28-31: of the blocks q = 0 .. 3 of 4 rows that a
// read takes, 0 and 3 at one column with 1 and 2 at the next.  With these patterns they differ in
// their place within 256 bytes, all banks (conflict counter: 0).  A read's blocks lie GAP rows apart.
template <int GAP>
__device__ __forceinline__ int along_pattern(int r) {
  return ((r >> 1) & 1) | ((r / GAP) & 3) << 1;
}
// Place of an across row k in LDS, in elements.  A load instruction fills 1024 bytes: rows k = 8 g + 4 h
// + r of one r together (h = 0, 1, and as many g as fit), 32 bytes before those of the next r: the 4
// rows of a read lie in different banks.
template <int SIDE> constexpr int kTogether = 256 / SIDE;  // g
template <int SIDE>
__device__ __forceinline__ int across_place(int k) {
  const int r = k & 3, h = (k >> 2) & 1, g = k >> 3;
  return (4 * (g / kTogether<SIDE>) + r) * (512 + 16) + (g % kTogether<SIDE> * 2 + h) * SIDE;
}

// 16 bytes a lane from offset `o` of the buffer to LDS, lane l's at lds + 16 l.  Written as an
// instruction because the compiler, which cannot tell the LDS buffers apart, would wait for every
// load under way before each LDS read; it writes no register but m0, and wait_loads is its wait.
__device__ __forceinline__ void load_to_lds(u32x4 r, uint32_t o, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(o), "s"(r) : "memory", "m0");
}

// One operand's tile of SIDE m by kStepK k, THREADS threads.
template <bool ALONG, int SIDE, int GAP, int THREADS, bool DIRECT>
struct Operand {
  static constexpr int K = kStepK;
  static constexpr int kChunks = SIDE * K / 8;          // of 16 bytes
  static constexpr int kEach = kChunks / THREADS;
  static constexpr int kElems = ALONG ? SIDE * K : SIDE * K / 512 * (512 + 16);  // of an LDS buffer
  static_assert(kChunks % THREADS == 0, "whole chunks a thread");
  static_assert(ALONG || SIDE == 256 || SIDE == 128 || SIDE == 64, "whole rows a load instruction");

  const uint16_t* base;  // (m0, k = 0)
  int64_t ld;
  int ms, ks;            // that lie inside from there on
  bool at_least_8;       // values in a row of the matrix
  uint32_t at[kEach];    // byte offset of a chunk, or kOutside
  u16x8_t reg[DIRECT ? 1 : kEach];

  // row of the matrix (m or k within the tile) and its chunk that a thread's i-th chunk holds
  __device__ __forceinline__ static void place(int i, int tid, int& row, int& chunk) {
    const int q = i * THREADS + tid;
    if constexpr (ALONG) {
      row = q / (K / 8);
      chunk = q % (K / 8) ^ along_pattern<GAP>(row);
    } else {
      const int u = q / 64, v = q % 64;  // load instruction, lane
      const int sub = v / (SIDE / 8);    // 2 g + h
      chunk = v % (SIDE / 8);
      row = 8 * ((u >> 2) * kTogether<SIDE> + (sub >> 1)) + 4 * (sub & 1) + (u & 3);
    }
  }
  // where a thread's i-th chunk lies in LDS, in elements: lane l's 8 l after lane 0's
  __device__ __forceinline__ static int lds_place(int i) {
    const int q = i * THREADS + threadIdx.x;
    return ALONG ? q * 8 : q / 64 * (512 + 16) + q % 64 * 8;
  }
  __device__ __forceinline__ void init(const uint16_t* p, int64_t stride, int m_left, int k_left, int row) {
    base = p;
    ld = stride;
    ms = m_left;
    ks = k_left;
    at_least_8 = row >= 8;
    const uint32_t pitch = static_cast<uint32_t>(stride) * 2;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      int row, chunk;
      place(i, threadIdx.x, row, chunk);
      const bool in = ALONG ? row < ms : chunk * 8 < ms;
      at[i] = in ? row * pitch + chunk * 16 : kOutside;
    }
  }
  // Steps whose loads need no look at the matrix's end: those with kFurther more k behind them (across,
  // a chunk at the edge reads up to 7 values on, of rows that are there, one value wide as they may be),
  // and none where a tile's byte offsets pass 2^31.
  static constexpr int kFurther = ALONG || DIRECT ? 0 : 7;
  __device__ __forceinline__ int whole_steps() const { return DIRECT || ld < (int64_t{1} << 21) ? max(ks - kFurther, 0) / K : 0; }
  // Starts the i-th load of step k0 (of kEach).  WHOLE: one of whole_steps().
  template <bool WHOLE>
  __device__ __forceinline__ void load(int i, int k0, uint16_t* s) {
    const uint16_t* p = base + (ALONG ? k0 : k0 * ld);
    const int left = ks - k0;
    int row, chunk;
    place(i, threadIdx.x, row, chunk);
    const bool near = ld < (int64_t{1} << 21);  // a tile's byte offsets stay below 2^31
    if constexpr (DIRECT) {
      const uint64_t u = reinterpret_cast<uint64_t>(p);
      const u32x4 r = {static_cast<uint32_t>(u), static_cast<uint32_t>(u >> 32) & 0xffffu, 0x7fffffffu, 0x00027000u};
      const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
      const int to = ALONG ? (i * THREADS + w * kWave) * 8 : (i * (THREADS / kWave) + w) * (512 + 16);
      uint32_t o = at[i];
      if (!WHOLE && left < K && (ALONG ? chunk * 8 : row) >= left) o = kOutside;
      load_to_lds(r, o, static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void*)(s + to))));
    } else if (WHOLE || left <= 0 || near) {
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p), 0, 0x7fffffff, 0x00027000);
      if (WHOLE || (near && left >= K + kFurther)) {
        // 16 bytes at any alignment; an across chunk at the edge brings m that are not stored
        reg[i] = __builtin_bit_cast(u16x8_t, __builtin_amdgcn_raw_buffer_load_b128(r, at[i], 0, 0));
      } else if (left <= 0) {
        reg[i] = u16x8_t{};
      } else {
        const int n = (ALONG ? row < ms : row < left) ? (ALONG ? left : ms) - chunk * 8 : 0;
        if (at_least_8) {
          // A row's last n < 8 values: its last 8, moved down.  Offsets count from 16 bytes before p, so that
          // a load may start there.
          const __amdgpu_buffer_rsrc_t before = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p - 8), 0, 0x7fffffff, 0x00027000);
          const int back = min(max(8 - n, 0), 7);  // values
          const uint32_t o = n > 0 ? at[i] + 16 - 2 * back : kOutside;
          const u32x4 x = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(before, o, 0, 0));
          uint64_t lo = x.x | static_cast<uint64_t>(x.y) << 32, hi = x.z | static_cast<uint64_t>(x.w) << 32;
          if (back >= 4) {
            lo = hi;
            hi = 0;
          }
          const int bits = 16 * (back & 3);
          lo = bits ? lo >> bits | hi << (64 - bits) : lo;
          hi >>= bits;
          const u32x4 y = {static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32)};
          reg[i] = __builtin_bit_cast(u16x8_t, y);
        } else {
          // rows of fewer than 8 values: one by one, what lies outside from an offset past the range
#pragma unroll
          for (int e = 0; e < 8; ++e)
            reg[i][e] = __builtin_amdgcn_raw_buffer_load_b16(r, e < n ? at[i] + 2 * e : kOutside, 0, 0);
        }
      }
    } else {
      Vec<uint16_t, 8> v;
      const int n = (ALONG ? row < ms : row < left) ? (ALONG ? left : ms) - chunk * 8 : 0;
      load_vec_part<uint16_t, 8>(p + row * ld + chunk * 8, n, v);
      __builtin_memcpy(&reg[i], v.e, 16);
    }
  }
  // Registers to LDS, where the loads went there: a thread's i-th chunk, or all of them.
  __device__ __forceinline__ void store(int i, uint16_t* s) { *reinterpret_cast<u16x8_t*>(s + lds_place(i)) = reg[i]; }
  __device__ __forceinline__ void store(uint16_t* s) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) store(i, s);
  }
  // This lane's place in a read of the 8 k from 8 (lane / 16) on of one m.  Along: of m itself.  Across:
  // m is the first of the 4 adjacent m that this lane reads for its 16 lanes; it gets the (lane %
  // 16)-th.  read() takes an m that is a multiple of 16 (or, along, of 4 within GAP) further.
  __device__ __forceinline__ static int read_place(int m) {
    const int l = lane_id(), g = l >> 4;
    return ALONG ? m * K + ((g ^ along_pattern<GAP>(m)) << 3) : across_place<SIDE>(8 * g + ((l & 15) >> 2)) + m;
  }
  // The place of the buffer's second 32 k.
  __device__ __forceinline__ static int second_half(int place) {
    return ALONG ? place ^ 32 : place + across_place<SIDE>(32);
  }
  __device__ __forceinline__ static u16x8_t read(const uint16_t* s, int m_further) {
    if constexpr (ALONG) {
      return *reinterpret_cast<const u16x8_t*>(s + m_further * K);
    } else {
      u16x8_t r;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const s16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(s + m_further + h * SIDE));
#pragma unroll
        for (int i = 0; i < 4; ++i) r[4 * h + i] = static_cast<uint16_t>(v[i]);
      }
      return r;
    }
  }
};

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

// Between a wave's LDS writes and its other lanes' reads of them, and before those places are written again: the LDS
// serves a wave's instructions in order, so nothing has to wait, but no access may move across.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A wave's results, MF x NF products, to rows `out` + m * pitch, of type S: through LDS, a few rows at a
// time, so that each row's bytes leave in whole cache lines.  STREAM: past the caches, where they would
// take the operands' place (1.07 GB of results of 131072 rows, inner 4096, outer 1024: backward by
// input 1.21 ms without, 1.03 ms with it, 0.96 ms with no results stored; streaming pieces of 32
// bytes straight from the registers, 1.40 ms).  `s`: this wave's part of LDS.
template <typename S, bool STREAM, int MF, int NF, int LEN, int BYTES, typename Value>
__device__ __forceinline__ void store_tile(S* out, int64_t pitch, int m_left, int n_left, char* s, Value value) {
  constexpr int kRow = NF * 16 * static_cast<int>(sizeof(S)), kPitch = kRow + 16;  // 16: the rows of a write in different banks
  constexpr int kFit = BYTES / (16 * kPitch);
  constexpr int R = kFit >= MF ? MF : kFit >= 4 ? 4 : kFit >= 2 ? 2 : 1;           // products of m at a time
  static_assert(kFit >= 1 && MF % R == 0, "16 rows fit");
  constexpr int kPer = 16 / static_cast<int>(sizeof(S)), kLanes = kRow / 16;       // values of 16 bytes, lanes of a row
  // rows that start on 16 bytes only: the pieces of others share their lines' ends
  const bool on_16 = pitch * static_cast<int64_t>(sizeof(S)) % 16 == 0 && !(reinterpret_cast<uintptr_t>(out) & 15);
  const int l = lane_id(), g = l >> 4;
#pragma unroll
  for (int i0 = 0; i0 < MF; i0 += R) {
#pragma unroll
    for (int i = i0; i < i0 + R; ++i) {
      char* p = s + (16 * (i - i0) + (l & 15)) * kPitch;
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        Vec<S, 4> v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v.e[e] = value(i, j, e);
        // products' n: 4 NF adjacent ones a lane (LEN > 4), or 4 of every 16
        __builtin_memcpy(p + (LEN > 4 ? g * LEN + 4 * j : 16 * j + 4 * g) * sizeof(S), v.e, 4 * sizeof(S));
      }
    }
    wave_order();
#pragma unroll
    for (int k = 0; k < 16 * R * kLanes / kWave; ++k) {
      const int m = k * (kWave / kLanes) + l / kLanes, n = (l % kLanes) * kPer;
      Vec<S, kPer> v;
      __builtin_memcpy(v.e, s + m * kPitch + n * sizeof(S), 16);
      if (16 * i0 + m >= m_left) continue;
      S* p = out + (16 * i0 + m) * pitch + n;
      if (STREAM && on_16 && n_left - n >= kPer) store_vec_stream<S, kPer>(p, v);
      else store_vec_part<S, kPer>(p, n_left - n, v);
    }
    wave_order();
  }
}

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
  uint16_t* const sa[2] = {reinterpret_cast<uint16_t*>(lds), reinterpret_cast<uint16_t*>(lds) + OA::kElems};
  uint16_t* const sb[2] = {sa[1] + OA::kElems, sa[1] + OA::kElems + OB::kElems};
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

  // this lane's place in a product's 16 m and 16 n
  const int a_place = OA::read_place(wm + (A_ALONG ? l & 15 : 4 * (l & 3)));
  const int b_place = OB::read_place(wn + (B_ALONG ? ((l & 15) >> 2) * (4 * NF) + (l & 3) : 4 * (l & 3)));
  const int a_half[2] = {a_place, OA::second_half(a_place)}, b_half[2] = {b_place, OB::second_half(b_place)};
  constexpr int kNext = B_ALONG ? 4 : 16;  // n from one product to the next
  const bool sums = OP == kBackwardWeight && a.grad_bias && n0 == 0 && wn == 0;
  f32x4 acc[MF][NF];
  float sum[OP == kBackwardWeight ? MF : 1];  // of this lane's values of A
#pragma unroll
  for (int i = 0; i < MF; ++i) {
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    if constexpr (OP == kBackwardWeight) sum[i] = 0.0f;
  }

  constexpr int kLoads = OA::kEach + OB::kEach;
  auto load = [&](int i, int step, uint16_t* pa, uint16_t* pb, auto whole) {
    constexpr bool WHOLE = decltype(whole)::value;
    if (i < OA::kEach) A.template load<WHOLE>(i, step * K, pa);
    else B.template load<WHOLE>(i - OA::kEach, step * K, pb);
  };
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
  constexpr std::false_type any{};
  // whole_steps: those whose loads are whole, without a look at the end or a branch; then the last ones
  auto walk = [&](auto step, int ahead) {
    const int whole_steps = min(min(A.whole_steps(), B.whole_steps()) - ahead, steps);
    int it = 0;
    for (; it < whole_steps; ++it) step(it, std::true_type{});
    for (; it < steps; ++it) step(it, any);
  };
  if constexpr (DIRECT) {
    // The operands of 32 k are in registers while those of the next 32 k are read from LDS, between the
    // products.  Two LDS buffers of 64 k each: when the second half of buffer `it` has been read by all
    // waves, the loads of it + 2 start there, also between the products, and have the products of 64
    // k to arrive.  Loads are started past the end too, with nothing in range.
    u16x8_t fa[2][MF], fb[2][NF];
    if (steps > 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) load(i, k, sa[k], sb[k], any);
      }
      wait_loads<kLoads>();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
#pragma unroll
      for (int j = 0; j < NF; ++j) fb[0][j] = OB::read(sb[0] + b_place, kNext * j);
#pragma unroll
      for (int i = 0; i < MF; ++i) fa[0][i] = OA::read(sa[0] + a_place, 16 * i);
    }
    walk([&](int it, auto whole) {
      const int cur = it & 1;
#pragma unroll
      for (int P = 0; P < 2; ++P) {  // the half in registers
        const int Q = 1 - P, from = P == 0 ? cur : cur ^ 1;
        if (P == 1) {
          wait_loads<0>();
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
        }
        const uint16_t *ra = sa[0] + from * OA::kElems + a_half[Q], *rb = sb[0] + from * OB::kElems + b_half[Q];
#pragma unroll
        for (int i = 0; i < MF; ++i) {
          fa[Q][i] = OA::read(ra, 16 * i);
#pragma unroll
          for (int j = i * NF / MF; j < (i + 1) * NF / MF; ++j) fb[Q][j] = OB::read(rb, kNext * j);
#pragma unroll
          for (int j = 0; j < NF; ++j) acc[i][j] = mfma16<DT>(fb[P][j], fa[P][i], acc[i][j]);
          if (P == 1) {
#pragma unroll
            for (int k = i * kLoads / MF; k < (i + 1) * kLoads / MF; ++k)
              load(k, it + 2, sa[0] + cur * OA::kElems, sb[0] + cur * OB::kElems, whole);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < MF; ++i) add_up(i, fa[P][i]);
      }
    }, 2);
  } else {
    // The registers that loads pass through are paid for by those of the operands: 16 m of A are read
    // two ahead of their products.  While the products of buffer `it` are taken, what was loaded for
    // it + 1 goes to the other buffer and the loads of it + 2 start.  One barrier a step, two products of m
    // before its end: what is left of buffer `it` is then in registers, and the next one is there.  (The
    // fragments of 32 k twice, as above, leave no room for 256 x 256: 60000 rows, 8 experts, 1777 x 1201
    // forward took 432 us with 256 x 128.  Here a few registers spill around the loop, none inside it.)
    constexpr int T2 = 2 * MF;
    u16x8_t fa[4], fb[2][NF];
    if (steps > 0) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) load(i, 0, nullptr, nullptr, any);
      A.store(sa[0]);
      B.store(sb[0]);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) load(i, 1, nullptr, nullptr, any);
      wait_loads<63>();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
#pragma unroll
      for (int j = 0; j < NF; ++j) fb[0][j] = OB::read(sb[0] + b_place, kNext * j);
#pragma unroll
      for (int i = 0; i < 2; ++i) fa[i] = OA::read(sa[0] + a_place, 16 * i);
    }
    walk([&](int it, auto whole) {
      const int cur = it & 1;
      uint16_t *ca = sa[0] + cur * OA::kElems, *cb = sb[0] + cur * OB::kElems;
      uint16_t *na = sa[0] + (cur ^ 1) * OA::kElems, *nb = sb[0] + (cur ^ 1) * OB::kElems;
#pragma unroll
      for (int t = 0; t < T2; ++t) {
        const int P = t / MF, i = t % MF, u = (t + 2) % T2;
        if (t == T2 - 2) {
          wait_loads<63>();
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
        }
        fa[(t + 2) % 4] = OA::read((t < T2 - 2 ? ca : na) + a_half[u / MF], 16 * (u % MF));
        if (P == 0) {
#pragma unroll
          for (int j = i * NF / MF; j < (i + 1) * NF / MF; ++j) fb[1][j] = OB::read(cb + b_half[1], kNext * j);
        } else if (t >= T2 - 2) {
#pragma unroll
          for (int j = (t - T2 + 2) * NF / 2; j < (t - T2 + 3) * NF / 2; ++j) fb[0][j] = OB::read(nb + b_half[0], kNext * j);
        }
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[i][j] = mfma16<DT>(fb[P][j], fa[t % 4], acc[i][j]);
        add_up(i, fa[t % 4]);
        if (t < T2 - 2) {
#pragma unroll
          for (int k = t * kLoads / (T2 - 2); k < (t + 1) * kLoads / (T2 - 2); ++k) {
            if (k < OA::kEach) A.store(k, na);
            else B.store(k - OA::kEach, nb);
            load(k, it + 2, nullptr, nullptr, whole);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }, 2);
  }
  wait_loads<0>();  // no load is under way when LDS takes the results
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");

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
