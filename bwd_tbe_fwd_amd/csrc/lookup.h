// Scaled lookup: what its kernels share, and the backward's sums (lookup.hip says how they are cut into shares).
#pragma once

#include "items.h"
#include "tower_device.h"

namespace tbe {

constexpr int kVec = 8;        // columns of a lane
constexpr int kWalk = 4;       // positions whose rows are summed while those of the next ones load
constexpr int kKeep = 32;      // positions of a row at most, less one, that a share takes over from the next one

// WHOLE: the width is whole vectors, kept as the words they were loaded as; else a lane has `left` columns of its vector.
template <int DT, bool WHOLE>
struct RowVec {
  using S = typename Fmt<DT>::S;
  static constexpr int kWords = kVec * static_cast<int>(sizeof(S)) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const S* p, int left) {
    if constexpr (WHOLE) {
#pragma unroll
      for (int k = 0; k < kWords; k += 4) __builtin_memcpy(&w[k], reinterpret_cast<const char*>(p) + 4 * k, 16);
    } else {
      Vec<S, kVec> v;
      load_vec_part<S, kVec>(p, left, v);
      __builtin_memcpy(w, v.e, sizeof(w));
    }
  }
  __device__ __forceinline__ float at(int e) const {
    if constexpr (DT == 0) return __uint_as_float(w[e]);
    else return Fmt<DT>::to_f(static_cast<uint16_t>(w[e / 2] >> (e % 2 * 16)));
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = 0;
  }
};
template <int DT, bool WHOLE>
__device__ __forceinline__ void store_row(typename Fmt<DT>::S* p, int left, const float (&x)[kVec], bool stream) {
  Vec<typename Fmt<DT>::S, kVec> v;
#pragma unroll
  for (int e = 0; e < kVec; ++e) v.e[e] = tower_from_f<DT>(x[e]);
  if (stream && (WHOLE || left >= kVec)) store_vec_stream<typename Fmt<DT>::S, kVec>(p, v);
  else if constexpr (WHOLE) store_vec_any<typename Fmt<DT>::S, kVec>(p, v);
  else store_vec_part<typename Fmt<DT>::S, kVec>(p, left, v);
}

// A launch's columns: blockIdx.y takes `cols` of them (a multiple of kVec), a group of G lanes a row of these.
struct Columns {
  int64_t width;
  int cols;
};

struct LookupGradArgs {
  int64_t items;
  const uint32_t* keys;      // sorted
  const uint32_t* pay;       // their positions
  const int32_t* n_sorted;
  const void* gy;
  int64_t gy_stride;
  float scale;
  void* grad;
  int64_t grad_stride;
  int32_t add;
  int32_t stream;            // overwriting, grad's rows start on 16 bytes
  int32_t share;             // length of a share
  int32_t shares;
  float* part;               // [shares][2][width]: the sum of a row that began before the share and ends in it, of one that
                             // goes on behind it
  int32_t* begun;            // [shares] of such a first row, the share in which it began; -1: none ends here
  int32_t* row;              // [shares] and which row it is
  Columns c;
};

// Lanes of this lane's group of G whose predicate holds, as bits 0 .. G - 1.
template <int G>
__device__ __forceinline__ uint64_t group_ballot(bool p) {
  const uint64_t b = __ballot(p);
  if constexpr (G == kWave) return b;
  else return (b >> (lane_id() / G * G)) & ((uint64_t{1} << G) - 1);
}

// First i of [lo, hi] with value(i) >= d for i < hi (value does not decrease): a group of lanes probes G places at a time.
template <int G, typename F>
__device__ __forceinline__ int64_t first_at_least(int64_t lo, int64_t hi, int64_t d, F value) {
  const int l = lane_id() % G;
  while (lo < hi) {
    const int64_t step = (hi - lo + G) / (G + 1);  // >= 1
    const int64_t i = lo + (l + 1) * step - 1;     // probes at lo + step - 1, lo + 2 step - 1, ...
    const bool below = i < hi && value(i) < d;
    const int n = __popcll(group_ballot<G>(below));  // the first n probes are below
    const int64_t from = lo + n * step;              // at most hi: probe n - 1 lies before hi
    if (n < G) hi = min(hi, from + step - 1);
    lo = from;
  }
  return lo;
}

// A cut of the merged sequence: positions before i and the ends of the rows before row lie before it.
struct Cut {
  int64_t i, row;
  bool split;  // row has positions on both sides
};
template <int G>
__device__ __forceinline__ Cut cut_at(const LookupGradArgs& a, int64_t n, int64_t d) {
  Cut c;
  const int64_t all = a.add ? n : n + a.items;
  if (d >= all) return Cut{n, a.items, false};
  if (a.add) {
    c.i = d;
    c.row = a.keys[d];
  } else {
    c.i = first_at_least<G>(max(int64_t{0}, d - a.items), min(n, d), d, [&](int64_t i) { return i + static_cast<int64_t>(a.keys[i]); });
    c.row = d - c.i;
  }
  c.split = false;
  if (c.i > 0 && a.keys[c.i - 1] == c.row) {
    // the row has begun: what is left of it, up to kKeep positions
    int more = 0;
    const int l = lane_id() % G;
#pragma unroll
    for (int k = 0; k < kKeep; k += G) {
      const int64_t i = c.i + k + l;
      more += __popcll(group_ballot<G>(k + l < kKeep && i < n && a.keys[i] == c.row));
    }
    if (more == kKeep) {
      c.split = true;
    } else {
      c.i += more;
      c.row += 1;
    }
  }
  return c;
}

// A group of G lanes walks a share, kWalk positions' rows summed while those of the next kWalk load.  Bound by memory: 131072
// ids, 131072 rows of 1024 bf16: 127 us, 4.0 TB/s, and the same with the ids in order; 1 M ids added to 2 M rows of 128 fp16: 110
// us, 3.9 TB/s (read twice and written once).  In fp32 a lane's 8 columns are two stores of 16 bytes 32 apart: 131072 rows of
// 1024 overwritten 316 us, 2.5 TB/s.
template <int YT, int WT, int G, bool ADD, bool WHOLE>
__global__ __launch_bounds__(kBlock) void lookup_sum_kernel(LookupGradArgs a) {
  using SY = typename Fmt<YT>::S;
  using SW = typename Fmt<WT>::S;
  constexpr int kGroups = kBlock / G;
  const int l = threadIdx.x % G;
  const int64_t share = static_cast<int64_t>(blockIdx.x) * kGroups + threadIdx.x / G;
  const int64_t n = *a.n_sorted;
  const int64_t d = share * a.share;
  // all lanes take part in the searches
  const Cut from = cut_at<G>(a, n, d), to = cut_at<G>(a, n, share + 1 < a.shares ? d + a.share : n + a.items);
  if (share >= a.shares) return;
  if (blockIdx.y == 0) {
    // a row that began earlier and ends here: the share that has its first position, whose place in the sequence is i + row, or
    // i (a share whose end was moved behind that place would not have split the row)
    int32_t begun = -1;
    if (from.split && !(to.split && to.row == from.row)) {
      const int64_t i = first_at_least<G>(0, n, from.row, [&](int64_t k) { return static_cast<int64_t>(a.keys[k]); });
      begun = static_cast<int32_t>((a.add ? i : i + from.row) / a.share);
    }
    if (l == 0) {
      a.begun[share] = begun;
      a.row[share] = static_cast<int32_t>(from.row);
    }
  }
  const int64_t c = static_cast<int64_t>(blockIdx.y) * a.c.cols + l * kVec;
  const int left = l * kVec < a.c.cols ? static_cast<int>(min(a.c.width - c, static_cast<int64_t>(kVec))) : 0;
  if (left <= 0) return;
  float acc[kVec];
#pragma unroll
  for (int e = 0; e < kVec; ++e) acc[e] = 0.0f;
  bool open = from.split;  // the row began in an earlier share
  auto keep = [&](int which) {
    Vec<float, kVec> v;
#pragma unroll
    for (int e = 0; e < kVec; ++e) v.e[e] = acc[e];
    float* p = a.part + (share * 2 + which) * a.c.width + c;
    if constexpr (WHOLE) store_vec_any<float, kVec>(p, v);
    else store_vec_part<float, kVec>(p, left, v);
  };
  // the row's sum is whole, or its last part; ADD: `old` is what it is added to
  auto finish = [&](int64_t row, const RowVec<WT, WHOLE>& old) {
    if (open) {
      keep(0);
      open = false;
    } else {
      float x[kVec];
#pragma unroll
      for (int e = 0; e < kVec; ++e) x[e] = ADD ? old.at(e) + acc[e] * a.scale : acc[e] * a.scale;
      store_row<WT, WHOLE>(static_cast<SW*>(a.grad) + row * a.grad_stride + c, left, x, a.stream);
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) acc[e] = 0.0f;
  };
  auto zeros = [&](int64_t row, int64_t end) {
    const float x[kVec] = {};
    for (; row < end; ++row) store_row<WT, WHOLE>(static_cast<SW*>(a.grad) + row * a.grad_stride + c, left, x, a.stream);
  };
  // kWalk positions: their ids and the id after each, their rows, and what the ids' rows hold where they end here
  struct Batch {
    uint32_t at[kWalk], key[kWalk + 1];
    RowVec<YT, WHOLE> row[kWalk];
    RowVec<WT, WHOLE> old[ADD ? kWalk : 1];
  };
  constexpr uint32_t kNone = ~0u;  // no id
  auto find = [&](Batch& b, int64_t i) {
#pragma unroll
    for (int u = 0; u < kWalk; ++u) {
      b.at[u] = i + u < to.i ? a.pay[i + u] : 0;
      b.key[u] = i + u < to.i ? a.keys[i + u] : kNone;
    }
    b.key[kWalk] = i + kWalk < to.i ? a.keys[i + kWalk] : kNone;
  };
  auto fetch = [&](Batch& b, int64_t i) {
#pragma unroll
    for (int u = 0; u < kWalk; ++u) {
      if (i + u < to.i) {
        b.row[u].load(static_cast<const SY*>(a.gy) + b.at[u] * a.gy_stride + c, left);
        if constexpr (ADD) {
          if (b.key[u] != b.key[u + 1]) b.old[u].load(static_cast<const SW*>(a.grad) + b.key[u] * a.grad_stride + c, left);
        }
      }
    }
  };
  int64_t row = from.row;      // overwriting: the row whose end comes next
  bool begun = from.split;     // it has positions already
  auto consume = [&](Batch& b, int64_t i) {
#pragma unroll
    for (int u = 0; u < kWalk; ++u) {
      if (i + u < to.i) {
        const int64_t k = b.key[u];
        if constexpr (!ADD) zeros(row, k);  // none where the row has begun
        row = k;
        begun = true;
#pragma unroll
        for (int e = 0; e < kVec; ++e) acc[e] += b.row[u].at(e);
        // the last of the row's positions here: a row that goes on behind the share is kept below
        if (b.key[u] != b.key[u + 1] && !(i + u + 1 == to.i && to.split && to.row == row)) {
          finish(row, b.old[ADD ? u : 0]);
          ++row;
          begun = false;
        }
      }
    }
  };
  Batch one, two;
  find(one, from.i);
  fetch(one, from.i);
  find(two, from.i + kWalk);
  for (int64_t i = from.i; i < to.i; i += 2 * kWalk) {
    fetch(two, i + kWalk);
    consume(one, i);
    find(one, i + 2 * kWalk);
    fetch(one, i + 2 * kWalk);
    consume(two, i + kWalk);
    find(two, i + 3 * kWalk);
  }
  if (begun) {
    if (to.split && to.row == row) {
      keep(1);
      return;
    }
    // overwriting, a row that began in an earlier share and has no more positions
    RowVec<WT, WHOLE> none;
    none.zero();
    finish(row, none);
    ++row;
  }
  if constexpr (!ADD) zeros(row, to.row);
}

// Defined in translation units of their own (lookup_sum_f32.hip and its siblings), by grad_y's type.  lanes: of a group.
template <int YT>
tbe_status launch_lookup_sum(const LookupGradArgs& a, int table_dtype, int lanes, dim3 grid, hipStream_t s);

template <typename F>
tbe_status by_type(int dt, F f) {
  if (dt == TBE_F32) return f(std::integral_constant<int, 0>{});
  if (dt == TBE_F16) return f(std::integral_constant<int, 1>{});
  return f(std::integral_constant<int, 2>{});
}
template <typename F>
tbe_status by_lanes(int lanes, F f) {
  if (lanes == 8) return f(std::integral_constant<int, 8>{});
  if (lanes == 16) return f(std::integral_constant<int, 16>{});
  if (lanes == 32) return f(std::integral_constant<int, 32>{});
  return f(std::integral_constant<int, 64>{});
}

template <int YT>
tbe_status lookup_sum(const LookupGradArgs& a, int table_dtype, int lanes, dim3 grid, hipStream_t s) {
  return by_type(table_dtype, [&](auto wt) {
    return by_lanes(lanes, [&](auto g) {
      constexpr int WT = decltype(wt)::value, G = decltype(g)::value;
      const bool whole = a.c.width % kVec == 0;
      auto kernel = a.add ? (whole ? lookup_sum_kernel<YT, WT, G, true, true> : lookup_sum_kernel<YT, WT, G, true, false>)
                          : (whole ? lookup_sum_kernel<YT, WT, G, false, true> : lookup_sum_kernel<YT, WT, G, false, false>);
      ProfScope ps("lookup_sum", s);
      hipLaunchKernelGGL(kernel, grid, dim3(kBlock), 0, s, a);
      return check_launch("lookup_sum");
    });
  });
}

}  // namespace tbe
