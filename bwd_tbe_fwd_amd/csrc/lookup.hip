// Scaled lookup of single rows and the table's dense gradient.  Declarations and the meaning of every argument are in
// include/tbe_items.h.
//
//   forward    y_i = s W[id_i]
//   backward   dW_v = s sum_{i: id_i = v} dy_i
//
// Both are bound by memory: the forward by n rows read and written, the backward by n rows read and the table's rows
// written (or, added to a gradient that is there, the touched rows read and written).
//
// The backward sorts the positions by id, stably, and walks the sorted positions once.  Overwriting, it walks the merged
// sequence of positions and of the rows' ends (row v's end follows its last position), so that one pass writes the sums and
// the zeros between them; adding, the positions alone.  That sequence is cut into shares of equal length, whatever the
// ids' popularity; a share finds its start by a search of d = i + key_i.  A row that a cut would split within its last 31
// positions stays with the share before, so most rows are summed and rounded where they are read; of the others each share
// leaves its sum in the workspace, and the share in which the row ends has them joined, in order.
#include "lookup.h"

namespace tbe {
namespace {

constexpr int kFlight = 4;       // forward: rows of a group of lanes whose loads are under way together
constexpr int kRankMost = 8192;  // ids that are sorted by counting, in one launch

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
struct LookupArgs {
  int64_t n, items;
  const void* table;
  int64_t table_stride;
  const void* ids;
  int32_t id64;
  float scale;
  void* y;
  int64_t y_stride;
  int32_t stream;  // y's rows start on 16 bytes
  Columns c;
};
__device__ __forceinline__ int64_t id_at(const void* ids, int id64, int64_t i) {
  return id64 ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
}

// A group of G lanes takes kFlight rows, a workgroup consecutive ones.  Bound by memory: 1 M ids, 128 columns fp16 to bf16, 0.1 of
// them padding: 83 us, 4.5 TB/s of the bytes that differ and 6.2 of all that are read and written (loads and stores of 16
// bytes, y past the caches).  Rows of y that do not start on 16 bytes go through the caches, which costs a third: 20011 ids, 1001
// columns fp32: 42 us, with y's rows 1004 apart 32, wherever the table's rows start.
template <int WT, int YT, int G, bool WHOLE>
__global__ __launch_bounds__(kBlock) void lookup_forward_kernel(LookupArgs a) {
  using S = typename Fmt<WT>::S;
  constexpr int kGroups = kBlock / G;
  const int g = threadIdx.x / G, l = threadIdx.x % G;
  const int64_t c = static_cast<int64_t>(blockIdx.y) * a.c.cols + l * kVec;
  const int left = l * kVec < a.c.cols ? static_cast<int>(min(a.c.width - c, static_cast<int64_t>(kVec))) : 0;
  if (left <= 0) return;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kGroups * kFlight) + g; i0 < a.n; i0 += static_cast<int64_t>(gridDim.x) * (kGroups * kFlight)) {
    int64_t id[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int64_t i = i0 + u * kGroups;
      id[u] = i < a.n ? id_at(a.ids, a.id64, i) : -1;
    }
    RowVec<WT, WHOLE> r[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      if (static_cast<uint64_t>(id[u]) < static_cast<uint64_t>(a.items))
        r[u].load(static_cast<const S*>(a.table) + id[u] * a.table_stride + c, left);
      else
        r[u].zero();
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int64_t i = i0 + u * kGroups;
      if (i >= a.n) break;
      const bool there = static_cast<uint64_t>(id[u]) < static_cast<uint64_t>(a.items);
      float x[kVec];
#pragma unroll
      for (int e = 0; e < kVec; ++e) x[e] = there ? r[u].at(e) * a.scale : 0.0f;  // 0, whatever the scale
      store_row<YT, WHOLE>(static_cast<typename Fmt<YT>::S*>(a.y) + i * a.y_stride + c, left, x, a.stream);
    }
  }
}

// ---------------------------------------------------------------------------
// backward: positions by id
// ---------------------------------------------------------------------------
// Keys of all ids (items: outside the table) and their positions, for the radix sort.
__global__ __launch_bounds__(kBlock) void lookup_keys_kernel(const void* ids, int id64, int64_t n, int64_t items,
                                                             uint32_t* __restrict__ keys, uint32_t* __restrict__ pay) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x;
  if (i >= n) return;
  const int64_t id = id_at(ids, id64, i);
  keys[i] = static_cast<uint32_t>(static_cast<uint64_t>(id) < static_cast<uint64_t>(items) ? id : items);
  pay[i] = static_cast<uint32_t>(i);
}

// Up to kRankMost ids: an id's place is the number of smaller ones and of equal ones before it.  A workgroup places 64 ids, each
// of its 16 waves counts a sixteenth of all of them.  One launch, where the radix sort takes seven to ten of 4 us and more: a
// call with 4096 ids added to rows of 64 columns takes 35 us (67 with 4 waves and two comparisons an id), 8190 48 (54 by the
// sort), 12000 57 (54).
constexpr int kRankWaves = 16;
__global__ __launch_bounds__(kRankWaves * kWave) void lookup_rank_kernel(const void* ids, int id64, int n, int64_t items,
                                                                         uint32_t* __restrict__ keys, uint32_t* __restrict__ pay,
                                                                         int32_t* __restrict__ n_sorted) {
  __shared__ __align__(16) uint32_t s_key[kRankMost];
  __shared__ int s_rank[kRankWaves][kWave];
  const int n4 = (n + 4 * kRankWaves - 1) / (4 * kRankWaves) * (4 * kRankWaves);  // a whole number of fours for each wave
  int valid = 0;
  for (int i = threadIdx.x; i < n4; i += kRankWaves * kWave) {
    const int64_t id = i < n ? id_at(ids, id64, i) : -1;
    const bool in = static_cast<uint64_t>(id) < static_cast<uint64_t>(items);
    s_key[i] = i < n ? static_cast<uint32_t>(in ? id : items) : ~0u;  // behind all others
    valid += in ? 1 : 0;
  }
  __syncthreads();
  const int w = threadIdx.x / kWave, l = lane_id();
  const int mine = blockIdx.x * kWave + l;
  const uint32_t k = mine < n ? s_key[mine] : ~0u;
  int rank = 0;
  const int part = n4 / kRankWaves;
#pragma unroll 2
  for (int j = w * part; j < (w + 1) * part; j += 4) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(s_key + j);
#pragma unroll
    for (int e = 0; e < 4; ++e) rank += v[e] < k + (j + e < mine ? 1u : 0u) ? 1 : 0;  // of the equal ones those before
  }
  s_rank[w][l] = rank;
  __syncthreads();
  if (w == 0 && mine < n) {
    rank = 0;
#pragma unroll
    for (int q = 0; q < kRankWaves; ++q) rank += s_rank[q][l];
    keys[rank] = k;
    pay[rank] = static_cast<uint32_t>(mine);
  }
  if (blockIdx.x) return;
  __syncthreads();
  for (int d = 1; d < kWave; d <<= 1) valid += __shfl_xor(valid, d);
  if (l == 0) s_rank[0][w] = valid;
  __syncthreads();
  if (threadIdx.x == 0) {
    int all = 0;
    for (int q = 0; q < kRankWaves; ++q) all += s_rank[0][q];
    *n_sorted = all;
  }
}

// ---------------------------------------------------------------------------
// backward: joins
// ---------------------------------------------------------------------------
// Joins the sums of the rows that several shares have parts of, 256 columns of a row at a time.  A workgroup looks at 16 shares
// for those in which such a row ends, a wave each, which adds up to kAlone parts by itself; where there are more all 16 waves
// add a contiguous part of them each, then the waves' sums are added in order.  (One row after the other by all waves took 55
// us with 1 M ids, 2 M rows of 128.)
constexpr int kAlone = 64;
template <int WT>
__global__ __launch_bounds__(1024) void lookup_join_kernel(LookupGradArgs a) {
  using SW = typename Fmt<WT>::S;
  constexpr int kWaves = 16, kCols = 4 * kWave;
  __shared__ __align__(16) float s_sum[kWaves][kCols];
  const int w = threadIdx.x / kWave, l = lane_id();
  const int64_t c = static_cast<int64_t>(blockIdx.y) * kCols + 4 * l;
  const int left = static_cast<int>(min(max(a.c.width - c, int64_t{0}), int64_t{4}));
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kWaves;
  const int32_t mine = l < kWaves && base + l < a.shares ? a.begun[base + l] : -1;
  // parts k of [lo, hi) of a row that ends in `share`: the shares' from `first` to the one before, then this one's
  auto add = [&](int64_t share, int64_t first, int64_t lo, int64_t hi) {
    f32x4 sum = {0, 0, 0, 0};
    if (left > 0) {
#pragma unroll 8
      for (int64_t k = lo; k < hi; ++k) {
        Vec<float, 4> v;
        load_vec_part<float, 4>(a.part + ((first + k) * 2 + (first + k < share ? 1 : 0)) * a.c.width + c, left, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += v.e[e];
      }
    }
    return sum;
  };
  auto finish = [&](int64_t share, f32x4 sum) {
    SW* p = static_cast<SW*>(a.grad) + a.row[share] * a.grad_stride + c;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (e < left) p[e] = tower_from_f<WT>(a.add ? Fmt<WT>::to_f(p[e]) + sum[e] * a.scale : sum[e] * a.scale);
    }
  };
  const bool alone = base + l - mine + 1 <= kAlone;
  const uint64_t few = __ballot(mine >= 0 && alone), many = __ballot(mine >= 0 && !alone);
  if (few >> w & 1) {
    const int64_t first = read_lane(mine, w);
    finish(base + w, add(base + w, first, 0, base + w - first + 1));
  }
  for (uint64_t found = many; found; found &= found - 1) {
    const int at = __ffsll(static_cast<unsigned long long>(found)) - 1;
    const int64_t share = base + at, first = read_lane(mine, at);
    const int64_t parts = share - first + 1, each = (parts + kWaves - 1) / kWaves;
    const int64_t lo = w * each < parts ? w * each : parts, hi = lo + each < parts ? lo + each : parts;
    f32x4 sum = add(share, first, lo, hi);
    *reinterpret_cast<f32x4*>(&s_sum[w][4 * l]) = sum;
    __syncthreads();
    if (w == 0 && left > 0) {
      for (int k = 1; k < kWaves; ++k) sum += *reinterpret_cast<const f32x4*>(&s_sum[k][4 * l]);
      finish(share, sum);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// Groups of 8 to 64 lanes, the fewest that hold a row; wider rows in equal parts.
struct Split {
  int lanes, parts;
  Columns c;
};
Split split_of(int64_t width) {
  Split s;
  s.lanes = width <= 8 * kVec ? 8 : width <= 16 * kVec ? 16 : width <= 32 * kVec ? 32 : 64;
  s.parts = static_cast<int>((width + kWave * kVec - 1) / (kWave * kVec));
  const int64_t vecs = (width + kVec - 1) / kVec;
  s.c = Columns{width, static_cast<int>((vecs + s.parts - 1) / s.parts) * kVec};
  return s;
}

// Length of a share, so that there are about kFewWaves waves (a group of lanes takes a share of a part of the columns), and how
// many shares there are at most for any sequence up to this length: a workspace serves every smaller batch.
constexpr int64_t kLeastShare = 16, kLongShare = 128, kFewWaves = 8192, kMostShares = 1 << 18;
int64_t share_of(int64_t all, const Split& s) {
  const int64_t even = all * s.lanes / kWave * s.parts / kFewWaves;
  return hmax((all + kMostShares - 1) / kMostShares, hmin(kLongShare, hmax(kLeastShare, even)));
}
int64_t shares_bound(int64_t all, const Split& s) {
  // even = k: all >= k * unit, so ceil(all / k) <= all / k + 1 < unit * (k + 1) / k + 2
  const int64_t unit = (kFewWaves * kWave + s.lanes * s.parts - 1) / (s.lanes * s.parts);
  const int64_t least = (all + kLeastShare - 1) / kLeastShare, few = unit + unit / kLeastShare + 2;
  return hmin(least, hmax(few, hmin(kMostShares, (all + kLongShare - 1) / kLongShare)));
}

// The workspace: sorted pairs twice, the sort's counts, the shares' sums.
struct LookupPlan {
  int64_t seg, shares;
  int nblocks, share;
  size_t keys[2], pay[2], hist, n_sorted, begun, row, part, total;
};
LookupPlan lookup_plan(int64_t n, int64_t items, int64_t width, bool add) {
  LookupPlan p = {};
  sort_segments(n, &p.seg, &p.nblocks);
  const int64_t all = add ? n : n + items, tiles = (n + kBlock * kRadixFewItems - 1) / (kBlock * kRadixFewItems);
  const Split sp = split_of(width);
  const int64_t bound = shares_bound(n + items, sp);
  p.share = static_cast<int>(share_of(all, sp));
  p.shares = (all + p.share - 1) / p.share;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  for (int i = 0; i < 2; ++i) {
    p.keys[i] = take(n * 4);
    p.pay[i] = take(n * 4);
  }
  p.hist = take(static_cast<size_t>(kRadixDigits) * (hmin(tiles, kMaxSortBlocks) + 1) * 4);
  p.n_sorted = take(4);
  p.begun = take(bound * 4);
  p.row = take(bound * 4);
  p.part = take(static_cast<size_t>(bound) * 2 * width * 4);
  p.total = at;
  return p;
}

}  // namespace

tbe_status launch_lookup_forward(int64_t n, int64_t items, int64_t width, const void* table, int64_t table_stride, int table_dtype,
                                 const void* ids, int id_type, float scale, void* y, int64_t y_stride, int y_dtype, hipStream_t s) {
  const Split sp = split_of(width);
  LookupArgs a = {};
  a.n = n; a.items = items; a.table = table; a.table_stride = table_stride; a.ids = ids; a.id64 = id_type == TBE_I64;
  a.scale = scale; a.y = y; a.y_stride = y_stride; a.c = sp.c;
  a.stream = rows_on_16(y, y_stride, y_dtype);
  return by_type(table_dtype, [&](auto wt) {
    return by_type(y_dtype, [&](auto yt) {
      return by_lanes(sp.lanes, [&](auto g) {
        constexpr int WT = decltype(wt)::value, YT = decltype(yt)::value, G = decltype(g)::value;
        // a launch has fewer than 2^32 threads
        const int64_t groups = hmin((n + kBlock / G * kFlight - 1) / (kBlock / G * kFlight), int64_t{1} << 23);
        auto kernel = width % kVec == 0 ? lookup_forward_kernel<WT, YT, G, true> : lookup_forward_kernel<WT, YT, G, false>;
        ProfScope ps("lookup_forward", s);
        hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(groups), sp.parts), dim3(kBlock), 0, s, a);
        return check_launch("lookup_forward");
      });
    });
  });
}

size_t lookup_backward_workspace(int64_t n, int64_t items, int64_t width) {
  return lookup_plan(n, items, width, false).total;
}

tbe_status launch_lookup_backward(int64_t n, int64_t items, int64_t width, const void* ids, int id_type, const void* gy,
                                  int64_t gy_stride, int y_dtype, float scale, void* grad, int64_t grad_stride, int table_dtype,
                                  bool add, void* workspace, hipStream_t s) {
  const LookupPlan p = lookup_plan(n, items, width, add);
  char* ws = static_cast<char*>(workspace);
  uint32_t* const keys[2] = {reinterpret_cast<uint32_t*>(ws + p.keys[0]), reinterpret_cast<uint32_t*>(ws + p.keys[1])};
  uint32_t* const pay[2] = {reinterpret_cast<uint32_t*>(ws + p.pay[0]), reinterpret_cast<uint32_t*>(ws + p.pay[1])};
  int32_t* n_sorted = reinterpret_cast<int32_t*>(ws + p.n_sorted);
  const int id64 = id_type == TBE_I64;
  int sorted = 0;
  tbe_status st;
  if (n == 0) {
    if ((st = launch_fill_i32(n_sorted, 0, 1, s))) return st;
  } else if (n <= kRankMost) {
    ProfScope ps("lookup_rank", s);
    hipLaunchKernelGGL(lookup_rank_kernel, dim3(static_cast<unsigned>((n + kWave - 1) / kWave)), dim3(kRankWaves * kWave), 0, s, ids, id64,
                       static_cast<int>(n), items, keys[0], pay[0], n_sorted);
    if ((st = check_launch("lookup_rank"))) return st;
  } else {
    {
      ProfScope ps("lookup_keys", s);
      hipLaunchKernelGGL(lookup_keys_kernel, dim3(static_cast<unsigned>((n + kBlock - 1) / kBlock)), dim3(kBlock), 0, s, ids, id64,
                         n, items, keys[0], pay[0]);
      if ((st = check_launch("lookup_keys"))) return st;
    }
    int bits = 1;  // of the largest id, items - 1: what is outside is left out before its digits count
    while (bits < 31 && ((items - 1) >> bits) != 0) ++bits;
    if ((st = launch_radix_sort(n, p.seg, p.nblocks, radix_plan(bits), keys, pay, reinterpret_cast<uint32_t*>(ws + p.hist), n_sorted,
                                static_cast<uint32_t>(items), &sorted, s)))
      return st;
  }
  const Split sp = split_of(width);
  LookupGradArgs a = {};
  a.items = items; a.keys = keys[sorted]; a.pay = pay[sorted]; a.n_sorted = n_sorted; a.gy = gy; a.gy_stride = gy_stride;
  a.scale = scale; a.grad = grad; a.grad_stride = grad_stride; a.add = add;
  a.stream = !add && rows_on_16(grad, grad_stride, table_dtype);
  a.share = p.share; a.shares = static_cast<int32_t>(p.shares); a.part = reinterpret_cast<float*>(ws + p.part); a.c = sp.c;
  a.begun = reinterpret_cast<int32_t*>(ws + p.begun); a.row = reinterpret_cast<int32_t*>(ws + p.row);
  const dim3 grid(static_cast<unsigned>((p.shares + kBlock / sp.lanes - 1) / (kBlock / sp.lanes)), sp.parts);
  st = y_dtype == TBE_F32   ? launch_lookup_sum<0>(a, table_dtype, sp.lanes, grid, s)
       : y_dtype == TBE_F16 ? launch_lookup_sum<1>(a, table_dtype, sp.lanes, grid, s)
                            : launch_lookup_sum<2>(a, table_dtype, sp.lanes, grid, s);
  // a row has kKeep positions at least on the far side of a cut that splits it
  if (st != TBE_OK || p.shares < 2 || n <= kKeep) return st;
  return by_type(table_dtype, [&](auto wt) {
    ProfScope ps("lookup_join", s);
    hipLaunchKernelGGL((lookup_join_kernel<decltype(wt)::value>),
                       dim3(static_cast<unsigned>((p.shares + 15) / 16), static_cast<unsigned>((width + 4 * kWave - 1) / (4 * kWave))), dim3(1024), 0, s, a);
    return check_launch("lookup_join");
  });
}

}  // namespace tbe
