// Softmax cross entropy over all items of a table: the rows that have a target, the joins of partial results, and the plan
// of a call.  The products are in cross_entropy_tile.h, a translation unit each.
#include "cross_entropy.h"

#include "grouped_linear.h"
#include "sort_common.h"

namespace tbe {
namespace {

// ---------------------------------------------------------------------------
// the rows that have a target
// ---------------------------------------------------------------------------
struct CeBatch {
  int64_t rows, items;
  const void* targets;
  int32_t target64;
  int32_t width, pitch;
  const uint16_t* x;
  int64_t x_stride;
  uint16_t* xc;            // x of the rows with a target side by side, rows of `pitch` (whole 16 bytes, zeros behind the width)
  int32_t flip;            // 0: as it is, 1: negated, 2: zeros
  int32_t* counts;         // many rows: of each 256, how many have a target
  float* tops;             // and their largest |grad_loss|
  int32_t* count;
  float* largest;
  int32_t* row;
  int32_t* target;
  const float* bias;       // NULL: none
  float* bias_over;        // narrow rows: the biases over the scale (0 without), -infinity up to a whole 64 items; else NULL
  float over;              // 1 / scale
  float most;              // what finite biases count as at most
  // forward
  const uint16_t* w;
  int64_t w_stride;
  float scale;
  float* picked;           // the target's logit
  float* loss;             // 0 for the rows without a target
  float* lse_out;
  // backward
  const float* grad_loss;
  const float* lse_in;
  int32_t* slot;           // of every row, -1: none
  float* lse;
  float* grad;
  uint16_t* xg;            // x times grad_loss over the largest; NULL: not asked for
  float* ref;              // narrow rows: -lse in powers of two (fp16: 15 more, kUnit), and grad_loss over the largest, with
  float* part;             // -infinity and 0 up to a whole 64 rows; NULL: not asked for
  float* weighed;          // ref and the factor's size in powers of two: the reference of probabilities times |part|
  float* far;              // lse where it is past kFar, else 0
};
__device__ __forceinline__ int target_of(const CeBatch& b, int64_t i) {
  if (i >= b.rows) return -1;
  const int64_t t = b.target64 ? static_cast<const int64_t*>(b.targets)[i] : static_cast<const int32_t*>(b.targets)[i];
  return static_cast<uint64_t>(t) < static_cast<uint64_t>(b.items) ? static_cast<int>(t) : -1;
}
__device__ __forceinline__ float block_max(float v, float* s_tmp) {
  for (int m = 1; m < kWave; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
  __syncthreads();
  if (lane_id() == 0) s_tmp[threadIdx.x >> 6] = v;
  __syncthreads();
  return fmaxf(fmaxf(s_tmp[0], s_tmp[1]), fmaxf(s_tmp[2], s_tmp[3]));
}

__global__ __launch_bounds__(kBlock) void ce_count_kernel(CeBatch b) {
  __shared__ uint32_t s_n[kWavesPerBlock];
  __shared__ float s_top[kWavesPerBlock];
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x;
  const bool has = target_of(b, i) >= 0;
  const uint32_t n = block_sum(has ? 1u : 0u, s_n);
  const float top = block_max(has && b.grad_loss ? fabsf(b.grad_loss[i]) : 0.0f, s_top);
  if (threadIdx.x == 0) {
    b.counts[blockIdx.x] = static_cast<int32_t>(n);
    b.tops[blockIdx.x] = top;
  }
}

// Weights whose rows do not start on 16 bytes, or are not whole 16 bytes: a piece's items at a pitch that is, zeros behind the
// width.  16 bytes a lane, rows one after the other; workgroup `block` of `blocks`.  213712 rows of 15: 11 us beside the batch's
// rows, where a wave a row took 37.
struct CePad {
  const uint16_t* from;
  int64_t stride;
  int32_t items, width, pitch;
  uint16_t* to;
};
__device__ __forceinline__ void ce_pad_rows(const CePad& p, unsigned block, unsigned blocks) {
  const unsigned each = p.pitch / 8, all = p.items * each;  // a piece's are fewer than 2^24
  for (unsigned k = block * kBlock + threadIdx.x; k < all; k += blocks * kBlock) {
    const unsigned v = k / each, d = k % each * 8;
    Vec<uint16_t, 8> x;
    load_vec_part<uint16_t, 8>(p.from + v * p.stride + d, p.width - static_cast<int>(d), x);
    store_vec_any<uint16_t, 8>(p.to + static_cast<int64_t>(k) * 8, x);
  }
}
__global__ __launch_bounds__(kBlock) void ce_pad_kernel(CePad p) { ce_pad_rows(p, blockIdx.x, gridDim.x); }

// Places the rows that have a target and copies what the products need of them.  A workgroup takes `each` rows (a multiple of
// kRowsAtOnce that 256 is a multiple of).  With `counted` it finds the rows before its own in ce_count_kernel's counts, else in
// the targets themselves: one launch for up to kCountHere rows.  `more` workgroups behind those of the rows take the biases of
// narrow rows, the ones behind them the copies of the first piece's weights.
constexpr int kRowsAtOnce = 4;  // a wave each
constexpr int64_t kCountHere = 4096;
template <int DT>
__global__ __launch_bounds__(kBlock) void ce_rows_kernel(CeBatch b, int each, int groups, int more, int counted, CePad pad) {
  __shared__ uint32_t s_n[kWavesPerBlock];
  __shared__ float s_top[kWavesPerBlock];
  __shared__ int s_target[kRowsAtOnce];
  __shared__ int s_slot[kRowsAtOnce];
  const int64_t first = static_cast<int64_t>(blockIdx.x) * each, end = min(first + each, b.rows);
  const int w = threadIdx.x >> 6, l = lane_id();
  if (static_cast<int>(blockIdx.x) >= groups + more) {
    ce_pad_rows(pad, blockIdx.x - (groups + more), gridDim.x - (groups + more));
    return;
  }
  if (static_cast<int>(blockIdx.x) >= groups) {
    // the biases' workgroups.  Finite ones stay finite: the lowest value is no mask where every item has it
    const int64_t end = (b.items + 63) / 64 * 64;
    for (int64_t v = static_cast<int64_t>(blockIdx.x - groups) * kBlock + threadIdx.x; v < end;
         v += static_cast<int64_t>(more) * kBlock) {
      b.bias_over[v] = ce_times(v >= b.items ? -kInfinity : b.bias ? ce_bias(b.bias[v], b.most) : 0.0f, b.over);
    }
    return;
  }
  uint32_t before = 0;
  float top = 0.0f;
  int64_t from = 0;
  if (counted) {
    const int64_t blocks = (b.rows + kBlock - 1) / kBlock, mine = first / kBlock;
    for (int64_t k = threadIdx.x; k < blocks; k += kBlock) {
      if (k < mine) before += b.counts[k];
      top = fmaxf(top, b.tops[k]);
    }
    from = mine * kBlock;
  }
  for (int64_t i = from + threadIdx.x; i < (counted || !b.grad_loss ? first : b.rows); i += kBlock) {
    const bool has = target_of(b, i) >= 0;
    if (has && i < first) ++before;
    if (has && !counted && b.grad_loss) top = fmaxf(top, fabsf(b.grad_loss[i]));
  }
  before = block_sum(before, s_n);
  top = block_max(top, s_top);
  for (int64_t i0 = first; i0 < end; i0 += kRowsAtOnce) {
    __syncthreads();
    if (w == 0) {
      const int64_t i = i0 + l;
      const int t = l < kRowsAtOnce ? target_of(b, i) : -1;
      const uint64_t has = __ballot(t >= 0);
      const int slot = t >= 0 ? static_cast<int>(before) + __popcll(has & lanemask_lt()) : -1;
      if (l < kRowsAtOnce) {
        s_target[l] = t;
        s_slot[l] = slot;
      }
      if (t >= 0) {
        b.row[slot] = static_cast<int32_t>(i);
        b.target[slot] = t;
        if (b.grad_loss) {
          const float lse = b.lse_in[i], grad = b.grad_loss[i];
          b.lse[slot] = lse;
          b.grad[slot] = grad;
          if (b.ref) {
            b.ref[slot] = ce_reference(lse, DT == 1 ? 15.0f : 0.0f);
            b.part[slot] = top > 0.0f ? grad / top : 0.0f * grad;
            b.weighed[slot] = b.ref[slot] + log2f(fabsf(b.part[slot]));
            b.far[slot] = ce_is_far(lse) ? lse : 0.0f;
          }
        }
      } else if (l < kRowsAtOnce && i < b.rows && b.loss) {
        b.loss[i] = 0.0f;
        b.lse_out[i] = 0.0f;
      }
      if (b.slot && l < kRowsAtOnce && i < b.rows) b.slot[i] = slot;
      if (l == 0) s_n[0] = static_cast<uint32_t>(__popcll(has));
    }
    __syncthreads();
    before += s_n[0];
    static_assert(kRowsAtOnce == kWavesPerBlock, "a row a wave");
    const int r = w, t = s_target[r], slot = s_slot[r];
    if (t >= 0) {
      const uint16_t* p = b.x + (i0 + r) * b.x_stride;
      const float g = b.xg ? (top > 0.0f ? b.grad_loss[i0 + r] / top : 0.0f * b.grad_loss[i0 + r]) : 1.0f;
      float dot = 0.0f;
      for (int d = l * 8; d < b.pitch; d += kWave * 8) {
        Vec<uint16_t, 8> v;
        load_vec_part<uint16_t, 8>(p + d, b.width - d, v);
        if (b.picked) {
          Vec<uint16_t, 8> u;
          load_vec_part<uint16_t, 8>(b.w + t * b.w_stride + d, b.width - d, u);
#pragma unroll
          for (int e = 0; e < 8; ++e) dot = fmaf(Fmt<DT>::to_f(v.e[e]), Fmt<DT>::to_f(u.e[e]), dot);
        }
        if (b.xg) {
          Vec<uint16_t, 8> u;
#pragma unroll
          for (int e = 0; e < 8; ++e) u.e[e] = tower_from_f<DT>(Fmt<DT>::to_f(v.e[e]) * g);
          store_vec_any<uint16_t, 8>(b.xg + static_cast<int64_t>(slot) * b.pitch + d, u);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v.e[e] = b.flip == 2 ? 0 : v.e[e] ^ (b.flip ? 0x8000 : 0);
        store_vec_any<uint16_t, 8>(b.xc + static_cast<int64_t>(slot) * b.pitch + d, v);
      }
      if (b.picked) {
        dot = lanes_sum<64>(dot);
        if (l == 0) b.picked[slot] = fmaf(dot, b.scale, b.bias ? ce_bias(b.bias[t], b.most) : 0.0f);
      }
    }
  }
  if (static_cast<int>(blockIdx.x) + 1 == groups) {
    const int more = static_cast<int>(before) + threadIdx.x;
    if (b.ref && more < (static_cast<int>(before) + 63) / 64 * 64) {
      b.ref[more] = -kInfinity;
      b.part[more] = 0.0f;
      b.weighed[more] = -kInfinity;
      b.far[more] = 0.0f;
      b.target[more] = -1;
    }
    if (threadIdx.x == 0) {
      *b.count = static_cast<int32_t>(before);
      *b.largest = top;
    }
  }
}

// ---------------------------------------------------------------------------
// joins
// ---------------------------------------------------------------------------
// A piece's maxima and sums of each row, its tiles in a fixed order, joined with the pieces before.  ROWS rows a workgroup of
// 1024 threads: 16, or 1 where there are few rows and many tiles.  The last piece's ends in the loss.
template <int ROWS>
__global__ __launch_bounds__(1024) void ce_join_kernel(const float2* __restrict__ part, int64_t rows, int tiles, float2* __restrict__ all, int first,
                                                       int last, CeBatch b) {
  constexpr int kGroups = 1024 / ROWS, kAhead = 8;
  __shared__ float2 s_all[kGroups][ROWS + (ROWS > 1 ? 1 : 0)];
  const int q = threadIdx.x / ROWS, k = threadIdx.x % ROWS, count = *b.count;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * ROWS + k;
  float2 sum = make_float2(-kInfinity, 0.0f);
  if (c < count) {
    for (int t = q; t < tiles; t += kAhead * kGroups) {
      float2 v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) v[u] = t + u * kGroups < tiles ? part[(t + u * kGroups) * rows + c] : make_float2(-kInfinity, 0.0f);
      float top = sum.x;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) top = fmaxf(top, v[u].x);
      const float from = top == -kInfinity ? 0.0f : top;
      float s = sum.y * expf(sum.x - from);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) s += v[u].y * expf(v[u].x - from);
      sum = make_float2(top, s);
    }
  }
  s_all[q][k] = sum;
  __syncthreads();
  for (int n = kGroups / 2; n > 0; n /= 2) {
    if (q < n) s_all[q][k] = ce_join(s_all[q][k], s_all[q + n][k]);
    __syncthreads();
  }
  if (q || c >= count) return;
  sum = s_all[0][k];
  if (!first) sum = ce_join(all[c], sum);
  if (!last) {
    all[c] = sum;
    return;
  }
  // no sum is left where every item is masked, or by the lowest value
  const float at = b.picked[c];
  float lse = sum.y == 0.0f ? sum.x : sum.x + logf(sum.y);
  // narrow rows that have only items whose biases over the scale are past the lowest value: these are not told apart, and lse is the
  // target's logit
  if (sum.y == 0.0f && lse <= b.most * -0.999999f && at < lse && at != -kInfinity) lse = at;
  const float loss = at == -kInfinity && !(lse != lse) ? kInfinity : lse - at;
  b.lse_out[b.row[c]] = lse;
  b.loss[b.row[c]] = loss < 0.0f ? 0.0f : loss;  // lse and the target's logit are rounded for themselves
}

// The rows' gradients: the parts' sums times scale * grad_loss; zero for a row without a target.
__device__ __forceinline__ f32x4 sum_parts(const float* p, int64_t stride, int n) {
  f32x4 all = {0, 0, 0, 0};
#pragma unroll 8
  for (int k = 0; k < n; ++k) all += load_f4(p + k * stride);
  return all;
}
template <int DT>
__global__ __launch_bounds__(kBlock) void ce_grad_x_kernel(const CeBatch b, const float* __restrict__ sum, int64_t pitch, int splits, int width, float factor,
                                                           uint16_t* __restrict__ gx, int64_t stride) {
  const int l = lane_id();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWavesPerBlock + (threadIdx.x >> 6); i < b.rows;
       i += static_cast<int64_t>(gridDim.x) * kWavesPerBlock) {
    const int64_t c = b.slot[i];
    const float g = c >= 0 ? b.grad[c] * factor : 0.0f;
    for (int d = l * 4; d < width; d += kWave * 4) {
      f32x4 all = {0, 0, 0, 0};
      if (c >= 0) all = sum_parts(sum + c * pitch + d, b.rows * pitch, splits);
      Vec<uint16_t, 4> out;
#pragma unroll
      for (int e = 0; e < 4; ++e) out.e[e] = c >= 0 ? tower_from_f<DT>(all[e] * g) : static_cast<uint16_t>(0);
      store_vec_part<uint16_t, 4>(gx + i * stride + d, width - d, out);
    }
  }
}

// The same for few rows with many parts: a workgroup a row, `lanes` lanes (a power of two) hold its columns, 4 each, and the
// groups of them a part each at a time.
template <int DT>
__global__ __launch_bounds__(1024) void ce_grad_x_each_kernel(const CeBatch b, const float* __restrict__ sum, int64_t pitch, int splits, int width, int lanes,
                                                              float factor, uint16_t* __restrict__ gx, int64_t stride) {
  __shared__ f32x4 s_sum[1024];
  const int q = threadIdx.x / lanes, d = threadIdx.x % lanes * 4, groups = 1024 / lanes;
  const int64_t i = blockIdx.x, c = b.slot[i];
  f32x4 all = {0, 0, 0, 0};
  if (c >= 0 && d < width && q < splits) all = sum_parts(sum + (q * b.rows + c) * pitch + d, groups * b.rows * pitch, (splits - q + groups - 1) / groups);
  s_sum[threadIdx.x] = all;
  __syncthreads();
  for (int n = groups / 2; n > 0; n /= 2) {
    if (q < n) s_sum[threadIdx.x] += s_sum[threadIdx.x + n * lanes];
    __syncthreads();
  }
  if (q || d >= width) return;
  const float g = c >= 0 ? b.grad[c] * factor : 0.0f;
  Vec<uint16_t, 4> out;
#pragma unroll
  for (int e = 0; e < 4; ++e) out.e[e] = c >= 0 ? tower_from_f<DT>(s_sum[threadIdx.x][e] * g) : static_cast<uint16_t>(0);
  store_vec_part<uint16_t, 4>(gx + i * stride + d, width - d, out);
}

// The weights' gradients of a piece whose rows were shared.
template <int DT>
__global__ __launch_bounds__(kBlock) void ce_grad_w_kernel(const float* __restrict__ sum, int64_t pitch, int splits, int items, int width, float scale,
                                                           const float* __restrict__ largest, uint16_t* __restrict__ gw, int64_t stride) {
  const float factor = scale * *largest;
  const int l = lane_id();
  for (int64_t v = static_cast<int64_t>(blockIdx.x) * kWavesPerBlock + (threadIdx.x >> 6); v < items;
       v += static_cast<int64_t>(gridDim.x) * kWavesPerBlock) {
    for (int d = l * 4; d < width; d += kWave * 4) {
      const f32x4 all = sum_parts(sum + v * pitch + d, items * pitch, splits);
      Vec<uint16_t, 4> out;
#pragma unroll
      for (int e = 0; e < 4; ++e) out.e[e] = tower_from_f<DT>(all[e] * factor);
      store_vec_part<uint16_t, 4>(gw + v * stride + d, width - d, out);
    }
  }
}

// A piece's bias gradients: the sums over its parts, in order.  The parts are tiles of bm rows, or `parts` of them where bm is 0,
// which then count in the largest |grad_loss| times `factor`.  64 items a workgroup, 16 groups.
__global__ __launch_bounds__(1024) void ce_grad_bias_kernel(const float* __restrict__ part, int64_t stride, CeBatch b, int bm, int parts,
                                                            float factor, int items, float* __restrict__ gb) {
  __shared__ float s_sum[16][kWave];
  const int q = threadIdx.x / kWave, l = lane_id(), tiles = bm ? (*b.count + bm - 1) / bm : parts;
  for (int64_t v0 = static_cast<int64_t>(blockIdx.x) * kWave; v0 < items; v0 += static_cast<int64_t>(gridDim.x) * kWave) {
    const int64_t v = v0 + l;
    float sum = 0.0f;
    if (v < items) {
#pragma unroll 4
      for (int t = q; t < tiles; t += 16) sum += part[t * stride + v];
    }
    __syncthreads();
    s_sum[q][l] = sum;
    __syncthreads();
    if (q || v >= items) continue;
    for (int k = 1; k < 16; ++k) sum += s_sum[k][l];
    gb[v] = bm ? sum : sum * (factor * *b.largest);
  }
}

// ---------------------------------------------------------------------------
// the plan, from sizes alone
// ---------------------------------------------------------------------------
// Bytes below never shrink with the rows, so a workspace for the largest batch serves every smaller one.
constexpr int64_t kPartBytes = int64_t{64} << 20;    // forward: of the rows' maxima and sums over a piece's tiles
constexpr int64_t kZElems = int64_t{1} << 27;        // backward: of z
constexpr int64_t kLeastPiece = 1024, kMostPiece = 131072;  // items of a piece, backward
// Of a piece's weights, copied: read again from the caches.  At least the first, and up to the second where the workspace has no
// more than its share without them (few rows, whose small pieces would leave CUs idle: 439 rows, 543790 items of 1363 backward
// 5.0 -> 3.7 ms).
constexpr int64_t kCopyBytes = int64_t{32} << 20, kCopyMost = int64_t{128} << 20;
constexpr int64_t kForwardShare = int64_t{110} << 20, kBackwardShare = int64_t{600} << 20;
constexpr int64_t kSumBytes = int64_t{128} << 20;    // of the sums over shares of k, beyond one share of x's gradient
constexpr int kMostSplits = 64;
// Of the items, for the gradient of so few narrow rows that their sums are joined by a workgroup each (17 rows, 693510 items of
// 13: 245 us with 64 shares, 76 with up to 512; 64 rows of 1000, 64 shares: 20 us by waves, 7 by workgroups).
constexpr int kMostFew = 512;
constexpr int64_t kFewRows = 1024;

// Rows of up to so many columns stay in registers (cross_entropy_narrow.h).
constexpr int64_t kNarrowWidth = 128;

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

struct Carve {
  size_t at = 0;
  size_t take(int64_t bytes) {
    const size_t here = at;
    at += static_cast<size_t>(up(hmax(bytes, 1), 256));
    return here;
  }
};
struct CeLayout {
  int64_t pitch, piece, copied;  // items of a piece, and of a piece whose weights are copied
  size_t counts, tops, count, largest, row, target, slot, lse, grad, xc, wc;
  size_t bias_over;                         // narrow rows
  size_t part, picked, all;                 // forward
  size_t xg, z, sum_x, sum_w, bias_part;    // backward
  size_t ref, part_of, weighed, far;        // backward, narrow rows
  size_t total;
};
// The last to be carved.  Bytes never shrink with the rows here either: max(others + 32 MB, min(others + 128 MB, share)), or what
// all items or kLeastPiece of them take.
void carve_copies(CeLayout& L, Carve& c, int64_t items, int64_t share) {
  const int64_t most = hmax(kCopyBytes, hmin(kCopyMost, share - static_cast<int64_t>(c.at)));
  // whether it is asked for depends on addresses and strides
  const int64_t all = up(items, 256), row = 2 * L.pitch;
  L.copied = hmin(all, hmax(kLeastPiece, most / row / 256 * 256));
  L.wc = c.take(hmax(hmin(most, all * row), hmin(all, kLeastPiece) * row));
  L.total = c.at;
}
void carve_rows(CeLayout& L, Carve& c, int64_t rows, int64_t items, int64_t width) {
  const int64_t blocks = (rows + kBlock - 1) / kBlock;
  L.pitch = up(width, 8);
  L.counts = c.take(blocks * 4);
  L.tops = c.take(blocks * 4);
  L.count = c.take(4);
  L.largest = c.take(4);
  L.row = c.take(rows * 4);
  L.target = c.take(up(rows, 64) * 4);
  L.xc = c.take(rows * L.pitch * 2);
  L.bias_over = c.take(width <= kNarrowWidth ? up(items, 64) * 4 : 0);
}
CeLayout forward_layout(int64_t rows, int64_t items, int64_t width) {
  CeLayout L = {};
  Carve c;
  carve_rows(L, c, rows, items, width);
  // pieces of whole 256s; the smallest tile has 64 items
  L.piece = hmin(up(items, 256), hmax(1, kPartBytes / (8 * hmax(rows, 1)) / 4) * 256);
  L.part = c.take(hmin(rows * (up(items, 256) / 64) * 8, hmax(kPartBytes, rows * 4 * 8)));
  L.picked = c.take(rows * 4);
  L.all = c.take(rows * 8);
  carve_copies(L, c, items, kForwardShare);
  return L;
}
int64_t sum_x_bytes(int64_t rows, int64_t width) {
  const int64_t one = rows * up(width, 4) * 4;
  return hmax(one, hmin(kSumBytes, (width <= kNarrowWidth ? kMostFew : kMostSplits) * one));
}
CeLayout backward_layout(int64_t rows, int64_t items, int64_t width) {
  CeLayout L = {};
  Carve c;
  carve_rows(L, c, rows, items, width);
  L.slot = c.take(rows * 4);
  L.lse = c.take(rows * 4);
  L.grad = c.take(rows * 4);
  L.xg = c.take(rows * L.pitch * 2);
  const int64_t all = up(items, 256), most = hmin(all, kMostPiece);
  L.piece = hmin(most, hmax(kLeastPiece, kZElems / hmax(rows, 1) / 256 * 256));
  const int64_t z = hmin(rows * most, hmax(kZElems, rows * kLeastPiece));
  const bool narrow = width <= kNarrowWidth;
  L.z = c.take(narrow ? 0 : (z + 64 * most) * 2);  // panels of whole 64 rows
  L.sum_x = c.take(sum_x_bytes(rows, width));
  L.sum_w = c.take(kSumBytes);
  // of 64 rows a part; of narrow rows fused_splits of them, which are one or fit kSumBytes with 16 bytes a sum
  L.bias_part = c.take(narrow ? items * 4 + kSumBytes / 4 : z / 64 * 4 + most * 4);
  L.ref = c.take(up(rows, 64) * 4);
  L.part_of = c.take(up(rows, 64) * 4);
  L.weighed = c.take(up(rows, 64) * 4);
  L.far = c.take(up(rows, 64) * 4);
  carve_copies(L, c, items, kBackwardShare);
  return L;
}

// The tile of least expected time for m x n of C, k deep, and into how many shares k goes where few tiles leave CUs idle.
struct TilePick {
  int tile, splits;
};
// What sharing costs: the weights' sums are written, read and added by another kernel, the rows' are there anyway, once.
double weight_shares_us(int split, double bytes) { return 4.0 + 2.0 * split * bytes / 4e6; }
double x_shares_us(int split, double bytes) { return 2.0 * (split - 1) * bytes / 6e6; }
template <int N>
TilePick pick_tile(const TileCost (&costs)[N], int64_t m, int64_t n, int64_t k, int most_splits, int64_t most_bytes,
                   double (*shares_us)(int, double)) {
  TilePick best = {0, 1};
  double least = -1.0;
  for (int t = 0; t < N; ++t) {
    const TileCost& c = costs[t];
    const double tiles = static_cast<double>(((m + c.bm - 1) / c.bm) * ((n + c.bn - 1) / c.bn));
    for (int split = 1; split <= most_splits; split *= 2) {
      if (split > 1 && (k / split < 256 || split * m * n * 4 > most_bytes)) break;
      const double kk = static_cast<double>(up((k + split - 1) / split, 64));
      const double us = tiles_us(c, tiles * split, kk, kk) + (split > 1 ? shares_us(split, static_cast<double>(m * n) * 4) : 0.0);
      if (least < 0.0 || us < least) {
        least = us;
        best = TilePick{t, split};
      }
    }
  }
  return best;
}
// Logits: of few rows the weights' bytes decide, and 64 x 256 reads the rows a quarter as often as 64 x 64 (64 rows, 131072 items of
// 1000, backward: 65 and 81 us; 64 rows, 400000 items of 1000, forward: 184 and 219; 300 rows, 131072 items of 1024, forward: 107,
// and 111 with 128 x 128).
constexpr TileCost kLogits[4] = {kDirectTiles[0], kDirectTiles[1], kDirectTiles[2], {64, 256, 256, 512, 4.0, 0.95, 0.95}};
// The gradient of x: a tile more.  Its shares' sums go on from piece to piece, whether there is one share or several.
constexpr TileCost kGradX[4] = {kDirectTiles[0], kDirectTiles[1], kDirectTiles[2], {256, 128, 512, 256, 5.0, 0.8, 0.8}};

// Into how many ranges their items go: about 2048 workgroups, of 16 tiles of 64 items at least, of fewer where that leaves
// CUs idle.
int narrow_splits(int64_t rows, int64_t items, bool few) {
  const int64_t row_tiles = few ? 1 : (rows + 255) / 256, tiles = (items + 63) / 64;
  return static_cast<int>(hmax(1, hmin(tiles, hmin(2048 / row_tiles, hmax(tiles / 16, 512 / row_tiles)))));
}

// Into how many shares the passing side of the fused kernels goes.  The fullest CU's workgroups count, two at a time in the time
// of a pair, one alone in 0.7 of it; four tiles a share at least.  A share more costs its sums, which are written, read and added.
int fused_splits(int64_t stay_tiles, int64_t pass, double pair_us, double share_bytes, int64_t most) {
  const int64_t tiles = (pass + 63) / 64, end = hmax(1, hmin(tiles / 4, most));
  int best = 1;
  double least = -1.0;
  for (int n = 1; n <= end; ++n) {
    const int64_t a_cu = (stay_tiles * n + 255) / 256;
    const double pairs = static_cast<double>(a_cu / 2) + (a_cu % 2 ? 0.7 : 0.0);
    const double us = pairs * static_cast<double>((tiles + n - 1) / n + 4) * pair_us + (n > 1 ? 2.0 * n * share_bytes / 4e6 : 0.0);
    if (least < 0.0 || us < least) {
      least = us;
      best = n;
    }
  }
  return best;
}

bool whole_16(const void* p, int64_t stride, int64_t width) {
  return !(reinterpret_cast<uintptr_t>(p) & 15) && stride % 8 == 0 && width % 8 == 0 && stride < (int64_t{1} << 21);
}

// Forward, rows of up to so many go without a copy of the weights (kTile64 through registers): 123 rows, 110262 items of 861: 68
// us, and 113 with copies; 250 rows 120 and 134; 500 rows 226 and 190.
constexpr int64_t kRegisterRows = 256;

// One CeBatch for both directions.  A negative scale of narrow rows goes into x (their kernel looks for the largest product),
// and so does 0, by which no bias can be divided.
CeBatch batch_of(char* ws, const CeLayout& L, int64_t rows, int64_t items, int64_t width, const void* x, int64_t x_stride,
                 const void* targets, int target_type, const float* bias, bool narrow, float& scale) {
  CeBatch b = {};
  b.rows = rows; b.items = items; b.targets = targets; b.target64 = target_type == TBE_I64;
  b.width = static_cast<int>(width); b.pitch = static_cast<int>(L.pitch);
  b.x = static_cast<const uint16_t*>(x); b.x_stride = x_stride; b.xc = reinterpret_cast<uint16_t*>(ws + L.xc);
  b.counts = reinterpret_cast<int32_t*>(ws + L.counts);
  b.tops = reinterpret_cast<float*>(ws + L.tops);
  b.count = reinterpret_cast<int32_t*>(ws + L.count);
  b.largest = reinterpret_cast<float*>(ws + L.largest);
  b.row = reinterpret_cast<int32_t*>(ws + L.row);
  b.target = reinterpret_cast<int32_t*>(ws + L.target);
  b.bias = bias;
  b.scale = scale;
  const float size = scale < 0.0f ? -scale : scale == 0.0f ? 1.0f : scale;
  b.most = size < 1.0f ? kLargest * size : kLargest;
  if (narrow) {
    b.flip = scale < 0.0f ? 1 : scale == 0.0f ? 2 : 0;
    scale = size;
    b.bias_over = reinterpret_cast<float*>(ws + L.bias_over);
    b.over = 1.0f / scale;
  }
  return b;
}
int pad_groups(const CePad& p) { return static_cast<int>(hmin((static_cast<int64_t>(p.items) * (p.pitch / 8) + kBlock - 1) / kBlock, 16384)); }
tbe_status launch_rows(const CeBatch& b, int dtype, const CePad& pad, hipStream_t s) {
  const bool counted = b.rows > kCountHere;
  ProfScope ps("ce_rows", s);
  if (counted) {
    hipLaunchKernelGGL(ce_count_kernel, dim3(static_cast<unsigned>((b.rows + kBlock - 1) / kBlock)), dim3(kBlock), 0, s, b);
    if (tbe_status st = check_launch("ce_count")) return st;
  }
  const int each = b.rows > (1 << 17) ? kBlock : b.rows > (1 << 15) ? 32 : kRowsAtOnce;
  const int groups = static_cast<int>(hmax(1, (b.rows + each - 1) / each));  // no rows: their count, 0
  const int more = b.bias_over ? static_cast<int>(hmin(2048, (b.items + 4 * kBlock - 1) / (4 * kBlock))) : 0;
  auto kernel = dtype == TBE_F16 ? ce_rows_kernel<1> : ce_rows_kernel<2>;
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(groups + more + pad_groups(pad))), dim3(kBlock), 0, s, b, each, groups, more,
                     counted ? 1 : 0, pad);
  return check_launch("ce_rows");
}
tbe_status launch_grad_w_sum(const CeArgs& a, bool f16, const float* largest, hipStream_t s) {
  ProfScope ps("ce_grad_w_sum", s);
  auto kernel = f16 ? ce_grad_w_kernel<1> : ce_grad_w_kernel<2>;
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(hmin((a.items + 3) / 4, 8192))), dim3(kBlock), 0, s, a.sum, a.sum_pitch, a.splits,
                     a.items, a.out_width, a.factor, largest, static_cast<uint16_t*>(a.out), a.out_stride);
  return check_launch("ce_grad_w_sum");
}
// A piece's weights into the workspace: the first one's beside the rows.
CePad pad_of(const void* weight, int64_t stride, int64_t items, int64_t width, char* ws, const CeLayout& L) {
  return CePad{static_cast<const uint16_t*>(weight), stride, static_cast<int32_t>(items), static_cast<int32_t>(width), static_cast<int32_t>(L.pitch),
               reinterpret_cast<uint16_t*>(ws + L.wc)};
}
tbe_status launch_pad(const CePad& p, hipStream_t s) {
  ProfScope ps("ce_pad", s);
  hipLaunchKernelGGL(ce_pad_kernel, dim3(static_cast<unsigned>(pad_groups(p))), dim3(kBlock), 0, s, p);
  return check_launch("ce_pad");
}
CeRows rows_of(const CeBatch& b) { return CeRows{b.count, b.row, b.target, b.lse, b.grad, b.largest, b.ref, b.part, b.far}; }

}  // namespace

size_t cross_entropy_forward_workspace(int64_t rows, int64_t items, int64_t width) { return forward_layout(rows, items, width).total; }
size_t cross_entropy_backward_workspace(int64_t rows, int64_t items, int64_t width) { return backward_layout(rows, items, width).total; }

tbe_status launch_cross_entropy_forward(int64_t rows, int64_t items, int64_t width, const void* x, int64_t x_stride, const void* weight,
                                        int64_t weight_stride, int dtype, const float* bias, const void* targets, int target_type,
                                        float scale, float* loss, float* lse, void* workspace, hipStream_t s) {
  const CeLayout L = forward_layout(rows, items, width);
  char* ws = static_cast<char*>(workspace);
  const bool narrow = width <= kNarrowWidth, few = rows <= 64, f16 = dtype == TBE_F16;
  const bool on_16 = whole_16(weight, weight_stride, width), copy = !on_16 && (narrow || rows > kRegisterRows), direct = on_16 || copy;
  CeBatch b = batch_of(ws, L, rows, items, width, x, x_stride, targets, target_type, bias, narrow, scale);
  b.w = static_cast<const uint16_t*>(weight); b.w_stride = weight_stride;
  b.picked = reinterpret_cast<float*>(ws + L.picked);
  b.loss = loss;
  b.lse_out = lse;
  const int64_t piece = hmin(narrow ? items : L.piece, copy ? L.copied : items);
  tbe_status st = launch_rows(b, dtype, copy ? pad_of(weight, weight_stride, hmin(piece, items), width, ws, L) : CePad{}, s);
  if (b.bias_over) bias = b.bias_over;
  CeArgs a = {};
  a.rows = rows; a.width = static_cast<int>(direct ? L.pitch : width); a.out_width = static_cast<int>(width);
  a.x = ws + L.xc; a.x_stride = L.pitch;
  a.scale = scale; a.over = b.over; a.most = b.most; a.r = rows_of(b);
  a.part = reinterpret_cast<float2*>(ws + L.part);
  for (int64_t first = 0; st == TBE_OK && first < items; first += piece) {
    a.first = static_cast<int>(first);
    a.items = static_cast<int>(hmin(piece, items - first));
    a.w = static_cast<const uint16_t*>(weight) + first * weight_stride;
    a.w_stride = weight_stride;
    a.bias = bias ? bias + first : nullptr;
    if (copy) {
      if (first > 0) st = launch_pad(pad_of(a.w, weight_stride, a.items, width, ws, L), s);
      a.w = ws + L.wc;
      a.w_stride = L.pitch;
    }
    if (st != TBE_OK) break;
    int parts;  // of a row
    if (narrow) {
      parts = a.splits = narrow_splits(rows, a.items, few);
      st = f16 ? ce_launch_narrow_forward<1>(a, few, s) : ce_launch_narrow_forward<2>(a, few, s);
    } else {
      const int tile = direct ? pick_tile(kLogits, rows, a.items, width, 1, 0, weight_shares_us).tile : kTile64;
      parts = (a.items + kLogits[tile].bn - 1) / kLogits[tile].bn;
      st = f16 ? ce_launch_forward<1>(a, tile, direct, s) : ce_launch_forward<2>(a, tile, direct, s);
    }
    if (st != TBE_OK) break;
    ProfScope ps("ce_join", s);
    const bool each = rows <= 256 && parts >= 128;  // a workgroup for each row
    auto join = each ? ce_join_kernel<1> : ce_join_kernel<16>;
    hipLaunchKernelGGL(join, dim3(static_cast<unsigned>(each ? rows : (rows + 15) / 16)), dim3(1024), 0, s, a.part, rows, parts,
                       reinterpret_cast<float2*>(ws + L.all), first == 0 ? 1 : 0, first + piece >= items ? 1 : 0, b);
    st = check_launch("ce_join");
  }
  return st;
}

tbe_status launch_cross_entropy_backward(int64_t rows, int64_t items, int64_t width, const void* x, int64_t x_stride, const void* weight,
                                         int64_t weight_stride, int dtype, const float* bias, const void* targets, int target_type,
                                         float scale, const float* lse, const float* grad_loss, void* grad_x, int64_t grad_x_stride,
                                         void* grad_weight, int64_t grad_weight_stride, float* grad_bias, void* workspace, hipStream_t s) {
  const CeLayout L = backward_layout(rows, items, width);
  char* ws = static_cast<char*>(workspace);
  const bool narrow = width <= kNarrowWidth, f16 = dtype == TBE_F16, copy = !whole_16(weight, weight_stride, width);
  const float unit = f16 ? kUnit<1> : kUnit<2>, x_factor = scale / unit;
  CeBatch b = batch_of(ws, L, rows, items, width, x, x_stride, targets, target_type, bias, narrow, scale);
  b.grad_loss = grad_loss;
  b.lse_in = lse;
  b.slot = reinterpret_cast<int32_t*>(ws + L.slot);
  b.lse = reinterpret_cast<float*>(ws + L.lse);
  b.grad = reinterpret_cast<float*>(ws + L.grad);
  b.xg = grad_weight && !narrow ? reinterpret_cast<uint16_t*>(ws + L.xg) : nullptr;
  if (narrow) {
    b.ref = reinterpret_cast<float*>(ws + L.ref);
    b.part = reinterpret_cast<float*>(ws + L.part_of);
    b.weighed = reinterpret_cast<float*>(ws + L.weighed);
    b.far = reinterpret_cast<float*>(ws + L.far);
  }
  const int64_t piece = hmin(narrow ? items : L.piece, copy ? L.copied : items);
  tbe_status st = launch_rows(b, dtype, copy ? pad_of(weight, weight_stride, hmin(piece, items), width, ws, L) : CePad{}, s);
  if (b.bias_over) bias = b.bias_over;
  CeArgs a = {};
  a.rows = rows; a.width = static_cast<int>(L.pitch); a.out_width = static_cast<int>(width);
  a.x = ws + L.xc; a.x_stride = L.pitch; a.xg = ws + L.xg;
  a.scale = scale; a.over = b.over; a.most = b.most; a.r = rows_of(b);
  a.z = reinterpret_cast<uint16_t*>(ws + L.z); a.panel = up(rows, 64) * 64;
  a.factor = scale / unit;  // of x as it was copied
  a.sum_pitch = up(width, 4);
  float* const bias_part = reinterpret_cast<float*>(ws + L.bias_part);
  if (rows == 0) grad_x = nullptr;  // the gradients of the weights and biases are zeros
  const int64_t stay = width <= 64 ? 256 : 192;  // narrow: rows or items of a workgroup
  const double pair_us = width <= 64 ? 2.6 : 3.0;                // of two workgroups with a tile each
  TilePick x_pick = {0, 1};
  for (int64_t first = 0; st == TBE_OK && first < items; first += piece) {
    a.first = static_cast<int>(first);
    a.items = static_cast<int>(hmin(piece, items - first));
    a.bias_stride = a.items;
    a.w = static_cast<const uint16_t*>(weight) + first * weight_stride;
    a.w_stride = weight_stride;
    a.bias = bias ? bias + first : nullptr;
    if (copy) {
      if (first > 0) st = launch_pad(pad_of(a.w, weight_stride, a.items, width, ws, L), s);
      a.w = ws + L.wc;
      a.w_stride = L.pitch;
    }
    // z, and the parts of the biases' gradient: of each tile of rows, or (bias_rows = 0) as many as there are shares of them
    a.bias_part = grad_bias && !narrow ? bias_part : nullptr;
    int bias_rows = 0;
    if (st == TBE_OK && !narrow && rows > 0) {
      const int tile = pick_tile(kLogits, rows, a.items, width, 1, 0, weight_shares_us).tile;
      bias_rows = kLogits[tile].bm;
      st = f16 ? ce_launch_z<1>(a, tile, s) : ce_launch_z<2>(a, tile, s);
    }
    CeArgs to_x = a, to_w = a;
    to_x.splits = to_w.splits = 0;
    to_x.bias_part = nullptr;
    TilePick w_pick = {0, 1};
    if (grad_x) {
      // the same shares for every piece: their sums go on
      if (first == 0 && narrow) {
        const int64_t share = rows * a.sum_pitch * 4;
        x_pick.splits = fused_splits((rows + stay - 1) / stay, a.items, pair_us, static_cast<double>(share),
                                     hmin(sum_x_bytes(rows, width) / share, rows <= kFewRows ? kMostFew : kMostSplits));
      }
      if (first == 0 && !narrow) x_pick = pick_tile(kGradX, rows, a.sum_pitch, a.items, kMostSplits, sum_x_bytes(rows, width), x_shares_us);
      to_x.sum = reinterpret_cast<float*>(ws + L.sum_x);
      to_x.splits = x_pick.splits;
      to_x.add = first > 0;
    }
    if (grad_weight || (grad_bias && narrow)) {
      if (narrow) {
        const int64_t share = a.items * a.sum_pitch * 4;
        w_pick.splits = fused_splits((a.items + stay - 1) / stay, rows, pair_us, static_cast<double>(share), hmin(kMostSplits, kSumBytes / share));
      } else {
        w_pick = pick_tile(kWeightTiles, a.items, a.sum_pitch, rows, kMostSplits, kSumBytes, weight_shares_us);
      }
      to_w.sum = reinterpret_cast<float*>(ws + L.sum_w);
      to_w.out = grad_weight ? static_cast<uint16_t*>(grad_weight) + first * grad_weight_stride : nullptr;
      to_w.out_stride = grad_weight_stride;
      to_w.splits = w_pick.splits;
      if (narrow) to_w.r.ref = b.weighed;
      if (narrow) to_w.bias_part = grad_bias ? bias_part : nullptr;
    }
    if (st == TBE_OK && narrow && (to_x.splits || to_w.splits))
      st = f16 ? ce_launch_fused<1>(to_x, to_w, s) : ce_launch_fused<2>(to_x, to_w, s);
    if (st == TBE_OK && !narrow && (to_x.splits || to_w.splits))
      st = f16 ? ce_launch_grads<1>(to_x, x_pick.tile, to_w, w_pick.tile, s) : ce_launch_grads<2>(to_x, x_pick.tile, to_w, w_pick.tile, s);
    if (st == TBE_OK && grad_weight && w_pick.splits > 1) st = launch_grad_w_sum(to_w, f16, b.largest, s);
    if (st == TBE_OK && grad_bias) {
      ProfScope ps("ce_grad_bias", s);
      const int64_t groups = hmin((static_cast<int64_t>(a.items) + kWave - 1) / kWave, 1 << 20);  // a launch has fewer than 2^32 threads
      hipLaunchKernelGGL(ce_grad_bias_kernel, dim3(static_cast<unsigned>(groups)), dim3(1024), 0, s, bias_part,
                         a.bias_stride, b, bias_rows, narrow ? w_pick.splits : 0, 1.0f / unit, a.items, grad_bias + first);
      st = check_launch("ce_grad_bias");
    }
  }
  if (st != TBE_OK || !grad_x) return st;
  ProfScope ps("ce_grad_x_sum", s);
  if (rows <= kFewRows && x_pick.splits >= 32 && width <= 1024) {
    int lanes = 1;
    while (lanes * 4 < width) lanes *= 2;
    auto each = f16 ? ce_grad_x_each_kernel<1> : ce_grad_x_each_kernel<2>;
    hipLaunchKernelGGL(each, dim3(static_cast<unsigned>(rows)), dim3(1024), 0, s, b, reinterpret_cast<const float*>(ws + L.sum_x), a.sum_pitch,
                       x_pick.splits, static_cast<int>(width), lanes, x_factor, static_cast<uint16_t*>(grad_x), grad_x_stride);
    return check_launch("ce_grad_x_sum");
  }
  auto kernel = f16 ? ce_grad_x_kernel<1> : ce_grad_x_kernel<2>;
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(hmin((rows + 3) / 4, 8192))), dim3(kBlock), 0, s, b,
                     reinterpret_cast<const float*>(ws + L.sum_x), a.sum_pitch, x_pick.splits, static_cast<int>(width), x_factor,
                     static_cast<uint16_t*>(grad_x), grad_x_stride);
  return check_launch("ce_grad_x_sum");
}

}  // namespace tbe
