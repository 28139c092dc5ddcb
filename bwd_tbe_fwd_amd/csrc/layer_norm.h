// Layer norm: kernels, one translation unit per type of x (layer_norm_f32.hip and its
// siblings); validation and dispatch are in layer_norm.hip.
//
// A row's sums need the whole row, so a row lives in the registers of the lanes that own it:
// it is read once, its mean and then the sum of squared deviations are taken from registers
// (two passes over registers lose nothing where the mean is large against the deviations, as
// sum x^2 - mean^2 would), and it is written once.  Both directions are bound by memory.  The
// lanes that own a row are 16 to 1024 by its width, so that a lane holds 4 to 32 elements: enough
// bytes in flight to cover the latency, few enough registers for several waves a SIMD next to the
// scale, the shift and (backward) their gradients' sums, which stay in registers while a workgroup
// walks its rows.
#pragma once

#include "tbe_internal.h"
#include "tower_device.h"

namespace tbe {

struct NormArgs {
  int64_t rows, width;
  const void* x;
  int64_t x_stride;
  const void* w;   // scale or NULL
  const void* b;   // shift or NULL
  int w_dt;
  float eps;
  void* y;         // forward: output
  int64_t y_stride;
  float* mean;     // forward: written (may be NULL); backward: read
  float* rstd;
  // backward
  const void* gy;
  int64_t gy_stride;
  void* gx;
  int64_t gx_stride;
  int stream;      // the rows written start on 16 bytes
  float* partial;  // [grid][2][width] sums of grad_y * h and of grad_y, or NULL
};

// Sums are divided by the width, not multiplied by its rounded inverse: the mean of a constant row is
// then that constant, and its deviations zero instead of a rounding error times 1 / sqrt(eps).
//
// Elements of one vector: 16 bytes of x.
template <int XT> constexpr int kNormVec = XT == 0 ? 4 : 8;

constexpr int kNormBlock = 256;
// Threads of a workgroup whose rows are owned by G lanes each.
constexpr int norm_block(int G) { return G > kWave ? G : kNormBlock; }

// Sum over the G threads that own a row, with one barrier where they are several waves.  s_red:
// a float for each wave.  A kernel uses two of them in turn: who writes one again has passed the
// other's barrier, so everyone has read it.
template <int G>
__device__ __forceinline__ float row_sum(float v, float* s_red) {
  if constexpr (G <= 64) {
    return lanes_sum<G>(v);
  } else {
    constexpr int kW = G / kWave;
    v = lanes_sum<64>(v);
    const int w = threadIdx.x >> 6;
    if (lane_id() == 0) s_red[w] = v;
    __syncthreads();
    float r = s_red[0];
#pragma unroll
    for (int i = 1; i < kW; ++i) r += s_red[i];
    return r;
  }
}

// Two sums with one barrier.  s_red: [2][waves] floats, another one of two in turn each row: who
// writes it again has passed the barrier of the row between, so everyone has read it.
template <int G>
__device__ __forceinline__ void row_sum2(float& u, float& v, float* s_red) {
  u = lanes_sum<G <= 64 ? G : 64>(u);
  v = lanes_sum<G <= 64 ? G : 64>(v);
  if constexpr (G > 64) {
    constexpr int kW = G / kWave;
    const int w = threadIdx.x >> 6;
    if (lane_id() == 0) {
      s_red[w] = u;
      s_red[kW + w] = v;
    }
    __syncthreads();
    u = s_red[0];
    v = s_red[kW];
#pragma unroll
    for (int i = 1; i < kW; ++i) {
      u += s_red[i];
      v += s_red[kW + i];
    }
  }
}

// VEC elements of the shared vector p from column c on (`left` of them valid), as floats; `none` where
// there is no vector.
template <int VEC>
__device__ __forceinline__ void load_shared(const void* p, int dt, int64_t c, int64_t left, float none, float (&v)[VEC]) {
  if (!p || left <= 0) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = none;
  } else if (dt == 0) {
    Vec<float, VEC> f;
    load_vec_part<float, VEC>(static_cast<const float*>(p) + c, left, f);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = f.e[i];
  } else {
    Vec<uint16_t, VEC> h;
    load_vec_part<uint16_t, VEC>(static_cast<const uint16_t*>(p) + c, left, h);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = dt == 1 ? Fmt<1>::to_f(h.e[i]) : Fmt<2>::to_f(h.e[i]);
  }
}

// A result vector: with the streaming policy where it is whole 16 bytes of a row that starts on 16.
// 65536 x 4096 in bf16: forward 252 -> 197 us, backward 349 -> 343 us; not for fp32 rows' gradients (131072
// x 4096: 1000 -> 1026 us).
template <typename S, int VEC>
__device__ __forceinline__ void store_row(S* p, int64_t left, bool stream, const Vec<S, VEC>& v) {
  if constexpr (VEC * sizeof(S) % 16 == 0) {
    if (stream && left >= VEC) {
      store_vec_stream<S, VEC>(p, v);
      return;
    }
  }
  store_vec_part<S, VEC>(p, left, v);
}

// Whether a kernel loads its next row before it works on this one: where a lane has at most 32 bytes of
// a row in flight.  (More cost the registers that the other waves' loads need: fp32 rows of 4096
// reach the memory's rate without.)
template <int XT, int NV> constexpr bool kNormAhead = NV * kNormVec<XT> * (XT == 0 ? 4 : 2) <= 32;

template <int XT, int YT, int G, int NV>
__global__ __launch_bounds__(norm_block(G)) void norm_forward_kernel(NormArgs a) {
  constexpr int VEC = kNormVec<XT>, B = norm_block(G), R = B / G;
  constexpr bool KEEP = NV * VEC <= 16;  // the scale and the shift stay in registers
  using XS = typename Fmt<XT>::S;
  using YS = typename Fmt<YT>::S;
  __shared__ float s_red[2][B / kWave];
  const int g = threadIdx.x % G;
  const XS* x = static_cast<const XS*>(a.x);
  YS* y = static_cast<YS*>(a.y);
  const float width = static_cast<float>(a.width);
  float w[KEEP ? NV : 1][VEC], b[KEEP ? NV : 1][VEC];
  if constexpr (KEEP) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t c = static_cast<int64_t>(v * G + g) * VEC;
      load_shared<VEC>(a.w, a.w_dt, c, a.width - c, 1.0f, w[v]);
      load_shared<VEC>(a.b, a.w_dt, c, a.width - c, 0.0f, b[v]);
    }
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * R;
  auto fetch = [&](int64_t r, Vec<XS, VEC>(&to)[NV]) {
    const XS* xr = x + min(r, a.rows - 1) * a.x_stride;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t c = static_cast<int64_t>(v * G + g) * VEC;
      load_vec_part<XS, VEC>(xr + c, a.width - c, to[v]);
    }
  };
  Vec<XS, VEC> raw[NV], ahead[kNormAhead<XT, NV> ? NV : 1];
  if constexpr (kNormAhead<XT, NV>) fetch(static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / G, ahead);
  // every thread of a workgroup makes the same number of steps (the barriers in row_sum)
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * R; r0 < a.rows; r0 += step) {
    const int64_t row = r0 + threadIdx.x / G;
    const bool live = row < a.rows;
    if constexpr (kNormAhead<XT, NV>) {
#pragma unroll
      for (int v = 0; v < NV; ++v) raw[v] = ahead[v];
      if (r0 + step < a.rows) fetch(row + step, ahead);
    } else {
      fetch(row, raw);
    }
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum += Fmt<XT>::to_f(raw[v].e[i]);
    const float mean = row_sum<G>(sum, s_red[0]) / width;
    float sq = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t left = a.width - static_cast<int64_t>(v * G + g) * VEC;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float d = Fmt<XT>::to_f(raw[v].e[i]) - mean;
        sq += i < left ? d * d : 0.0f;
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<G>(sq, s_red[1]) / width + a.eps);
    if (live) {
      if (g == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
      }
      YS* yr = y + row * a.y_stride;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int64_t c = static_cast<int64_t>(v * G + g) * VEC;
        if constexpr (!KEEP) {
          load_shared<VEC>(a.w, a.w_dt, c, a.width - c, 1.0f, w[0]);
          load_shared<VEC>(a.b, a.w_dt, c, a.width - c, 0.0f, b[0]);
        }
        Vec<YS, VEC> o;
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          o.e[i] = tower_from_f<YT>((Fmt<XT>::to_f(raw[v].e[i]) - mean) * rstd * w[KEEP ? v : 0][i] + b[KEEP ? v : 0][i]);
        store_row<YS, VEC>(yr + c, a.width - c, a.stream, o);
      }
    }
  }
}

// Rows wider than registers hold: one workgroup of 1024 a row, which reads it three times (from
// the caches after the first).
constexpr int kNormWide = 1024;
template <int XT, int YT>
__global__ __launch_bounds__(kNormWide) void norm_forward_wide_kernel(NormArgs a) {
  constexpr int VEC = kNormVec<XT>;
  using XS = typename Fmt<XT>::S;
  using YS = typename Fmt<YT>::S;
  __shared__ float s_red[2][kNormWide / kWave];
  const float width = static_cast<float>(a.width);
  constexpr int64_t kStep = static_cast<int64_t>(kNormWide) * VEC;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const XS* xr = static_cast<const XS*>(a.x) + row * a.x_stride;
    YS* yr = static_cast<YS*>(a.y) + row * a.y_stride;
    Vec<XS, VEC> raw;
    float sum = 0.0f, sq = 0.0f;
    for (int64_t c = threadIdx.x * VEC; c < a.width; c += kStep) {
      load_vec_part<XS, VEC>(xr + c, a.width - c, raw);
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum += Fmt<XT>::to_f(raw.e[i]);
    }
    const float mean = row_sum<kNormWide>(sum, s_red[0]) / width;
    for (int64_t c = threadIdx.x * VEC; c < a.width; c += kStep) {
      load_vec_part<XS, VEC>(xr + c, a.width - c, raw);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float d = Fmt<XT>::to_f(raw.e[i]) - mean;
        sq += i < a.width - c ? d * d : 0.0f;
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<kNormWide>(sq, s_red[1]) / width + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    for (int64_t c = threadIdx.x * VEC; c < a.width; c += kStep) {
      float w[VEC], b[VEC];
      load_vec_part<XS, VEC>(xr + c, a.width - c, raw);
      load_shared<VEC>(a.w, a.w_dt, c, a.width - c, 1.0f, w);
      load_shared<VEC>(a.b, a.w_dt, c, a.width - c, 0.0f, b);
      Vec<YS, VEC> o;
#pragma unroll
      for (int i = 0; i < VEC; ++i) o.e[i] = tower_from_f<YT>((Fmt<XT>::to_f(raw.e[i]) - mean) * rstd * w[i] + b[i]);
      store_row<YS, VEC>(yr + c, a.width - c, a.stream, o);
    }
  }
}

// Backward.  Each workgroup walks rows blockIdx.x, + gridDim.x, ... and keeps its columns' sums
// of grad_y * h and grad_y in registers; at the end the lane groups that share columns add up
// through LDS in their order and the workgroup writes one partial row pair.
template <int XT, int YT, int G, int NV>
__global__ __launch_bounds__(norm_block(G)) void norm_backward_kernel(NormArgs a) {
  constexpr int VEC = kNormVec<XT>, B = norm_block(G), R = B / G;
  using XS = typename Fmt<XT>::S;
  using YS = typename Fmt<YT>::S;
  __shared__ float s_red[2][2 * B / kWave];
  __shared__ float s_part[R > 1 ? B * VEC : 1];
  const int g = threadIdx.x % G;
  const float width = static_cast<float>(a.width);
  float w[NV][VEC], gw[NV][VEC], gb[NV][VEC];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int64_t c = static_cast<int64_t>(v * G + g) * VEC;
    load_shared<VEC>(a.w, a.w_dt, c, a.width - c, 1.0f, w[v]);
#pragma unroll
    for (int i = 0; i < VEC; ++i) gw[v][i] = gb[v][i] = 0.0f;
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * R;
  // A wave that owns whole rows of 16 bits loads its next row before it works on this one: 10007 rows of
  // 1001, where a wave has two or three, 27.1 -> 22.2 us.  Wider rows lose more by the registers
  // (65536 rows of 4096: 0.41 -> 0.52 ms).
  constexpr bool AHEAD = G == 64 && XT != 0;
  auto fetch = [&](int64_t r, Vec<XS, VEC>(&xs)[NV], Vec<YS, VEC>(&gs)[NV], float& mean, float& rstd) {
    const bool live = r < a.rows;
    const int64_t row = live ? r : a.rows - 1;
    const XS* xr = static_cast<const XS*>(a.x) + row * a.x_stride;
    const YS* gr = static_cast<const YS*>(a.gy) + row * a.gy_stride;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t c = static_cast<int64_t>(v * G + g) * VEC;
      // a group without a row reads the last row and adds zeros
      load_vec_part<XS, VEC>(xr + c, a.width - c, xs[v]);
      load_vec_part<YS, VEC>(gr + c, live ? a.width - c : 0, gs[v]);
    }
    mean = a.mean[row];
    rstd = a.rstd[row];
  };
  Vec<XS, VEC> raw[NV], raw_ahead[AHEAD ? NV : 1];
  Vec<YS, VEC> gin[NV], gin_ahead[AHEAD ? NV : 1];
  float mean, rstd, mean_ahead, rstd_ahead;
  if constexpr (AHEAD) fetch(static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / G, raw_ahead, gin_ahead, mean_ahead, rstd_ahead);
  int turn = 0;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * R; r0 < a.rows; r0 += step, turn ^= 1) {
    const int64_t row = r0 + threadIdx.x / G;
    const bool live = row < a.rows;
    if constexpr (AHEAD) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        raw[v] = raw_ahead[v];
        gin[v] = gin_ahead[v];
      }
      mean = mean_ahead;
      rstd = rstd_ahead;
      if (r0 + step < a.rows) fetch(row + step, raw_ahead, gin_ahead, mean_ahead, rstd_ahead);
    } else {
      fetch(row, raw, gin, mean, rstd);
    }
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t c = static_cast<int64_t>(v * G + g) * VEC, left = live ? a.width - c : 0;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        // columns past the row have no h (mean * rstd there could be infinite)
        const float h = i < left ? (Fmt<XT>::to_f(raw[v].e[i]) - mean) * rstd : 0.0f;
        const float gy = Fmt<YT>::to_f(gin[v].e[i]);
        const float d = gy * w[v][i];
        c1 += d;
        c2 += d * h;
        gw[v][i] += gy * h;
        gb[v][i] += gy;
      }
    }
    row_sum2<G>(c1, c2, s_red[turn]);
    c1 /= width;
    c2 /= width;
    if (live && a.gx) {
      XS* xo = static_cast<XS*>(a.gx) + row * a.gx_stride;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int64_t c = static_cast<int64_t>(v * G + g) * VEC;
        Vec<XS, VEC> o;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float h = (Fmt<XT>::to_f(raw[v].e[i]) - mean) * rstd;
          o.e[i] = tower_from_f<XT>((Fmt<YT>::to_f(gin[v].e[i]) * w[v][i] - c1 - h * c2) * rstd);
        }
        store_row<XS, VEC>(xo + c, a.width - c, XT != 0 && a.stream, o);
      }
    }
  }
  if (!a.partial) return;
  float* out = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.width;
  if constexpr (R == 1) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t c = static_cast<int64_t>(v * G + g) * VEC;
      Vec<float, VEC> o, p;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        o.e[i] = gw[v][i];
        p.e[i] = gb[v][i];
      }
      store_vec_part<float, VEC>(out + c, a.width - c, o);
      store_vec_part<float, VEC>(out + a.width + c, a.width - c, p);
    }
  } else {
#pragma unroll
    for (int v = 0; v < 2 * NV; ++v) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < VEC; ++i) s_part[threadIdx.x * VEC + i] = v < NV ? gw[v % NV][i] : gb[v % NV][i];
      __syncthreads();
      for (int e = threadIdx.x; e < G * VEC; e += B) {
        float sum = 0.0f;
        for (int k = 0; k < R; ++k) sum += s_part[k * G * VEC + e];
        const int64_t c = static_cast<int64_t>(v % NV) * G * VEC + e;
        if (c < a.width) out[(v < NV ? 0 : a.width) + c] = sum;
      }
    }
  }
}

// Rows wider than registers hold: the row kernel takes grad_x in two passes; the column kernel
// below takes the partial sums, a slice of rows and 256 columns a workgroup.
template <int XT, int YT>
__global__ __launch_bounds__(kNormWide) void norm_backward_wide_kernel(NormArgs a) {
  constexpr int VEC = kNormVec<XT>;
  constexpr int64_t kStep = static_cast<int64_t>(kNormWide) * VEC;
  using XS = typename Fmt<XT>::S;
  using YS = typename Fmt<YT>::S;
  Vec<XS, VEC> raw;
  Vec<YS, VEC> gin;
  __shared__ float s_red[2][2 * kNormWide / kWave];
  const float width = static_cast<float>(a.width);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const XS* xr = static_cast<const XS*>(a.x) + row * a.x_stride;
    const YS* gr = static_cast<const YS*>(a.gy) + row * a.gy_stride;
    XS* xo = static_cast<XS*>(a.gx) + row * a.gx_stride;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float c1 = 0.0f, c2 = 0.0f;
    for (int64_t c = threadIdx.x * VEC; c < a.width; c += kStep) {
      float w[VEC];
      load_vec_part<XS, VEC>(xr + c, a.width - c, raw);
      load_vec_part<YS, VEC>(gr + c, a.width - c, gin);  // zeros past the row
      load_shared<VEC>(a.w, a.w_dt, c, a.width - c, 1.0f, w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float d = Fmt<YT>::to_f(gin.e[i]) * w[i];
        c1 += d;
        c2 += i < a.width - c ? d * ((Fmt<XT>::to_f(raw.e[i]) - mean) * rstd) : 0.0f;
      }
    }
    row_sum2<kNormWide>(c1, c2, s_red[turn]);
    c1 /= width;
    c2 /= width;
    for (int64_t c = threadIdx.x * VEC; c < a.width; c += kStep) {
      float w[VEC];
      load_vec_part<XS, VEC>(xr + c, a.width - c, raw);
      load_vec_part<YS, VEC>(gr + c, a.width - c, gin);
      load_shared<VEC>(a.w, a.w_dt, c, a.width - c, 1.0f, w);
      Vec<XS, VEC> o;
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        o.e[i] = tower_from_f<XT>((Fmt<YT>::to_f(gin.e[i]) * w[i] - c1 - (Fmt<XT>::to_f(raw.e[i]) - mean) * rstd * c2) * rstd);
      store_row<XS, VEC>(xo + c, a.width - c, XT != 0 && a.stream, o);
    }
  }
}
template <int XT, int YT>
__global__ __launch_bounds__(kNormBlock) void norm_columns_kernel(NormArgs a) {
  using XS = typename Fmt<XT>::S;
  using YS = typename Fmt<YT>::S;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kNormBlock + threadIdx.x;
  if (c >= a.width) return;
  float gw = 0.0f, gb = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float gy = Fmt<YT>::to_f(static_cast<const YS*>(a.gy)[row * a.gy_stride + c]);
    gw += gy * (Fmt<XT>::to_f(static_cast<const XS*>(a.x)[row * a.x_stride + c]) - a.mean[row]) * a.rstd[row];
    gb += gy;
  }
  float* out = a.partial + static_cast<int64_t>(blockIdx.y) * 2 * a.width;
  out[c] = gw;
  out[a.width + c] = gb;
}

// ---------------------------------------------------------------------------
// dispatch: the lanes of a row and the vectors of a lane by the width
// ---------------------------------------------------------------------------
// Workgroups of the backward, at most: each writes a pair of partial rows, which the final sum
// reads.  At most 2^23 elements of them (32 MiB a sum), but 8 for the widest rows.
inline int64_t norm_partials(int64_t width) { return hmax(8, hmin(1024, (int64_t{1} << 23) / width)); }

template <typename K>
tbe_status norm_launch(const char* what, K* kernel, int64_t work, int threads, int64_t cap, const NormArgs& a,
                       hipStream_t s, int* grid_out) {
  const int grid = static_cast<int>(hmin(resident_grid(kernel, work, 0, threads), cap));
  if (grid_out) *grid_out = grid;
  ProfScope ps(what, s);
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(threads), 0, s, a);
  return check_launch(what);
}

template <int XT, int YT, int G, int NV>
tbe_status norm_forward_as(const NormArgs& a, hipStream_t s) {
  constexpr int B = norm_block(G);
  constexpr int64_t R = B / G;
  return norm_launch("norm_forward", norm_forward_kernel<XT, YT, G, NV>, (a.rows + R - 1) / R, B, 0x7fffffff, a, s, nullptr);
}
template <int XT, int YT, int G, int NV>
tbe_status norm_backward_as(const NormArgs& a, hipStream_t s, int* grid) {
  constexpr int B = norm_block(G);
  constexpr int64_t R = B / G;
  // at least two rows a lane group: a workgroup's partial rows are as many bytes as one or two rows
  return norm_launch("norm_backward", norm_backward_kernel<XT, YT, G, NV>, (a.rows + 2 * R - 1) / (2 * R), B,
                     norm_partials(a.width), a, s, grid);
}

// Up to 16 elements a lane (32 for the widest rows), by as few lanes as that takes.
template <int XT, int YT>
tbe_status norm_forward_types(const NormArgs& a, hipStream_t s) {
  constexpr int F = XT == 0 ? 2 : 1;  // vectors of 8 elements
  const int64_t n = (a.width + kNormVec<XT> - 1) / kNormVec<XT>;  // vectors of a row
  if (n <= 16) return norm_forward_as<XT, YT, 16, 1>(a, s);
  if (n <= 32) return norm_forward_as<XT, YT, 16, 2>(a, s);
  if (n <= 64) return norm_forward_as<XT, YT, 64, 1>(a, s);
  if (n <= 64 * 2 * F) return norm_forward_as<XT, YT, 64, 2 * F>(a, s);
  if (n <= 256 * F) return norm_forward_as<XT, YT, 256, F>(a, s);
  if (n <= 256 * 2 * F) return norm_forward_as<XT, YT, 256, 2 * F>(a, s);
  if (n <= 512 * 2 * F) return norm_forward_as<XT, YT, 512, 2 * F>(a, s);
  if (n <= 1024 * 2 * F) return norm_forward_as<XT, YT, 1024, 2 * F>(a, s);
  if (n <= 1024 * 4 * F) return norm_forward_as<XT, YT, 1024, 4 * F>(a, s);
  return norm_launch("norm_forward", norm_forward_wide_kernel<XT, YT>, a.rows, kNormWide, 0x7fffffff, a, s, nullptr);
}

// 16 elements a lane for x of fp32, 8 where several waves own a row of 16 bits: more waves a row, fewer
// registers (65536 rows of 4096: 256 lanes 0.41 ms, 512 lanes 0.36 ms).
template <int XT, int YT>
tbe_status norm_backward_types(const NormArgs& a, hipStream_t s, int* grid) {
  const int64_t n = (a.width + kNormVec<XT> - 1) / kNormVec<XT>;
  if (n <= 16) return norm_backward_as<XT, YT, 16, 1>(a, s, grid);
  if (n <= 32) return norm_backward_as<XT, YT, 16, 2>(a, s, grid);
  if (n <= 64) return norm_backward_as<XT, YT, 64, 1>(a, s, grid);
  if constexpr (XT == 0) {
    if (n <= 128) return norm_backward_as<XT, YT, 64, 2>(a, s, grid);
    if (n <= 256) return norm_backward_as<XT, YT, 64, 4>(a, s, grid);
    if (n <= 512) return norm_backward_as<XT, YT, 256, 2>(a, s, grid);
    if (n <= 1024) return norm_backward_as<XT, YT, 256, 4>(a, s, grid);
    if (n <= 2048) return norm_backward_as<XT, YT, 512, 4>(a, s, grid);
    if (n <= 4096) return norm_backward_as<XT, YT, 1024, 4>(a, s, grid);
  } else {
    if (n <= 128) return norm_backward_as<XT, YT, 64, 2>(a, s, grid);
    if (n <= 256) return norm_backward_as<XT, YT, 256, 1>(a, s, grid);
    if (n <= 512) return norm_backward_as<XT, YT, 512, 1>(a, s, grid);
    if (n <= 1024) return norm_backward_as<XT, YT, 1024, 1>(a, s, grid);
    if (n <= 2048) return norm_backward_as<XT, YT, 1024, 2>(a, s, grid);
  }
  tbe_status st = TBE_OK;
  if (a.gx) st = norm_launch("norm_backward", norm_backward_wide_kernel<XT, YT>, a.rows, kNormWide, 0x7fffffff, a, s, nullptr);
  if (st != TBE_OK || !a.partial) return st;
  *grid = static_cast<int>(hmin(a.rows, norm_partials(a.width)));
  ProfScope ps("norm_columns", s);
  hipLaunchKernelGGL((norm_columns_kernel<XT, YT>), dim3((a.width + kNormBlock - 1) / kNormBlock, *grid), dim3(kNormBlock), 0, s, a);
  return check_launch("norm_columns");
}

// one of these per translation unit
template <int XT> tbe_status norm_forward_x(const NormArgs& a, int y_dt, hipStream_t s);
template <int XT> tbe_status norm_backward_x(const NormArgs& a, int y_dt, hipStream_t s, int* grid);

#define TBE_NORM_TYPE(XT)                                                                              \
  template <> tbe_status norm_forward_x<XT>(const NormArgs& a, int y_dt, hipStream_t s) {              \
    return y_dt == 0 ? norm_forward_types<XT, 0>(a, s)                                                 \
                     : y_dt == 1 ? norm_forward_types<XT, 1>(a, s) : norm_forward_types<XT, 2>(a, s);  \
  }                                                                                                    \
  template <> tbe_status norm_backward_x<XT>(const NormArgs& a, int y_dt, hipStream_t s, int* grid) {  \
    return y_dt == 0 ? norm_backward_types<XT, 0>(a, s, grid)                                          \
                     : y_dt == 1 ? norm_backward_types<XT, 1>(a, s, grid)                              \
                                 : norm_backward_types<XT, 2>(a, s, grid);                             \
  }

}  // namespace tbe
