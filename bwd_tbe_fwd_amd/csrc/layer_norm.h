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

// Sums are divided by the width, not multiplied by its rounded inverse: the mean of a constant row is then
// that constant where its sum is exact.
//
// An fp32 sum rounds, also where all values are equal, so a mean is off by some units in its last place: a row of a
// thousand 1000.1 by 1.2e-4, 0.04 in y at eps 1e-5.  The deviations from it round only by themselves, so their sum
// divided by the width corrects the mean to its own rounding, and the squares' mean less the square of that
// correction is the variance.  This is taken (`correct`, once more through the row's registers) for rows whose
// mean is more than four standard deviations from zero; for the others the error is below 5 * 256 units of 2^-24 in
// y.  Taken for every row it cost 2 to 5% of the time (131072 rows of 512 fp32 87.0 -> 89.4 us, 67 M values in rows of
// 200 90.5 -> 95.1); asking costs less than 1%, but 4% where instructions bound the kernel (rows of 16 193 -> 201
// us).  Where all rows are far from zero they take 5 to 8% longer (512 wide 87.9 -> 92.5 us), rows of 16 25% and fp16
// rows of 9001 28%.  Values of 16 bits are left alone where a row of them has exact sums if it is far from zero:
// multiples of one step, up to 2^9 steps in bf16 and 2^12 in fp16, 2^15 and 2^12 of which fp32 adds exactly.
template <int XT, int64_t MOST> constexpr bool kNormCorrect = XT == 0 || MOST > (XT == 1 ? 4096 : 32768);
__device__ __forceinline__ bool far_from_zero(float mean, float var) { return mean * mean > 16.0f * var; }
__device__ __forceinline__ void correct(float off, float& mean, float& var) {
  mean += off;
  var -= off * off;
  var = var < 0.0f ? 0.0f : var;
}

// Elements of one vector: 16 bytes of x.
template <int XT> constexpr int kNormVec = XT == 0 ? 4 : 8;

constexpr int kNormBlock = 256;
// Threads of a workgroup whose rows are owned by G lanes each.
constexpr int norm_block(int G) { return G > kWave ? G : kNormBlock; }

// Sum over the G threads that own a row, with one barrier where they are several waves.  s_red:
// a float for each wave.  A kernel uses two of them in turn, or more: who writes one again has passed another's
// barrier, so everyone has read it.
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

// Where a lane's v-th vector of a row lies.  EDGE kFull: every lane's vectors lie inside the row; kWhole: some
// lie past it (skip = VEC); kRagged: the width is no multiple of VEC.  The row's last vector then ends at its
// last column: it starts earlier, and `skip` of its elements are the vector's before it too, which both
// compute and store alike and only the first adds to sums.  So every access is a whole vector, and no lane
// walks through a vector's elements (67 M values of bf16, backward: rows of 900 131 -> 83 us, of 361 162 ->
// 86; rows of 4096 92 -> 80 by the packed zeros below).
enum { kFull = 0, kWhole = 1, kRagged = 2 };
inline int norm_edge(int64_t width, int G, int vec, int nv) { return width % vec ? kRagged : width == static_cast<int64_t>(G) * vec * nv ? kFull : kWhole; }
template <int G, int VEC, int EDGE>
struct Place {
  static constexpr bool RAGGED = EDGE == kRagged;
  int64_t c;  // first column; negative for rows narrower than a vector
  int skip;
  __device__ __forceinline__ Place(int v, int64_t width) {
    c = static_cast<int64_t>(v * G + threadIdx.x % G) * VEC;
    skip = EDGE == kFull ? 0 : c >= width ? VEC : RAGGED ? static_cast<int>(max(c + VEC - width, static_cast<int64_t>(0))) : 0;
    if (RAGGED) c -= skip;
  }
  __device__ __forceinline__ bool in() const { return EDGE == kFull || skip < VEC; }
  // A row narrower than a vector goes element by element; it is one of the 16-lane kernels'.
  __device__ __forceinline__ static bool narrow(int64_t width) { return RAGGED && G == 16 && width < VEC; }
  __device__ __forceinline__ bool has(int i) const { return !RAGGED || i >= skip; }
  template <typename S>
  __device__ __forceinline__ void load(const S* p, int64_t width, bool live, Vec<S, VEC>& v) const {
    // Packed until it is used: the compiler otherwise takes a vector apart where the zeros and the loaded
    // values meet, and waits there for one load before it starts the next.
    constexpr int kBytes = VEC * static_cast<int>(sizeof(S)), kPart = kBytes < 16 ? kBytes : 16;
    typedef uint32_t Part __attribute__((ext_vector_type(kPart / 4)));
    Part x[kBytes / kPart] = {};
    if (live && in()) {
      if (!narrow(width)) {
#pragma unroll
        for (int k = 0; k < kBytes / kPart; ++k) __builtin_memcpy(&x[k], reinterpret_cast<const char*>(p + c) + k * kPart, kPart);
      } else {
        Vec<S, VEC> e;
#pragma unroll
        for (int i = 0; i < VEC; ++i) e.e[i] = i >= skip ? p[c + i] : S(0);
        __builtin_memcpy(x, e.e, kBytes);
      }
    }
    __builtin_memcpy(v.e, x, kBytes);
  }
  // stream: the rows start on 16 bytes, and results go past the caches (65536 rows of 4096 in bf16: forward 252 ->
  // 197 us, backward 349 -> 343 us; not fp32 rows' gradients: 131072 rows of 4096 1000 -> 1026 us)
  template <typename S>
  __device__ __forceinline__ void store(S* p, int64_t width, bool stream, const Vec<S, VEC>& v) const {
    if (!in()) return;
    if (narrow(width)) {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (i >= skip) p[c + i] = v.e[i];
      return;
    }
    if constexpr (VEC * sizeof(S) % 16 == 0) {
      if (stream && (!RAGGED || skip == 0)) {
        store_vec_stream<S, VEC>(p + c, v);
        return;
      }
    }
    store_vec_any<S, VEC>(p + c, v);
  }
  // of a vector that every row shares, as floats; `none` where there is none
  __device__ __forceinline__ void shared(const void* p, int dt, int64_t width, float none, float (&v)[VEC]) const {
    if (!p || !in()) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = none;
    } else if (narrow(width)) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = i >= skip ? load_any(p, dt, c + i) : none;
    } else {
      load_shared<VEC>(p, dt, c, VEC, none, v);
    }
  }
};

// A result vector of a wider row: with the streaming policy where it is whole 16 bytes of a row that starts on 16.
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

// Whether the forward loads its next row before it works on this one: where a lane has at most 32 bytes of
// a row in flight.  (More cost the registers that the other waves' loads need: fp32 rows of 4096
// reach the memory's rate without.)
template <int XT, int NV> constexpr bool kNormAhead = NV * kNormVec<XT> * (XT == 0 ? 4 : 2) <= 32;

template <int XT, int YT, int G, int NV, int EDGE>
__global__ __launch_bounds__(norm_block(G)) void norm_forward_kernel(NormArgs a) {
  constexpr int VEC = kNormVec<XT>, B = norm_block(G), R = B / G;
  constexpr bool KEEP = NV * VEC <= 16;  // the scale and the shift stay in registers
  using At = Place<G, VEC, EDGE>;
  using XS = typename Fmt<XT>::S;
  using YS = typename Fmt<YT>::S;
  __shared__ float s_red[3][B / kWave];
  const int g = threadIdx.x % G;
  const XS* x = static_cast<const XS*>(a.x);
  YS* y = static_cast<YS*>(a.y);
  const float width = static_cast<float>(a.width);
  float w[KEEP ? NV : 1][VEC], b[KEEP ? NV : 1][VEC];
  if constexpr (KEEP) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const At at(v, a.width);
      at.shared(a.w, a.w_dt, a.width, 1.0f, w[v]);
      at.shared(a.b, a.w_dt, a.width, 0.0f, b[v]);
    }
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * R;
  auto fetch = [&](int64_t r, Vec<XS, VEC>(&to)[NV]) {
    const XS* xr = x + min(r, a.rows - 1) * a.x_stride;
#pragma unroll
    for (int v = 0; v < NV; ++v) At(v, a.width).load(xr, a.width, true, to[v]);
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
    for (int v = 0; v < NV; ++v) {
      const At at(v, a.width);  // zeros past the row
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum += at.has(i) ? Fmt<XT>::to_f(raw[v].e[i]) : 0.0f;
    }
    float mean = row_sum<G>(sum, s_red[0]) / width, sq = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const At at(v, a.width);
      const float middle = at.in() ? mean : 0.0f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float d = Fmt<XT>::to_f(raw[v].e[i]) - middle;
        sq += at.has(i) ? d * d : 0.0f;
      }
    }
    float var = row_sum<G>(sq, s_red[1]) / width;
    if constexpr (kNormCorrect<XT, static_cast<int64_t>(G) * NV * VEC>) {
      if (far_from_zero(mean, var)) {  // the same for all who own the row
        float off = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const At at(v, a.width);
          const float middle = at.in() ? mean : 0.0f;
#pragma unroll
          for (int i = 0; i < VEC; ++i) off += at.has(i) ? Fmt<XT>::to_f(raw[v].e[i]) - middle : 0.0f;
        }
        correct(row_sum<G>(off, s_red[2]) / width, mean, var);
      }
    }
    const float rstd = 1.0f / sqrtf(var + a.eps);
    if (live) {
      if (g == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
      }
      YS* yr = y + row * a.y_stride;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const At at(v, a.width);
        if constexpr (!KEEP) {
          at.shared(a.w, a.w_dt, a.width, 1.0f, w[0]);
          at.shared(a.b, a.w_dt, a.width, 0.0f, b[0]);
        }
        Vec<YS, VEC> o;
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          o.e[i] = tower_from_f<YT>((Fmt<XT>::to_f(raw[v].e[i]) - mean) * rstd * w[KEEP ? v : 0][i] + b[KEEP ? v : 0][i]);
        at.store(yr, a.width, a.stream, o);
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
  __shared__ float s_red[3][kNormWide / kWave];
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
    float mean = row_sum<kNormWide>(sum, s_red[0]) / width;
    for (int64_t c = threadIdx.x * VEC; c < a.width; c += kStep) {
      load_vec_part<XS, VEC>(xr + c, a.width - c, raw);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float d = Fmt<XT>::to_f(raw.e[i]) - mean;
        sq += i < a.width - c ? d * d : 0.0f;
      }
    }
    float var = row_sum<kNormWide>(sq, s_red[1]) / width;
    if (far_from_zero(mean, var)) {
      float off = 0.0f;
      for (int64_t c = threadIdx.x * VEC; c < a.width; c += kStep) {
        load_vec_part<XS, VEC>(xr + c, a.width - c, raw);
#pragma unroll
        for (int i = 0; i < VEC; ++i) off += i < a.width - c ? Fmt<XT>::to_f(raw.e[i]) - mean : 0.0f;
      }
      correct(row_sum<kNormWide>(off, s_red[2]) / width, mean, var);
    }
    const float rstd = 1.0f / sqrtf(var + a.eps);
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
template <int XT, int YT, int G, int NV, int EDGE>
__global__ __launch_bounds__(norm_block(G)) void norm_backward_kernel(NormArgs a) {
  constexpr int VEC = kNormVec<XT>, B = norm_block(G), R = B / G;
  using At = Place<G, VEC, EDGE>;
  using XS = typename Fmt<XT>::S;
  using YS = typename Fmt<YT>::S;
  __shared__ float s_red[2][2 * B / kWave];
  __shared__ float s_part[R > 1 ? B * VEC : 1];
  const int g = threadIdx.x % G;
  const float width = static_cast<float>(a.width);
  float w[NV][VEC], gw[NV][VEC], gb[NV][VEC];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    At(v, a.width).shared(a.w, a.w_dt, a.width, 1.0f, w[v]);
#pragma unroll
    for (int i = 0; i < VEC; ++i) gw[v][i] = gb[v][i] = 0.0f;
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * R;
  // A wave that owns whole rows of 16 bits loads its next row before it works on this one: 10007 rows of
  // 1001, where a wave has five, 20.7 -> 19.1 us.  Wider rows have several waves to wait for each other (65536
  // rows of 4096: 297 us with and without).
  constexpr bool AHEAD = G == 64 && XT != 0;
  auto fetch = [&](int64_t r, Vec<XS, VEC>(&xs)[NV], Vec<YS, VEC>(&gs)[NV], float& mean, float& rstd) {
    const bool live = r < a.rows;
    const int64_t row = live ? r : a.rows - 1;  // a group without a row reads the last one's x and adds zeros
    const XS* xr = static_cast<const XS*>(a.x) + row * a.x_stride;
    const YS* gr = static_cast<const YS*>(a.gy) + row * a.gy_stride;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const At at(v, a.width);
      at.load(xr, a.width, true, xs[v]);
      at.load(gr, a.width, live, gs[v]);
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
      const At at(v, a.width);
      const float scale = at.in() ? rstd : 0.0f;  // columns past the row have no h (mean * rstd there could be infinite)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float h = at.has(i) ? (Fmt<XT>::to_f(raw[v].e[i]) - mean) * scale : 0.0f;
        const float gy = at.has(i) ? Fmt<YT>::to_f(gin[v].e[i]) : 0.0f;
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
        Vec<XS, VEC> o;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float h = (Fmt<XT>::to_f(raw[v].e[i]) - mean) * rstd;
          o.e[i] = tower_from_f<XT>((Fmt<YT>::to_f(gin[v].e[i]) * w[v][i] - c1 - h * c2) * rstd);
        }
        At(v, a.width).store(xo, a.width, XT != 0 && a.stream, o);
      }
    }
  }
  if (!a.partial) return;
  float* out = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.width;
  if constexpr (R == 1) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const At at(v, a.width);
      if (!at.in()) continue;
      Vec<float, VEC> o, p;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        o.e[i] = gw[v][i];
        p.e[i] = gb[v][i];
      }
      if (at.skip == 0) {
        store_vec_any<float, VEC>(out + at.c, o);
        store_vec_any<float, VEC>(out + a.width + at.c, p);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (i >= at.skip) {
            out[at.c + i] = o.e[i];
            out[a.width + at.c + i] = p.e[i];
          }
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < 2 * NV; ++v) {
      __syncthreads();
      const At at(v % NV, a.width);
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (i >= at.skip) s_part[threadIdx.x * VEC + i - at.skip] = v < NV ? gw[v % NV][i] : gb[v % NV][i];
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
  const int edge = norm_edge(a.width, G, kNormVec<XT>, NV);
  auto kernel = edge == kFull ? norm_forward_kernel<XT, YT, G, NV, kFull>
                              : edge == kWhole ? norm_forward_kernel<XT, YT, G, NV, kWhole> : norm_forward_kernel<XT, YT, G, NV, kRagged>;
  // No more workgroups than keep the memory busy, by the bytes that each reads at a time, as in the backward.
  // 512 / 768 / 1024 / all resident: 131072 rows of 4096 fp32, 16 KB: 569 / 597 / 649 / 618 us; 400000 rows of 1001 of 16
  // bits, 8 KB: - / 302 / 333 / 339; 200000 rows of 2048, 4 KB: - / 325 / 289 / 331; 67 M values in rows of 200 fp32, 3 KB: - /
  // - / 111 / 95.
  const int64_t bytes = R * a.width * static_cast<int64_t>(sizeof(typename Fmt<XT>::S));
  const int64_t cap = bytes >= 12000 ? 512 : bytes >= 6500 ? 768 : bytes >= 3800 ? 1024 : 0x7fffffff;
  return norm_launch("norm_forward", kernel, (a.rows + R - 1) / R, B, cap, a, s, nullptr);
}
template <int XT, int YT, int G, int NV>
tbe_status norm_backward_as(const NormArgs& a, hipStream_t s, int* grid) {
  constexpr int B = norm_block(G);
  constexpr int64_t R = B / G;
  // At least two rows a lane group: a workgroup's partial rows are as many bytes as one or two rows.  And no more
  // workgroups than keep the memory busy, two to four a CU by the bytes that each reads at a time: more make reads
  // and writes meet.  512 / 768 / 1024 workgroups: 131072 rows of 4096, fp32 and bf16, 24 KB: 991 / 1034 / 1149 us; 67 M
  // values of bf16 in rows of 2048, 8 KB: 92 / 77 / 81; of 1501, 6 KB: - / 104 / 91.
  const int64_t bytes = R * a.width * static_cast<int64_t>(sizeof(typename Fmt<XT>::S) + sizeof(typename Fmt<YT>::S));
  const int edge = norm_edge(a.width, G, kNormVec<XT>, NV);
  auto kernel = edge == kFull ? norm_backward_kernel<XT, YT, G, NV, kFull>
                              : edge == kWhole ? norm_backward_kernel<XT, YT, G, NV, kWhole> : norm_backward_kernel<XT, YT, G, NV, kRagged>;
  return norm_launch("norm_backward", kernel, (a.rows + 2 * R - 1) / (2 * R), B,
                     hmin(bytes >= 12000 ? 512 : bytes >= 6500 ? 768 : 1024, norm_partials(a.width)), a, s, grid);
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
  if constexpr (XT != 0) {
    if (n <= 192) return norm_forward_as<XT, YT, 192, 1>(a, s);
    if (n > 256 && n <= 384) return norm_forward_as<XT, YT, 192, 2>(a, s);
    if (n > 1024 && n <= 1536) return norm_forward_as<XT, YT, 768, 2>(a, s);
  }
  if (n <= 256 * F) return norm_forward_as<XT, YT, 256, F>(a, s);
  if (n <= 256 * 2 * F) return norm_forward_as<XT, YT, 256, 2 * F>(a, s);
  if (n <= 512 * 2 * F) return norm_forward_as<XT, YT, 512, 2 * F>(a, s);
  if (n <= 1024 * 2 * F) return norm_forward_as<XT, YT, 1024, 2 * F>(a, s);
  if (n <= 1024 * 4 * F) return norm_forward_as<XT, YT, 1024, 4 * F>(a, s);
  return norm_launch("norm_forward", norm_forward_wide_kernel<XT, YT>, a.rows, kNormWide, 0x7fffffff, a, s, nullptr);
}

// 16 elements a lane for x of fp32; 8 or 16 where several waves own a row of 16 bits (65536 rows of 4096: 512 lanes
// of one vector 297 us, 256 lanes of two 284).
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
    if (n <= 3072) return norm_backward_as<XT, YT, 1024, 3>(a, s, grid);
    // 67 M values, 1024 lanes of 4 vectors or 512 of 8: rows of 16384 167 / 205 us, of 14001 295 / 192
    if (n <= 4096 && a.width % kNormVec<XT>) return norm_backward_as<XT, YT, 512, 8>(a, s, grid);
    if (n <= 4096) return norm_backward_as<XT, YT, 1024, 4>(a, s, grid);
  } else {
    if (n <= 128) return norm_backward_as<XT, YT, 64, 2>(a, s, grid);
    if (n <= 256) return norm_backward_as<XT, YT, 256, 1>(a, s, grid);
    if (n <= 512) return norm_backward_as<XT, YT, 256, 2>(a, s, grid);
    if (n <= 1024) return norm_backward_as<XT, YT, 1024, 1>(a, s, grid);
    if (n <= 2048) return norm_backward_as<XT, YT, 512, 4>(a, s, grid);
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
