// AdamW over many tensors: the step and the reading of states of 8 bits.  Declarations, formulas
// and the format of the states are in include/tbe_tower.h.
//
// Every value is read and written once and the arithmetic is a few operations a value, so the
// step is bound by memory.  A launch takes up to kTensors tensors, whose descriptors travel in the
// kernel's arguments (no table to upload, nothing kept between calls); a workgroup finds its
// tensor among the chunk counts with one load and one ballot.  A lane holds 8 values at a time:
// 16 or 32 bytes of each array, and 16 lanes share one block of an 8-bit state, whose largest
// magnitude they find among themselves in registers.
#include "tbe_internal.h"
#include "tower_device.h"

#include <cmath>

#include "../../include/tbe_tower.h"

namespace tbe {
namespace {

constexpr int kVals = 8;                             // values a lane holds at a time
// Values a workgroup takes.  One round of its lanes: the next workgroup's loads replace its own sooner
// than a loop does (200 M fp32 values: 4 rounds 1093, 2 rounds 1070, one 1026 us; states of 8 bits:
// 443, 416, 388 us).  Two rounds where states are read, all loads before the first store.
constexpr int kStepVals = kBlock * kVals;
constexpr int kReadSteps = 2;
constexpr int kReadVals = kStepVals * kReadSteps;
constexpr int kTensors = 48;                         // descriptors in a launch's arguments
static_assert(TBE_ADAMW_BLOCK == 16 * kVals, "16 lanes share a block");
static_assert(kTensors <= kWave, "one lane a tensor");

struct AdamTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* master;
  uint8_t* ms;
  uint8_t* vs;
  int64_t n;
};
struct AdamArgs {
  AdamTensor t[kTensors];
  float decay[kTensors];      // weight_decay
  int32_t first[kTensors];    // first chunk; those past `count` INT32_MAX
  int32_t count;
  float lr, beta1, beta2, om1, om2, eps;  // om: 1 - beta
  float size, root;           // lr / (1 - beta1^step), 1 / sqrt(1 - beta2^step)
  double dlr, dbeta1, dbeta2; // for a step read from control
  const double* control;
};
static_assert(sizeof(AdamArgs) <= 4096, "kernel arguments");

struct ReadTensor {
  const uint8_t* m;
  const uint8_t* v;
  const uint8_t* ms;
  const uint8_t* vs;
  void* mo;
  void* vo;
  int64_t n;
};
struct ReadArgs {
  ReadTensor t[kTensors];
  int32_t first[kTensors];
  int32_t count;
};
static_assert(sizeof(ReadArgs) <= 4096, "kernel arguments");

// The tensor that owns chunk `chunk`: the last one that starts at or before it.
template <typename A>
__device__ __forceinline__ int tensor_of(const A& a, int chunk) {
  const int l = lane_id();
  const bool at = l < kTensors && a.first[l < kTensors ? l : 0] <= chunk;
  return __popcll(__ballot(at)) - 1;
}

// beta^n for n >= 0
__device__ __forceinline__ double power(double beta, int64_t n) {
  double r = 1.0;
  for (; n > 0; n >>= 1, beta *= beta)
    if (n & 1) r *= beta;
  return r;
}

// Bits of a finite magnitude; an infinity or a NaN does not scale its block (it becomes a NaN code).
__device__ __forceinline__ uint32_t finite_bits(uint32_t u) { return u < 0x7f800000u ? u : 0u; }
// Scale byte of a block from the bits of its largest finite magnitude.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) { return min(max(top >> 23, 24u), 250u); }
__device__ __forceinline__ float unit_of(uint32_t e) { return __uint_as_float(e << 23); }            // 2^(e - 127)
__device__ __forceinline__ float inverse_unit(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// The scale byte of 16 lanes' values x, and whether one of them is an infinity or a NaN.
__device__ __forceinline__ uint32_t block_scale(const float (&x)[kVals], bool& odd) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kVals; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
  top = lanes16_max(top);
  odd = top >= 0x7f800000u;
  if (odd) {  // rare
    top = 0;
#pragma unroll
    for (int i = 0; i < kVals; ++i) top = max(top, finite_bits(__float_as_uint(x[i]) & 0x7fffffffu));
    top = lanes16_max(top);
  }
  return scale_byte(top);
}

__device__ __forceinline__ void open_m(const uint32_t (&c)[2], uint32_t e, float (&m)[kVals]) {
  const float unit = unit_of(e) * 0.0078125f;  // 2^(e - 134): exact, e >= 24 (0 for zeroed bytes)
  typedef float f32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(c[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(c[i], true);
    m[4 * i] = lo.x * unit;
    m[4 * i + 1] = lo.y * unit;
    m[4 * i + 2] = hi.x * unit;
    m[4 * i + 3] = hi.y * unit;
  }
}
__device__ __forceinline__ void open_v(const uint32_t (&c)[2], uint32_t e, float (&v)[kVals]) {
  const float unit = unit_of(e);
#pragma unroll
  for (int i = 0; i < kVals; ++i) {
    const uint32_t k = (c[i / 4] >> (8 * (i % 4))) & 0xffu;
    v[i] = k == 0 ? 0.0f : __uint_as_float((k << 20) + (776u << 20)) * unit;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t t = ~c[i];  // a byte of 255 is a zero byte here
    if ((t - 0x01010101u) & ~t & 0x80808080u) {  // rare: a NaN
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (((c[i] >> (8 * k)) & 0xffu) == 255u) v[4 * i + k] = __uint_as_float(0x7fc00000u);
    }
  }
}
// The conversion makes an infinity a NaN, and a finite value beyond 448 too.  Such are there only where the scale
// byte is at its end: they take the largest code.
__device__ __forceinline__ void pack_m(float (&m)[kVals], uint32_t e, uint32_t (&c)[2]) {
  const float inverse = inverse_unit(e) * 128.0f;  // a power of two: the products are exact, below 256 with e < 250
  if (e == 250u) {  // rare
    constexpr float kMost = 448.0f * 0x1.0p+116f;
#pragma unroll
    for (int i = 0; i < kVals; ++i)
      if (fabsf(m[i]) > kMost && fabsf(m[i]) < __builtin_inff()) m[i] = copysignf(kMost, m[i]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int k = __builtin_amdgcn_cvt_pk_fp8_f32(m[4 * i] * inverse, m[4 * i + 1] * inverse, 0, false);
    k = __builtin_amdgcn_cvt_pk_fp8_f32(m[4 * i + 2] * inverse, m[4 * i + 3] * inverse, k, true);
    c[i] = static_cast<uint32_t>(k);
  }
}
__device__ __forceinline__ void pack_v(const float (&v)[kVals], uint32_t e, bool odd, uint32_t (&c)[2]) {
  const float inverse = inverse_unit(e);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t u = __float_as_uint(v[4 * i + j] * inverse);
      // to three mantissa bits, ties to even, then the exponent counted from 2^-30 / unit on
      const int k = static_cast<int>(u + ((u >> 20) & 1u) + (0x7ffffu - (776u << 20))) >> 20;
      // v itself tells zero: far below its block's largest value (by 2^149), the product is zero too
      uint32_t code = v[4 * i + j] != 0.0f ? static_cast<uint32_t>(min(max(k, 1), 254)) : 0u;
      if (odd && u >= 0x7f800000u) code = 255u;
      word |= code << (8 * j);
    }
    c[i] = word;
  }
}

// With states of 8 bits, sqrt and 1 / x to one unit in the last place: the step's own products and sums round as
// much.  (The correctly rounded ones are 25 more instructions a value, which 10 bytes a value leave no
// time for; states of 32 bits, 22 bytes a value and more, do: 200 M fp32 values 1020 us with either, in bf16
// 802.)  The square root instruction takes numbers below 2^-126 for zero.
__device__ __forceinline__ float root_of(float v) {
  const bool small = v < 0x1.0p-96f;
  return __builtin_amdgcn_sqrtf(small ? v * 0x1.0p+32f : v) * (small ? 0x1.0p-16f : 1.0f);
}

__device__ __forceinline__ void load_codes(const uint8_t* p, int64_t left, uint32_t (&c)[2]) {
  Vec<uint8_t, kVals> b;
  load_vec_part<uint8_t, kVals>(p, left, b);
  __builtin_memcpy(c, b.e, kVals);
}
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t left, const uint32_t (&c)[2]) {
  Vec<uint8_t, kVals> b;
  __builtin_memcpy(b.e, c, kVals);
  store_vec_part<uint8_t, kVals>(p, left, b);
}

// A lane's results, with the streaming policy: nothing of a step is read again before the next
// forward (200 M fp32 values 1148 -> 1093 us, 50 M with master weights 333 -> 300 us).
template <typename S>
__device__ __forceinline__ void store_stream(S* p, int64_t left, const Vec<S, kVals>& v) {
  if (left >= kVals) store_vec_stream<S, kVals>(p, v);
  else store_vec_part<S, kVals>(p, left, v);
}

// S8: states of 8 bits; MASTER: the step is taken on fp32 weights.
template <int PT, int GT, bool S8, bool MASTER>
__global__ __launch_bounds__(kBlock) void adamw_kernel(AdamArgs a) {
  // sums and products each rounded by themselves: the codes then follow from the inputs alone
#pragma clang fp contract(off)
  using PS = typename Fmt<PT>::S;
  using GS = typename Fmt<GT>::S;
  const int which = __builtin_amdgcn_readfirstlane(tensor_of(a, blockIdx.x));
  const AdamTensor& t = a.t[which];
  const int64_t at = static_cast<int64_t>(static_cast<int>(blockIdx.x) - a.first[which]) * kStepVals + threadIdx.x * kVals;
  const int64_t left = t.n - at;
  if (left + kVals * 16 <= 0) return;  // whole blocks past the end; lanes of the last block stay
  Vec<GS, kVals> gr;
  load_vec_part<GS, kVals>(static_cast<const GS*>(t.g) + at, left, gr);
  Vec<float, kVals> w;
  Vec<PS, kVals> pr;
  if constexpr (MASTER) {
    load_vec_part<float, kVals>(t.master + at, left, w);
  } else {
    load_vec_part<PS, kVals>(static_cast<const PS*>(t.p) + at, left, pr);
#pragma unroll
    for (int i = 0; i < kVals; ++i) w.e[i] = Fmt<PT>::to_f(pr.e[i]);
  }
  float m[kVals], v[kVals];
  uint32_t mc[2], vc[2];
  Vec<float, kVals> m32, v32;
  if constexpr (S8) {
    load_codes(static_cast<const uint8_t*>(t.m) + at, left, mc);
    load_codes(static_cast<const uint8_t*>(t.v) + at, left, vc);
    const uint32_t me = left > 0 ? t.ms[at / TBE_ADAMW_BLOCK] : 0, ve = left > 0 ? t.vs[at / TBE_ADAMW_BLOCK] : 0;
    open_m(mc, me, m);
    open_v(vc, ve, v);
  } else {
    load_vec_part<float, kVals>(static_cast<const float*>(t.m) + at, left, m32);
    load_vec_part<float, kVals>(static_cast<const float*>(t.v) + at, left, v32);
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      m[i] = m32.e[i];
      v[i] = v32.e[i];
    }
  }
  // with a control tensor, while the loads are under way
  float size = a.size, root = a.root, lr = a.lr, factor = 1.0f;
  if (a.control) {
    if (a.control[3] != 0.0) return;
    const double dlr = a.dlr * a.control[1];
    const int64_t step = static_cast<int64_t>(a.control[0]);
    lr = static_cast<float>(dlr);
    size = static_cast<float>(dlr / (1.0 - power(a.dbeta1, step)));
    root = static_cast<float>(1.0 / sqrt(1.0 - power(a.dbeta2, step)));
    factor = static_cast<float>(a.control[2]);
  }
  const float keep = 1.0f - lr * a.decay[which];
#pragma unroll
  for (int i = 0; i < kVals; ++i) {
    const float g = Fmt<GT>::to_f(gr.e[i]) * factor;
    m[i] = m[i] * a.beta1 + g * a.om1;
    v[i] = v[i] * a.beta2 + g * g * a.om2;
    if constexpr (S8) w.e[i] = w.e[i] * keep - size * m[i] * __builtin_amdgcn_rcpf(root_of(v[i]) * root + a.eps);
    else w.e[i] = w.e[i] * keep - size * m[i] / (sqrtf(v[i]) * root + a.eps);
  }
  if constexpr (S8) {
    // values past the tensor's end are zeros here: zero moments, gradients and weights
    bool m_odd, v_odd;
    const uint32_t mt = block_scale(m, m_odd), vt = block_scale(v, v_odd);
    pack_m(m, mt, mc);
    pack_v(v, vt, v_odd, vc);
    if (left > 0) {
      store_codes(static_cast<uint8_t*>(t.m) + at, left, mc);
      store_codes(static_cast<uint8_t*>(t.v) + at, left, vc);
      if ((threadIdx.x & 15) == 0) {
        t.ms[at / TBE_ADAMW_BLOCK] = static_cast<uint8_t>(mt);
        t.vs[at / TBE_ADAMW_BLOCK] = static_cast<uint8_t>(vt);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      m32.e[i] = m[i];
      v32.e[i] = v[i];
    }
    store_stream<float>(static_cast<float*>(t.m) + at, left, m32);
    store_stream<float>(static_cast<float*>(t.v) + at, left, v32);
  }
  if constexpr (MASTER) store_stream<float>(t.master + at, left, w);
#pragma unroll
  for (int i = 0; i < kVals; ++i) pr.e[i] = tower_from_f<PT>(w.e[i]);
  store_stream<PS>(static_cast<PS*>(t.p) + at, left, pr);
}

template <int OT>
__global__ __launch_bounds__(kBlock) void adamw_read_kernel(ReadArgs a) {
  using OS = typename Fmt<OT>::S;
  const int which = __builtin_amdgcn_readfirstlane(tensor_of(a, blockIdx.x));
  const ReadTensor& t = a.t[which];
  const int64_t at0 = static_cast<int64_t>(static_cast<int>(blockIdx.x) - a.first[which]) * kReadVals + threadIdx.x * kVals;
  // every load of the chunk is on its way before the first value is stored: 16 bytes a lane and step
  uint32_t mc[kReadSteps][2], vc[kReadSteps][2], me[kReadSteps], ve[kReadSteps];
#pragma unroll
  for (int k = 0; k < kReadSteps; ++k) {
    const int64_t at = at0 + static_cast<int64_t>(k) * kStepVals, left = t.n - at;
    load_codes(t.m + at, left, mc[k]);
    load_codes(t.v + at, left, vc[k]);
    me[k] = left > 0 ? t.ms[at / TBE_ADAMW_BLOCK] : 0;
    ve[k] = left > 0 ? t.vs[at / TBE_ADAMW_BLOCK] : 0;
  }
#pragma unroll
  for (int k = 0; k < kReadSteps; ++k) {
    const int64_t at = at0 + static_cast<int64_t>(k) * kStepVals, left = t.n - at;
    if (left <= 0) return;
    float m[kVals], v[kVals];
    open_m(mc[k], me[k], m);
    open_v(vc[k], ve[k], v);
    Vec<OS, kVals> mo, vo;
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      mo.e[i] = tower_from_f<OT>(m[i]);
      vo.e[i] = tower_from_f<OT>(v[i]);
    }
    store_stream<OS>(static_cast<OS*>(t.mo) + at, left, mo);
    store_stream<OS>(static_cast<OS*>(t.vo) + at, left, vo);
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
bool dtype_ok(int dt) { return dt == TBE_F32 || dt == TBE_F16 || dt == TBE_BF16; }
bool aligned_to(const void* p, int dt) { return !(reinterpret_cast<uintptr_t>(p) & (dt == TBE_F32 ? 3u : 1u)); }

// Kinds of tensors: param type, gradient type, state, master.
int kind_of(const tbe_adamw_tensor& t) {
  return ((t.param_dtype * 3 + t.grad_dtype) * 2 + t.state) * 2 + (t.master ? 1 : 0);
}
constexpr int kKinds = 36;

tbe_status check_tensor(const tbe_adamw_tensor& t, int i) {
  if (!dtype_ok(t.param_dtype) || !dtype_ok(t.grad_dtype) || (t.state != TBE_STATE_F32 && t.state != TBE_STATE_8BIT)) {
    set_error("adamw tensor %d: unknown type or state (param %d, gradient %d, state %d)", i, t.param_dtype, t.grad_dtype, t.state);
    return TBE_ERR_UNSUPPORTED;
  }
  if (t.master && t.param_dtype == TBE_F32) {
    set_error("adamw tensor %d: fp32 master weights go with a param of 16 bits", i);
    return TBE_ERR_UNSUPPORTED;
  }
  if (t.numel < 0 || t.numel > int64_t{1} << 34) {
    set_error("adamw tensor %d: numel %lld", i, static_cast<long long>(t.numel));
    return TBE_ERR_ARG;
  }
  if (t.numel == 0) return TBE_OK;
  const bool eight = t.state == TBE_STATE_8BIT;
  if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq || (eight && (!t.exp_avg_scale || !t.exp_avg_sq_scale))) {
    set_error("adamw tensor %d: a NULL pointer", i);
    return TBE_ERR_ARG;
  }
  if (!aligned_to(t.param, t.param_dtype) || !aligned_to(t.grad, t.grad_dtype) || !aligned_to(t.master, TBE_F32) ||
      (!eight && (!aligned_to(t.exp_avg, TBE_F32) || !aligned_to(t.exp_avg_sq, TBE_F32)))) {
    set_error("adamw tensor %d: a pointer is not aligned to its element", i);
    return TBE_ERR_ARG;
  }
  return TBE_OK;
}

constexpr int64_t kMaxChunks = (int64_t{1} << 24) - 1;

// The launches of one kind: up to kTensors tensors and kMaxChunks chunks each (a launch has fewer
// than 2^32 threads).  add(args, slot, i)
// fills a descriptor, launch(args, chunks) runs what has been gathered.  vals: of a chunk.
template <typename A, typename Add, typename Launch>
tbe_status gather(A& a, const tbe_adamw_tensor* tensors, int count, int kind, int vals, Add add, Launch launch) {
  int64_t chunks = 0;
  a.count = 0;
  for (int i = 0; i <= count; ++i) {
    const bool mine = i < count && tensors[i].numel > 0 && (kind < 0 || kind_of(tensors[i]) == kind);
    const int64_t c = mine ? (tensors[i].numel + vals - 1) / vals : 0;
    if (a.count > 0 && (i == count || a.count == kTensors || chunks + c > kMaxChunks)) {
      for (int k = a.count; k < kTensors; ++k) a.first[k] = 0x7fffffff;
      const tbe_status st = launch(a, static_cast<int>(chunks));
      if (st != TBE_OK) return st;
      a.count = 0;
      chunks = 0;
    }
    if (!mine) continue;
    a.first[a.count] = static_cast<int32_t>(chunks);
    add(a, a.count++, i);
    chunks += c;
  }
  return TBE_OK;
}

template <int PT, int GT, bool S8, bool MASTER>
tbe_status step_launch(const AdamArgs& a, int chunks, hipStream_t s) {
  ProfScope ps("adamw", s);
  hipLaunchKernelGGL((adamw_kernel<PT, GT, S8, MASTER>), dim3(chunks), dim3(kBlock), 0, s, a);
  return check_launch("adamw");
}
template <int PT, int GT>
tbe_status step_types(const AdamArgs& a, int chunks, bool eight, bool master, hipStream_t s) {
  if constexpr (PT != 0) {
    if (master) return eight ? step_launch<PT, GT, true, true>(a, chunks, s) : step_launch<PT, GT, false, true>(a, chunks, s);
  }
  return eight ? step_launch<PT, GT, true, false>(a, chunks, s) : step_launch<PT, GT, false, false>(a, chunks, s);
}
template <int PT>
tbe_status step_param(const AdamArgs& a, int chunks, int gt, bool eight, bool master, hipStream_t s) {
  return gt == 0 ? step_types<PT, 0>(a, chunks, eight, master, s)
                 : gt == 1 ? step_types<PT, 1>(a, chunks, eight, master, s) : step_types<PT, 2>(a, chunks, eight, master, s);
}

}  // namespace
}  // namespace tbe

using namespace tbe;

extern "C" tbe_status tbe_adamw_step(const tbe_adamw_tensor* tensors, int32_t count, int64_t step, double lr, double beta1,
                                     double beta2, double eps, const double* control, tbe_stream_t stream) {
  clear_error();
  if (count < 0 || (count > 0 && !tensors)) {
    set_error("adamw: %d tensors at %p", count, static_cast<const void*>(tensors));
    return TBE_ERR_ARG;
  }
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) || !std::isfinite(lr) ||
      (!control && step < 1)) {
    set_error("adamw: step %lld, lr %g, beta1 %g, beta2 %g, eps %g", static_cast<long long>(step), lr, beta1, beta2, eps);
    return TBE_ERR_ARG;
  }
  if (reinterpret_cast<uintptr_t>(control) & 7) {
    set_error("adamw: control is aligned to its element");
    return TBE_ERR_ARG;
  }
  bool has[kKinds] = {};
  for (int i = 0; i < count; ++i) {
    const tbe_status st = check_tensor(tensors[i], i);
    if (st != TBE_OK) return st;
    if (tensors[i].numel > 0) has[kind_of(tensors[i])] = true;
  }
  AdamArgs a = {};
  a.lr = static_cast<float>(lr);
  a.beta1 = static_cast<float>(beta1);
  a.beta2 = static_cast<float>(beta2);
  a.om1 = static_cast<float>(1.0 - beta1);
  a.om2 = static_cast<float>(1.0 - beta2);
  a.eps = static_cast<float>(eps);
  a.dlr = lr;
  a.dbeta1 = beta1;
  a.dbeta2 = beta2;
  a.control = control;
  if (!control) {
    a.size = static_cast<float>(lr / (1.0 - std::pow(beta1, static_cast<double>(step))));
    a.root = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(beta2, static_cast<double>(step))));
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  for (int kind = 0; kind < kKinds; ++kind) {
    if (!has[kind]) continue;
    const int pt = kind / 12, gt = kind / 4 % 3;
    const bool eight = kind & 2, master = kind & 1;
    const tbe_status st = gather(
        a, tensors, count, kind, kStepVals,
        [&](AdamArgs& x, int slot, int i) {
          const tbe_adamw_tensor& t = tensors[i];
          x.t[slot] = AdamTensor{t.param, t.grad, t.exp_avg, t.exp_avg_sq, t.master, t.exp_avg_scale, t.exp_avg_sq_scale, t.numel};
          x.decay[slot] = t.weight_decay;
        },
        [&](const AdamArgs& x, int chunks) {
          return pt == 0 ? step_param<0>(x, chunks, gt, eight, master, s)
                         : pt == 1 ? step_param<1>(x, chunks, gt, eight, master, s)
                                   : step_param<2>(x, chunks, gt, eight, master, s);
        });
    if (st != TBE_OK) return st;
  }
  return TBE_OK;
}

extern "C" tbe_status tbe_adamw_state_read(const tbe_adamw_tensor* tensors, int32_t count, void* const* exp_avg_out,
                                           void* const* exp_avg_sq_out, int32_t out_dtype, tbe_stream_t stream) {
  clear_error();
  if (count < 0 || (count > 0 && (!tensors || !exp_avg_out || !exp_avg_sq_out))) {
    set_error("adamw state read: %d tensors, a NULL array", count);
    return TBE_ERR_ARG;
  }
  if (out_dtype != TBE_F32 && out_dtype != TBE_BF16) {
    set_error("adamw state read: values go to fp32, where they are exact, or to bf16 (type %d)", out_dtype);
    return TBE_ERR_UNSUPPORTED;
  }
  for (int i = 0; i < count; ++i) {
    const tbe_status st = check_tensor(tensors[i], i);
    if (st != TBE_OK) return st;
    if (tensors[i].state != TBE_STATE_8BIT) {
      set_error("adamw state read: tensor %d has states of 32 bits", i);
      return TBE_ERR_ARG;
    }
    if (tensors[i].numel > 0 && (!exp_avg_out[i] || !exp_avg_sq_out[i] || !aligned_to(exp_avg_out[i], out_dtype) ||
                                 !aligned_to(exp_avg_sq_out[i], out_dtype))) {
      set_error("adamw state read: output %d is NULL or not aligned to its element", i);
      return TBE_ERR_ARG;
    }
  }
  ReadArgs a = {};
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return gather(
      a, tensors, count, -1, kReadVals,
      [&](ReadArgs& x, int slot, int i) {
        const tbe_adamw_tensor& t = tensors[i];
        x.t[slot] = ReadTensor{static_cast<const uint8_t*>(t.exp_avg), static_cast<const uint8_t*>(t.exp_avg_sq), t.exp_avg_scale,
                               t.exp_avg_sq_scale, exp_avg_out[i], exp_avg_sq_out[i], t.numel};
      },
      [&](const ReadArgs& x, int chunks) {
        ProfScope ps("adamw_read", s);
        if (out_dtype == TBE_F32) hipLaunchKernelGGL(adamw_read_kernel<0>, dim3(chunks), dim3(kBlock), 0, s, x);
        else hipLaunchKernelGGL(adamw_read_kernel<2>, dim3(chunks), dim3(kBlock), 0, s, x);
        return check_launch("adamw_read");
      });
}
