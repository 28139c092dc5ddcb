// Device-side helpers of the dense tower's kernels (gfx950, wave64): vectors at element
// alignment, sums over lanes without LDS, 16-bit storage formats.
#pragma once

#include "tbe_device.h"

namespace tbe {

// Rounded to nearest even (v_cvt_pk_bf16_f32 / v_cvt_f16_f32); NaN stays NaN.
template <int DT>
__device__ __forceinline__ typename Fmt<DT>::S tower_from_f(float x) {
  if constexpr (DT == 2) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
  else return Fmt<DT>::from_f(x);
}

// N elements at any element alignment as one access: global loads and stores of up to 16 bytes
// need no alignment on gfx950 beyond the element's.  An odd row pitch so costs some accesses
// that cross a cache line, not a scalar loop.
template <typename S, int N>
struct Vec {
  S e[N];
};
template <typename S, int N>
__device__ __forceinline__ void load_vec_any(const S* p, Vec<S, N>& v) {
  constexpr int kPart = 16 / static_cast<int>(sizeof(S)) < N ? 16 / static_cast<int>(sizeof(S)) : N;
#pragma unroll
  for (int i = 0; i < N; i += kPart) __builtin_memcpy(&v.e[i], p + i, kPart * sizeof(S));
}
template <typename S, int N>
__device__ __forceinline__ void store_vec_any(S* p, const Vec<S, N>& v) {
  constexpr int kPart = 16 / static_cast<int>(sizeof(S)) < N ? 16 / static_cast<int>(sizeof(S)) : N;
#pragma unroll
  for (int i = 0; i < N; i += kPart) __builtin_memcpy(p + i, &v.e[i], kPart * sizeof(S));
}
// Same with the streaming cache policy, 16 bytes at a time: for results that nothing reads back soon.
template <typename S, int N>
__device__ __forceinline__ void store_vec_stream(S* p, const Vec<S, N>& v) {
  typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
  static_assert(N * sizeof(S) % 16 == 0, "whole 16 bytes");
#pragma unroll
  for (int i = 0; i < N; i += 16 / static_cast<int>(sizeof(S))) {
    u32x4_any x;
    __builtin_memcpy(&x, &v.e[i], 16);
    __builtin_nontemporal_store(x, reinterpret_cast<u32x4_any*>(p + i));
  }
}
// The first `left` of N elements (all of them where left >= N); the others are zero.
template <typename S, int N>
__device__ __forceinline__ void load_vec_part(const S* p, int64_t left, Vec<S, N>& v) {
  if (left >= N) {
    load_vec_any<S, N>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v.e[i] = i < left ? p[i] : S(0);
  }
}
template <typename S, int N>
__device__ __forceinline__ void store_vec_part(S* p, int64_t left, const Vec<S, N>& v) {
  if (left >= N) {
    store_vec_any<S, N>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < left) p[i] = v.e[i];
  }
}

// One element of a runtime tbe_dtype, for vectors that every row shares (scales, shifts, biases
// and their gradients).
__device__ __forceinline__ float load_any(const void* p, int dt, int64_t i) {
  if (dt == 0) return static_cast<const float*>(p)[i];
  const uint16_t h = static_cast<const uint16_t*>(p)[i];
  return dt == 1 ? Fmt<1>::to_f(h) : Fmt<2>::to_f(h);
}
__device__ __forceinline__ void store_any(void* p, int dt, int64_t i, float v) {
  if (dt == 0) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = dt == 1 ? tower_from_f<1>(v) : tower_from_f<2>(v);
}

template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
  return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(v), CTRL, 0xf, 0xf, false));
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
  return __builtin_amdgcn_mov_dpp(v, CTRL, 0xf, 0xf, false);
}
// lane xor 1, xor 2, mirror of 8, mirror of 16: together every lane of a row of 16
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

// Sum over aligned groups of G lanes (16 or 64), the same bits in every lane.
template <int G>
__device__ __forceinline__ float lanes_sum(float v) {
  static_assert(G == 16 || G == 64, "groups of 16 or 64 lanes");
  v += dpp_f<kDppXor1>(v);
  v += dpp_f<kDppXor2>(v);
  v += dpp_f<kDppHalfMirror>(v);
  v += dpp_f<kDppMirror>(v);
  if constexpr (G == 64) {
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
  }
  return v;
}
__device__ __forceinline__ uint32_t lanes16_max(uint32_t v) {
  v = max(v, dpp_u<kDppXor1>(v));
  v = max(v, dpp_u<kDppXor2>(v));
  v = max(v, dpp_u<kDppHalfMirror>(v));
  return max(v, dpp_u<kDppMirror>(v));
}

}  // namespace tbe
