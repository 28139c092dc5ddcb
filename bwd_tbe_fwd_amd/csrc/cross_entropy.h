// Softmax cross entropy over all items of a table: what its kernels share.  Declarations and the meaning of every argument
// are in include/tbe_items.h.
//
//   l_iv = s (x_i . w_v) + b_v,  lse_i = log sum_v exp l_iv,  loss_i = lse_i - l_it;   p_iv = exp(l_iv - lse_i)
//   z_iv = p_iv - [v = t_i];  dx_i = s g_i sum_v z_iv w_v,  dw_v = s sum_i g_i z_iv x_i,  db_v = sum_i g_i z_iv
//
// The rows that have a target are copied side by side first (their count stays on the device): a batch's padding costs no
// products, and every row starts on 16 bytes.  Weights whose rows do not are copied too, a piece at a time.  Then, with
// C(m, n) = sum_k A(m, k) B(n, k) as in tile_products.h:
//   logits            m = row,  n = item,   k = column: A = x, B = weight, both along
//   gradient of x     m = row,  n = column, k = item:   A = z along, B = weight across
//   of the weights    m = item, n = column, k = row:    A = z across, B = x * grad_loss across
// Forward, the logits' tile ends in each row's maximum and sum of exponentials over the tile's items.  Backward, it ends in
// z, 16 bits each, for a piece of the items: small enough for the Infinity Cache, large enough for its two products.  Rows of
// up to 128 columns have kernels of their own in both directions (cross_entropy_narrow.h, cross_entropy_fused.h).
// z in 16 bits is what the matrix instructions take; the row's loss weight is applied in fp32 to the sums of dx, and to x's copy
// for dw, so that z, between -1 and 1, needs no range of its own (fp16: times 2^15, kUnit).
#pragma once

#include "items.h"

namespace tbe {

// Rows that have a target, in order, and what the kernels need of each.
struct CeRows {
  const int32_t* count;    // of them
  const int32_t* row;      // in the caller's arrays
  const int32_t* target;
  const float* lse;        // backward
  const float* grad;       // backward: grad_loss
  const float* largest;    // backward: of |grad_loss|
  const float* ref;        // backward, narrow rows: -lse in powers of two, -infinity up to a whole 64 rows; for the gradient of
                           // the weights less what |part| is below 1
  const float* part;       // backward, narrow rows: grad_loss over the largest
  const float* far;        // backward, narrow rows: lse where it is past kFar, else 0
};

struct CeArgs {
  int64_t rows;            // of the caller's batch: at least as many as have a target
  int32_t width;           // of x and w as they are read: whole 16 bytes, zeros behind out_width (not for kTile64 through registers)
  int32_t out_width;       // the caller's
  const void* x;           // [count][x_stride], 16 bits
  int64_t x_stride;
  const void* w;           // the piece's first item
  int64_t w_stride;
  const float* bias;       // the piece's; NULL: none; for narrow rows over the scale
  float scale, over;       // over: narrow rows, 1 / scale
  float most;              // what finite biases count as at most
  CeRows r;
  int32_t first, items;    // of the piece
  float2* part;            // forward: [tiles of items][rows] maximum and sum
  uint16_t* z;             // backward: panels of 64 items, each [rows][64], `panel` elements apart
  int64_t panel;
  float* bias_part;        // backward: [tiles or shares of rows][items of the piece]; NULL: none
  int64_t bias_stride;
  // products of z
  const void* xg;          // x * grad_loss / largest, like x
  float* sum;              // [splits][rows or items][sum_pitch] fp32 sums
  int64_t sum_pitch;
  int32_t splits;          // of k; of the items for narrow rows
  int32_t add;             // to what is there
  float factor;            // of a product of z
  void* out;               // gradient of the weights, the piece's first item, with one split
  int64_t out_stride;
};

// z is stored times this, so that fp16 holds probabilities down to 2^-29 as normal numbers.
template <int DT> constexpr float kUnit = DT == 1 ? 32768.0f : 1.0f;

constexpr float kInfinity = __builtin_huge_valf();
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLargest = 3.4028234663852886e38f;  // of all finite ones
// Logits of that size: one times kLog2e is rounded by 2^-10 powers of two, 0.07% of an exponential, and by more the larger it is.
constexpr float kFar = 0x1p14f;
constexpr float kFloor = -1e38f;  // lower logits count as masked where they would overflow as powers of two

// What the backward's exponentials of base 2 add for narrow rows: -lse in powers of two and `shift` more; no probability where
// every item is masked.  lse past kFar is taken off the logits by ce_near instead.
__device__ __forceinline__ bool ce_is_far(float lse) { return fabsf(lse) > kFar && lse != -kInfinity; }
__device__ __forceinline__ float ce_reference(float lse, float shift) {
  return lse == -kInfinity ? -kInfinity : ce_is_far(lse) ? shift : fmaf(lse, -kLog2e, shift);
}
// A logit less lse, both over the scale.  lse is at least the largest rounded product with the scale, so that product is rounded here as
// well: the largest logit's difference is 0 to the bit, and none is above.
__device__ __forceinline__ float ce_near(float product, float scale, float over, float lse) {
#pragma clang fp contract(off)
  const float logit = product * scale, less = logit - lse;
  return (less > 0.0f ? 0.0f : less) * over;
}

// A bias as it counts: finite ones no higher than `most`, the largest value times the scale where that is below 1.  The narrow
// rows' kernels hold biases over the scale, and there is one rule for all widths.
__device__ __forceinline__ float ce_bias(float b, float most) { return b > most && b != kInfinity ? most : b; }
// A finite value's product with the scale or its inverse, at most the largest value.
__device__ __forceinline__ float ce_times(float x, float by) {
  return fabsf(x) == kInfinity ? x : x != x ? x : fminf(fmaxf(x * by, -kLargest), kLargest);
}

// Two parts of a row: their maximum, and the sum of the exponentials less it.
__device__ __forceinline__ float2 ce_join(float2 a, float2 b) {
  const float top = fmaxf(a.x, b.x), from = top == -kInfinity ? 0.0f : top;
  return make_float2(top, a.y * expf(a.x - from) + b.y * expf(b.x - from));
}

// A tile of C and how it is walked, as for the grouped layers; the logits and the gradient of x have one more.
enum { kTile256 = 0, kTile128 = 1, kTile64 = 2, kTile64x256 = 3, kTile256x128 = 3 };

// Defined in translation units of their own (cross_entropy_forward_f16.hip and its siblings).
template <int DT> tbe_status ce_launch_forward(const CeArgs& a, int tile, bool direct, hipStream_t s);
template <int DT> tbe_status ce_launch_z(const CeArgs& a, int tile, hipStream_t s);
template <int DT> tbe_status ce_launch_narrow_forward(const CeArgs& a, bool few, hipStream_t s);
// The gradients of x and of the weights; one of them where the other's splits are 0.
template <int DT> tbe_status ce_launch_fused(const CeArgs& x, const CeArgs& w, hipStream_t s);
template <int DT> tbe_status ce_launch_grads(const CeArgs& x, int x_tile, const CeArgs& w, int w_tile, hipStream_t s);

}  // namespace tbe
