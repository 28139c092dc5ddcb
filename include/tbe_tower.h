/*
 * tbe_tower.h - operators of the dense tower above the pooled embeddings.
 *
 * A model that trains its tables with tbe.h feeds the pooled output
 * (B x sum_t D_t, fp32) to a dense tower.  These are the tower's operators:
 *
 *   layer norm       y = (x - mean) * rstd * weight + bias per row, and its
 *                    backward with the weight's and bias's gradients;
 *   grouped linear   y_i = W_e x_i + b_e for rows grouped by expert e (one
 *                    expert per market, domain or routed group), and its
 *                    backward by input and by weight;
 *   AdamW            one step over all the tower's tensors, with states of
 *                    32 or of 8 bits.
 *
 * They follow the conventions of tbe.h: device pointers unless marked [host],
 * caller-owned buffers and workspaces, no allocation, no synchronization, no
 * copy to the host, every kernel on the caller's stream, errors found on the
 * host before anything is launched and returned as a tbe_status with
 * tbe_last_error().  Every result is computed in a fixed order: the same
 * inputs give the same bits.  Sizes and strides are in elements.  Element
 * pointers need the alignment of their element type only; larger alignment
 * (16 bytes, rows that start on it) is faster.
 */
#ifndef TBE_TOWER_H_
#define TBE_TOWER_H_

#include "tbe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Layer norm over the last dimension.  x is [rows][width] with rows x_stride
 * elements apart (x_stride >= width), y the same with y_stride; x and y may
 * have different types (fp32 pooled rows into a bf16 tower), and y may be x
 * when they have one type and stride.  mean = sum x / width and
 * rstd = 1 / sqrt(sum (x - mean)^2 / width + eps) are taken in fp32, the
 * squares after the mean is known; a mean far from zero is corrected by the
 * deviations' sum, so a row of equal values gives exactly its bias (eps > 0,
 * up to 2^22 wide; beyond, to a unit of the mean's last place).  weight and
 * bias [width] of type w_dtype may each be NULL (1 and 0).  mean and rstd
 * [rows] fp32 may be NULL where no backward follows.  A row with an infinity
 * or a NaN gives NaN in that row only.  eps >= 0.  1 <= width <=
 * TBE_LAYER_NORM_MAX_WIDTH; rows may be 0 and at most 2^31 - 1, at most 2^31
 * elements apart.
 */
#define TBE_LAYER_NORM_MAX_WIDTH (1 << 24)
tbe_status tbe_layer_norm_forward(int64_t rows, int64_t width, const void* x, int64_t x_stride,
                                  int32_t x_dtype, const void* weight, const void* bias,
                                  int32_t w_dtype, float eps, void* y, int64_t y_stride,
                                  int32_t y_dtype, float* mean, float* rstd, tbe_stream_t stream);

/*
 * Backward of tbe_layer_norm_forward: with h = (x - mean) * rstd and
 * d = grad_y * weight,
 *   grad_x      = rstd * (d - sum d / width - h * sum (d * h) / width)
 *   grad_weight = sum over rows of grad_y * h,  grad_bias = sum of grad_y.
 * x and mean / rstd are the forward's; grad_y has its own type and stride,
 * grad_x is of x's type with its own stride.  Any of grad_x, grad_weight and
 * grad_bias may be NULL; grad_weight and grad_bias [width] are of type
 * w_dtype and are overwritten (zeros for no rows).  Their sums are kept in
 * fp32, first over each workgroup's rows, then over the workgroups in their
 * order.  workspace: at least tbe_layer_norm_backward_workspace_bytes(rows,
 * width) bytes, 256-byte aligned; it is not read where both are NULL.
 */
size_t tbe_layer_norm_backward_workspace_bytes(int64_t rows, int64_t width);
tbe_status tbe_layer_norm_backward(int64_t rows, int64_t width, const void* x, int64_t x_stride,
                                   int32_t x_dtype, const void* grad_y, int64_t grad_y_stride,
                                   int32_t y_dtype, const float* mean, const float* rstd,
                                   const void* weight, int32_t w_dtype, void* grad_x,
                                   int64_t grad_x_stride, void* grad_weight, void* grad_bias,
                                   void* workspace, size_t workspace_bytes, tbe_stream_t stream);

/*
 * Linear layers of E experts on rows grouped by expert.  x is [rows][inner]
 * with rows x_stride apart, weight [E][outer][inner] contiguous, bias
 * [E][outer] or NULL.  offsets [E+1] (offset_type) lies on the device:
 * expert e owns rows offsets[e] .. offsets[e+1]; offsets[0] is 0, they do not
 * decrease, and offsets[E] <= rows.  Rows from offsets[E] on belong to no
 * expert (a batch padded to its capacity) and their y is zero, whatever x
 * holds there.  Other offsets give undefined results, but every access stays
 * inside the buffers.  x, weight, bias and grad_y have one type, dtype: fp16
 * or bf16; y and the gradients are of out_dtype: dtype or fp32.  Products are
 * summed in fp32 and rounded once.  E, inner, outer >= 1; rows may be 0 and
 * at most 2^29; inner and outer at most 2^20, E at most 65535, rows at most
 * 2^31 elements apart.  Sizes whose 256 x 256 tiles (by weight: of every
 * expert, elsewhere of those that have rows) are 2^23 and more are refused
 * with TBE_ERR_UNSUPPORTED.
 */
tbe_status tbe_grouped_linear_forward(int64_t rows, int32_t experts, int64_t inner, int64_t outer,
                                      const void* x, int64_t x_stride, const void* weight,
                                      const void* bias, int32_t dtype, const void* offsets,
                                      int32_t offset_type, void* y, int64_t y_stride,
                                      int32_t out_dtype, tbe_stream_t stream);

/* grad_x_i = W_e^T grad_y_i; zero for rows of no expert. */
tbe_status tbe_grouped_linear_backward_input(int64_t rows, int32_t experts, int64_t inner,
                                             int64_t outer, const void* grad_y,
                                             int64_t grad_y_stride, const void* weight,
                                             int32_t dtype, const void* offsets,
                                             int32_t offset_type, void* grad_x,
                                             int64_t grad_x_stride, int32_t out_dtype,
                                             tbe_stream_t stream);

/*
 * grad_weight_e [outer][inner] = sum over expert e's rows of grad_y_i x_i^T
 * and grad_bias_e [outer] = sum of grad_y_i (NULL: not computed), both
 * overwritten, zero for an expert without rows, in out_dtype.  workspace: at
 * least tbe_grouped_linear_backward_weight_workspace_bytes bytes, 256-byte
 * aligned (0 below 512 rows: then workspace may be NULL).  The bytes grow with
 * the rows, so a workspace for the largest batch serves every smaller one, and
 * are at most 1 GiB, or an eighth of x and grad_y where that is more.
 */
size_t tbe_grouped_linear_backward_weight_workspace_bytes(int64_t rows, int32_t experts,
                                                          int64_t inner, int64_t outer);
tbe_status tbe_grouped_linear_backward_weight(int64_t rows, int32_t experts, int64_t inner,
                                              int64_t outer, const void* x, int64_t x_stride,
                                              const void* grad_y, int64_t grad_y_stride,
                                              int32_t dtype, const void* offsets,
                                              int32_t offset_type, void* grad_weight,
                                              void* grad_bias, int32_t out_dtype, void* workspace,
                                              size_t workspace_bytes, tbe_stream_t stream);

/*
 * AdamW.  One tensor of the step; all pointers are device pointers.
 *
 * With states of 8 bits (state = TBE_STATE_8BIT), exp_avg and exp_avg_sq hold
 * one byte per value and each TBE_ADAMW_BLOCK values of a tensor (the last
 * block may be shorter) share one byte of exp_avg_scale / exp_avg_sq_scale:
 * the biased exponent s of the block's largest finite magnitude, at least 24
 * and at most 250.  A first moment is an e4m3 number times 2^(s - 134).  A second
 * moment c is an unsigned number of 5 exponent and 3 mantissa bits: 0 for
 * c = 0, NaN for c = 255, else the fp32 number with bits (c + 776) << 20,
 * times 2^(s - 127): 30 powers of two below the block's largest.  Finite
 * values beyond the largest code's at s = 250, 448 * 2^116 and 3.5 * 2^123,
 * take that code.  Both round to nearest, ties to even; a second moment
 * above zero never becomes zero, so that no later step divides by eps alone.
 * An infinity or a NaN becomes a NaN and leaves its block's other values as
 * they are.  Zeroed bytes are zero states.
 */
#define TBE_ADAMW_BLOCK 128
typedef enum { TBE_STATE_F32 = 0, TBE_STATE_8BIT = 1 } tbe_adamw_state;
typedef struct {
  void* param;             /* param_dtype, updated */
  const void* grad;        /* grad_dtype */
  void* exp_avg;           /* fp32, or codes */
  void* exp_avg_sq;
  float* master;           /* fp32 weights that the step is taken on, param becomes their rounded
                              copy; NULL: the step is taken on param itself */
  uint8_t* exp_avg_scale;  /* ceil(numel / TBE_ADAMW_BLOCK) bytes with states of 8 bits, else unused */
  uint8_t* exp_avg_sq_scale;
  int64_t numel;           /* may be 0, at most 2^34 */
  float weight_decay;      /* of this tensor */
  int32_t param_dtype, grad_dtype; /* tbe_dtype */
  int32_t state;           /* tbe_adamw_state */
} tbe_adamw_tensor;

/*
 * One step on every tensor of tensors [host, count entries]; tensors must
 * not overlap.  In fp32, each operation rounded by itself (so that the moments
 * and their codes are the same on any machine), but with states of 8 bits the
 * weight's square root and division are good to one unit in the last place:
 *   m = beta1 * m + (1 - beta1) * g
 *   v = beta2 * v + (1 - beta2) * (g * g)
 *   p = p * (1 - lr * weight_decay)
 *       - lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * The update uses m and v before they are rounded to 8 bits.  step counts
 * from 1.  control [device, TBE_ADAMW_CONTROL doubles] may be NULL; otherwise
 * control[0] takes the place of step, control[1] is a factor of lr,
 * control[2] a factor of every gradient (the inverse loss scale times a
 * clipping factor), and where control[3] is not zero nothing is written: a
 * captured graph then steps with values that change from replay to replay.
 * 0 <= beta1, beta2 < 1, eps >= 0.
 */
#define TBE_ADAMW_CONTROL 4
tbe_status tbe_adamw_step(const tbe_adamw_tensor* tensors, int32_t count, int64_t step, double lr,
                          double beta1, double beta2, double eps, const double* control,
                          tbe_stream_t stream);

/*
 * The values of states of 8 bits: exp_avg_out[i] and exp_avg_sq_out[i]
 * [host arrays of count device pointers, out_dtype fp32 or bf16] receive
 * tensor i's numel values.  fp32 holds them exactly, bf16 from 2^-126 on;
 * smaller second moments (of blocks with s below 31) are rounded to bf16's
 * nearest, and none above zero becomes zero.  Every tensor must have
 * states of 8 bits.
 */
tbe_status tbe_adamw_state_read(const tbe_adamw_tensor* tensors, int32_t count,
                                void* const* exp_avg_out, void* const* exp_avg_sq_out,
                                int32_t out_dtype, tbe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TBE_TOWER_H_ */
