/*
 * tbe_items.h - the two ends of a model that reads and predicts the rows of
 * one table (next item, retrieval, language).
 *
 *   lookup           y_i = scale * table[id_i], one row for each id, and the
 *                    table's dense gradient;
 *   cross entropy    softmax cross entropy of each row over all items of a
 *                    table, without the logits ever being kept, and its
 *                    gradients.
 *
 * Between them stand the operators of tbe_tower.h.  With tied weights the same
 * table is at both ends: the lookup's gradient is then added to the loss's.
 * They follow the conventions of tbe.h and tbe_tower.h: device pointers,
 * caller-owned buffers and workspaces, no allocation, no synchronization, no
 * copy to the host, every kernel on the caller's stream, errors found on the
 * host before anything is launched.  Every result is computed in a fixed
 * order: the same inputs give the same bits.  Sizes and strides are in
 * elements.  Element pointers need the alignment of their element type only;
 * larger alignment (16 bytes, rows that start on it) is faster.  A workspace
 * may be used by any number of calls that follow each other on one stream, and
 * holds nothing between calls; calls that may run at the same time (two
 * streams, two captured graphs) need one each.  Outputs must not overlap
 * inputs or each other.
 */
#ifndef TBE_ITEMS_H_
#define TBE_ITEMS_H_

#include "tbe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * y [ids][width] with rows y_stride apart: y_i = scale * table[id_i], rounded
 * once to y's type; zero for an id outside [0, items) (padding).  table is
 * [items][width] with rows table_stride apart; table and y may have different
 * types.  0 <= num_ids <= TBE_MAX_LOOKUPS, 1 <= items < 2^31 - 1,
 * 1 <= width <= TBE_ITEMS_MAX_WIDTH, rows at most 2^31 elements apart.
 */
#define TBE_ITEMS_MAX_WIDTH (1 << 20)
tbe_status tbe_lookup_forward(int64_t num_ids, int64_t items, int64_t width, const void* table,
                              int64_t table_stride, int32_t table_dtype, const void* ids,
                              int32_t id_type, float scale, void* y, int64_t y_stride,
                              int32_t y_dtype, tbe_stream_t stream);

/*
 * The table's gradient: row v of grad_table [items][width] becomes
 * scale * (sum of grad_y_i over the i with id_i = v), zero where there is none
 * (accumulate = 0), or has it added (accumulate = 1: rows that no id names are
 * neither read nor written).  The sum is kept in fp32 over the positions in
 * their order, with the row that it is added to, and rounded once.  ids
 * outside [0, items) contribute nothing, whatever their grad_y holds.
 * grad_y, grad_table and the table may have different types.  workspace: at
 * least tbe_lookup_backward_workspace_bytes bytes, 256-byte aligned; the bytes
 * grow with the ids, so one for the largest batch serves every smaller one.
 */
size_t tbe_lookup_backward_workspace_bytes(int64_t num_ids, int64_t items, int64_t width);
tbe_status tbe_lookup_backward(int64_t num_ids, int64_t items, int64_t width, const void* ids,
                               int32_t id_type, const void* grad_y, int64_t grad_y_stride,
                               int32_t y_dtype, float scale, void* grad_table,
                               int64_t grad_table_stride, int32_t table_dtype, int32_t accumulate,
                               void* workspace, size_t workspace_bytes, tbe_stream_t stream);

/*
 * Softmax cross entropy of each row over all items.  x is [rows][width] with
 * rows x_stride apart, weight [items][width] with rows weight_stride apart,
 * both of one type, dtype: fp16 or bf16; bias [items] fp32 may be NULL (0).
 *   logit_iv = scale * (x_i . weight_v) + bias_v
 *   lse_i    = log (sum over v of exp logit_iv)
 *   loss_i   = lse_i - logit_{i, target_i}
 * loss and lse [rows] are fp32.  A row whose target lies outside [0, items) is
 * left out: its loss and lse are 0 and its x is not looked at.  An item whose
 * bias is -infinity is masked: its probability is 0, and the loss of a row
 * with such a target is +infinity; a row with every item masked has lse
 * -infinity.  A row with an infinity or a NaN gives NaN (or an infinity) in
 * that row only.  scale is 0 or from 2^-64 to 2^64, of either sign.  Biases of
 * the lowest value mask an item beside others that are not masked.  Where |scale|
 * is below 1, finite biases count as the largest value times |scale| at most, in
 * the target's logit too; items with biases below the lowest value times |scale|
 * are not told apart by rows of up to 128 columns, and where a row has no others
 * its lse is the target's logit.  Products, logits, maxima and sums are kept in
 * fp32.  Logits that are so large that fp32 has no digits behind their point have
 * the probabilities of the rounded logits: the largest one's is 1 where no other
 * is near.  Losses are not below 0.  The logits go through registers, a tile of
 * items at a time, and are never stored.  rows may be 0 and at most
 * TBE_CROSS_ENTROPY_MAX_ROWS; 1 <= items < 2^31 - 1; 1 <= width <=
 * TBE_CROSS_ENTROPY_MAX_WIDTH.  workspace: at least
 * tbe_cross_entropy_forward_workspace_bytes bytes, 256-byte aligned; the bytes
 * grow with the rows, so one for the largest batch serves every smaller one.
 */
#define TBE_CROSS_ENTROPY_MAX_ROWS (1 << 22)
#define TBE_CROSS_ENTROPY_MAX_WIDTH (1 << 16)
size_t tbe_cross_entropy_forward_workspace_bytes(int64_t rows, int64_t items, int64_t width);
tbe_status tbe_cross_entropy_forward(int64_t rows, int64_t items, int64_t width, const void* x,
                                     int64_t x_stride, const void* weight, int64_t weight_stride,
                                     int32_t dtype, const float* bias, const void* targets,
                                     int32_t target_type, float scale, float* loss, float* lse,
                                     void* workspace, size_t workspace_bytes, tbe_stream_t stream);

/*
 * Backward of tbe_cross_entropy_forward, with its inputs and its lse.  With
 *   z_iv = grad_loss_i * (exp(logit_iv - lse_i) - [v = target_i])
 * for the rows that have a target and 0 for the others,
 *   grad_x_i      = scale * sum over v of z_iv weight_v
 *   grad_weight_v = scale * sum over i of z_iv x_i
 *   grad_bias_v   = sum over i of z_iv.
 * Any of the three may be NULL.  grad_x and grad_weight are of type dtype with
 * strides of their own, grad_bias [items] is fp32; all are overwritten (zeros
 * for rows without a target).  The logits are computed again, a piece of the
 * items at a time.  exp(...) - [...] is rounded to dtype for its two products,
 * as x times grad_loss over the largest |grad_loss| is (exactly x where all
 * are equal); rows of up to 128 columns have exp(...) - [...] times grad_loss
 * over the largest rounded instead for the weights' gradient.  Sums are kept in
 * fp32 and rounded once.  In fp16 probabilities keep their digits down to
 * 2^-29, and the weights' gradient those of rows whose |grad_loss| is not below
 * 2^-14 of the largest.
 */
size_t tbe_cross_entropy_backward_workspace_bytes(int64_t rows, int64_t items, int64_t width);
tbe_status tbe_cross_entropy_backward(int64_t rows, int64_t items, int64_t width, const void* x,
                                      int64_t x_stride, const void* weight, int64_t weight_stride,
                                      int32_t dtype, const float* bias, const void* targets,
                                      int32_t target_type, float scale, const float* lse,
                                      const float* grad_loss, void* grad_x, int64_t grad_x_stride,
                                      void* grad_weight, int64_t grad_weight_stride,
                                      float* grad_bias, void* workspace, size_t workspace_bytes,
                                      tbe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TBE_ITEMS_H_ */
