/*
 * gptq_tuning.h - C ABI of the operators with which a model of stored layers is tuned and
 * evaluated (AMD Instinct MI355X, gfx950).
 *
 * gptq.h makes a layer's codes, scales and zeros, gptq_serving.h serves them token by token.
 * The operators here take whole batches through stored experts, the gradient back through
 * stored layers, and a stored head's logits to a loss and its gradient.  Stored layers stay
 * as they are: gradients are those of the activations.
 *
 * Conventions: those of gptq_serving.h (device pointers, caller-owned buffers and
 * workspaces, row-major matrices, all work enqueued on `stream` of the current device,
 * nothing allocated, no synchronization, argument errors returned before anything is
 * enqueued; every call can be captured into a graph; no atomics on results, so equal calls
 * give equal bits; calls that may overlap in time share no outputs or workspaces; outputs and
 * workspaces overlap no input and no other output).  Workspace contents on entry are ignored;
 * sizes do not fall as the number of rows grows, so one made for the largest batch serves all
 * smaller ones.  A stored layer is codes, scales_f16 and zeros_f16 as for
 * gptq_quantized_linear, What[r][c] = S (u - z), with bits 3, 4 or 8 and group_size 32, 64,
 * 128, 0 (per row) or -1 (per tensor, as 0).
 */
#ifndef GPTQ_TUNING_MI355X_H
#define GPTQ_TUNING_MI355X_H

#include "gptq.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Products grouped by expert: y[t] = What_e x[t] for the rows t of expert e, offsets[e] <= t <
 * offsets[e + 1].  Products are exact and sums are fp32.  In calls of many rows per expert (more
 * than 160, by sizes alone) bfloat16 elements of x enter as fp16 relative to their row: themselves
 * down to 2^-28 of the row's largest, below that to 2^-39 of it.  A row of x with infinities gives
 * infinities with the weights' signs (NaN where a weight there is zero or the signs differ), one
 * with a NaN gives NaN; others are not touched by it.
 *
 *  codes ..   the experts' rows one after another: n_experts * d_row rows of d_col columns
 *  x          n_rows x d_col, pitch ldx >= d_col, dtype x_dtype: GPTQ_BF16 or GPTQ_F16
 *  offsets    n_experts + 1 int32, or NULL with n_experts == 1: all rows.  Taken clamped to 0 ..
 *             n_rows and to never fall; rows of no expert are left as they were in y.
 *  y          n_rows x d_row, pitch d_row, dtype y_dtype
 *  ws         at least gptqt_linear_grouped_workspace_size(...) bytes, 16-byte aligned; NULL where
 *             that is 0 (few rows per expert)
 * Errors: n_rows < 0, n_experts, d_row or d_col < 1, a pitch below d_col, a group that does not
 * divide d_col, odd d_col with 4-bit codes (3-bit: not a multiple of 8), a bad dtype, a NULL
 * pointer -> GPTQ_ERR_INVALID_ARG; x_dtype GPTQ_F32, bits or group_size not listed, n_rows >
 * 4194240, n_experts > 4096, d_col >= 2^17, ldx > 2^23, d_row > 2^25, n_experts * d_row > 2^26,
 * more than 2^24 tiles of 64 x 128 outputs -> GPTQ_ERR_UNSUPPORTED; a missing, misaligned or short
 * workspace -> GPTQ_ERR_WORKSPACE.  n_rows == 0 is a no-op.
 */
size_t gptqt_linear_grouped_workspace_size(int64_t n_rows, int32_t n_experts, int64_t d_row, int64_t d_col,
                                           int32_t group_size);
gptq_status gptqt_linear_grouped(const uint8_t* codes, const uint16_t* scales_f16, const uint16_t* zeros_f16,
                                 int32_t n_experts, int64_t d_row, int64_t d_col, int32_t bits, int32_t group_size,
                                 const void* x, gptq_dtype x_dtype, int64_t n_rows, int64_t ldx,
                                 const int32_t* offsets, void* y, gptq_dtype y_dtype, void* ws, size_t ws_bytes,
                                 void* stream);

/*
 * The gradient through them: dx[t] = What_e^T dy[t] for the rows t of expert e; with n_experts
 * == 1 and offsets NULL, through any stored layer.  Sums are fp32.  Weights enter in fp16 parts
 * times a power of two that brings their row's largest scale to 16 .. 32 (where zeros beyond 1024
 * need it to 1 .. 2, beyond 32000 to 1/4 .. 1/2): one part, 2^-11 of a weight and 2^-25, where dx
 * is bfloat16; two, 2^-23 of it and 2^-25, where dx is fp16 or fp32.  (A scale of 32 or more may cost
 * the smallest scales of its row their last bits, 2^-25 again.)  Elements of dy are themselves
 * down to 2^-28 of their row's largest (elements taken times their weight row's power of two),
 * below that to 2^-39 of it.  A row of dy with infinities gives infinities with the weights' signs (NaN where a weight
 * there is zero or the signs differ), one with a NaN gives NaN; others are not touched by it.
 *
 *  dy         n_rows x d_row, pitch ld_dy >= d_row, dtype dy_dtype: GPTQ_BF16 or GPTQ_F16
 *  dx         n_rows x d_col, pitch d_col, dtype dx_dtype; rows of no expert are left as they were
 *  ws         at least gptqt_linear_grouped_backward_workspace_size(...) bytes, 16-byte aligned
 * Errors: as gptqt_linear_grouped, but any ld_dy, and tiles of 32 x 128 outputs; a missing,
 * misaligned or short workspace -> GPTQ_ERR_WORKSPACE.
 */
size_t gptqt_linear_grouped_backward_workspace_size(int64_t n_rows, int32_t n_experts, int64_t d_row, int64_t d_col,
                                                    int32_t group_size);
gptq_status gptqt_linear_grouped_backward(const uint8_t* codes, const uint16_t* scales_f16, const uint16_t* zeros_f16,
                                          int32_t n_experts, int64_t d_row, int64_t d_col, int32_t bits,
                                          int32_t group_size, const void* dy, gptq_dtype dy_dtype, int64_t n_rows,
                                          int64_t ld_dy, const int32_t* offsets, void* dx, gptq_dtype dx_dtype,
                                          void* ws, size_t ws_bytes, void* stream);

/*
 * Cross entropy at a stored head, and its gradient, in pieces of the vocabulary: with z = What
 * x[t],
 *   loss[t] = w_t (log sum_v exp z_v - z_target),
 *   dx[t]   = w_t (sum_v softmax(z)_v What_v - What_target)        (the gradient of sum_t loss[t]).
 * A token whose target is outside 0 .. vocab - 1 (by convention -100) or whose weight is 0 is
 * masked: loss and gradient 0, whatever its x holds.
 * Logits are fp32, as gptqt_linear_grouped gives them.  In dx the target's own
 * weight softmax - 1 is fp32; the other words' enter as in gptqt_linear_grouped_backward, the
 * weights in one or two fp16 parts by dx_dtype and exp(z - max) likewise.
 *
 *  codes ..   the head: vocab rows of d columns
 *  x          n_tokens x d, pitch ldx >= d, dtype x_dtype: GPTQ_BF16 or GPTQ_F16
 *  targets    n_tokens int32
 *  weights    n_tokens fp32, or NULL for 1
 *  loss       n_tokens fp32
 *  dx         n_tokens x d, pitch d, dtype dx_dtype; NULL: the loss alone
 *  ws         at least gptqt_cross_entropy_workspace_size(...) bytes (with_grad: dx is not NULL),
 *             16-byte aligned
 * Errors: as gptqt_linear_grouped, vocab for d_row, d for d_col, n_tokens for n_rows, with no limit
 * on tiles (tokens are taken 4096 at a time); an ldx above 2^23 -> GPTQ_ERR_UNSUPPORTED; a missing,
 * misaligned or short workspace -> GPTQ_ERR_WORKSPACE.
 */
size_t gptqt_cross_entropy_workspace_size(int64_t n_tokens, int64_t d, int64_t vocab, int32_t group_size,
                                          int32_t with_grad);
gptq_status gptqt_cross_entropy(const uint8_t* codes, const uint16_t* scales_f16, const uint16_t* zeros_f16,
                                int64_t vocab, int64_t d, int32_t bits, int32_t group_size, const void* x,
                                gptq_dtype x_dtype, int64_t n_tokens, int64_t ldx, const int32_t* targets,
                                const float* weights, float* loss, void* dx, gptq_dtype dx_dtype,
                                void* ws, size_t ws_bytes, void* stream);

/*
 * Distillation from a teacher's top logits at a stored head, and its gradient: with T the
 * temperature, p = softmax(top / T) over the token's entries and q = softmax(What x[t] / T) over
 * the vocabulary,
 *   loss[t] = w_t T^2 sum_j p_j (log p_j - log q_id_j),
 *   dx[t]   = w_t T (sum_v q_v What_v - sum_j p_j What_id_j).
 * An id outside 0 .. vocab - 1 (by convention -1) is no entry, so tokens may have fewer than
 * top_k; one without an entry, with no entry above -infinity, or with weight 0 is masked.  A
 * word may be several entries of a token: its p add up.
 * Precision as gptqt_cross_entropy; q_v - p of the entries' words is fp32.
 *
 *  ids        n_tokens x top_k int32, in any order
 *  top        n_tokens x top_k, dtype top_dtype: the teacher's logits of those words
 * Errors: as gptqt_cross_entropy; top_k < 1, a temperature that is not positive and finite ->
 * GPTQ_ERR_INVALID_ARG; top_k > 1024 -> GPTQ_ERR_UNSUPPORTED.
 */
size_t gptqt_distill_workspace_size(int64_t n_tokens, int64_t d, int64_t vocab, int32_t group_size, int32_t top_k,
                                    int32_t with_grad);
gptq_status gptqt_distill(const uint8_t* codes, const uint16_t* scales_f16, const uint16_t* zeros_f16, int64_t vocab,
                          int64_t d, int32_t bits, int32_t group_size, const void* x, gptq_dtype x_dtype,
                          int64_t n_tokens, int64_t ldx, const int32_t* ids, const void* top, gptq_dtype top_dtype,
                          int32_t top_k, float temperature, const float* weights, float* loss, void* dx,
                          gptq_dtype dx_dtype, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* GPTQ_TUNING_MI355X_H */
