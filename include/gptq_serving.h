/*
 * gptq_serving.h - C ABI of the serving operators around the product on stored codes
 * (AMD Instinct MI355X, gfx950).
 *
 * gptq.h makes a layer's codes, scales and zeros and holds the plain product on them
 * (gptq_quantized_linear).  The operators here stand next to that product when such
 * layers are served: the norm that feeds it with 8-bit rows, the product on 8-bit rows,
 * the product with low-rank adapters of many requests beside it, and a whole
 * mixture-of-experts layer whose experts are stored layers.
 *
 * Conventions: those of gptq.h (device pointers unless said otherwise, caller-owned
 * buffers and workspaces, row-major matrices, all work enqueued on `stream` of the
 * current device, nothing allocated, no synchronization, argument errors returned before
 * anything is enqueued).  Every call can be captured into a graph.  No call uses
 * atomics on results, so equal calls give equal bits.  Calls that may overlap in time
 * must not share outputs or workspaces; graphs that share a workspace must not be
 * replayed at the same time.  Outputs and workspaces overlap no input and no other output,
 * but where a call allows it.  Rows need no alignment; pitches are in elements.
 */
#ifndef GPTQ_SERVING_MI355X_H
#define GPTQ_SERVING_MI355X_H

#include "gptq.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * RMS norm with the residual's addition, written as 8-bit rows with one scale each.
 * For every row, with T = x_dtype:
 *     h     = T(x + residual)                (h = x without a residual)
 *     p_c   = h_c weight_c,  rstd = 1 / sqrt(mean_c h_c^2 + eps)
 *     am    = max_c |p_c|
 *     q_c   = 127 p_c / am rounded to nearest, ties to even
 *     scale = am rstd / 127                  (fp32; 1 when am = 0, and then q = 0)
 * so q_c scale is the normalised value p_c rstd to within half a scale.  rstd cancels
 * from q: for 16-bit x the codes are the exact roundings for these inputs, whatever the
 * order of the sum (fp32 x: of a quotient in 64 bits).  The squares are summed in 64
 * bits.  A row with an infinity or a NaN among its p gets q = 0 and scale = NaN, so that
 * a product on it gives NaN.
 *
 *  x             n_tokens x d, pitch ldx >= d, dtype x_dtype
 *  residual      NULL, or n_tokens x d, pitch ld_residual, dtype x_dtype
 *  weight        d values, dtype w_dtype: x_dtype or GPTQ_F32
 *  residual_out  NULL, or n_tokens x d, pitch ld_residual_out, dtype x_dtype: h
 *  normed        NULL, or n_tokens x d, pitch ld_normed, dtype x_dtype: T(p_c rstd)
 *  q             n_tokens x d int8, pitch ldq
 *  scale         n_tokens fp32
 * residual_out and normed may each be the buffer of x or of residual with its pitch (not
 * both the same one); no other outputs and inputs may overlap.
 * Errors: negative sizes, a pitch below d, eps negative or NaN, a bad dtype, a NULL
 * needed pointer -> GPTQ_ERR_INVALID_ARG; n_tokens > 65535 * 64 = 4194240 or
 * d > 2^30 -> GPTQ_ERR_UNSUPPORTED.  n_tokens == 0 or d == 0 is a no-op.
 */
gptq_status gptqs_rmsnorm_int8(const void* x, gptq_dtype x_dtype, int64_t ldx,
                               const void* residual, int64_t ld_residual,
                               const void* weight, gptq_dtype w_dtype, float eps,
                               int64_t n_tokens, int64_t d,
                               void* residual_out, int64_t ld_residual_out,
                               void* normed, int64_t ld_normed,
                               int8_t* q, int64_t ldq, float* scale, void* stream);

/*
 * The product on stored codes with 8-bit rows:
 *   y[t][r] = x_scale[t] sum_g S16[r][g] sum_{c in g} xq[t][c] (u[r][c] - z[r][g]).
 * The products run on the int8 matrix cores: u - z (u - 128 for 8-bit codes) is taken in
 * 8 bits with z rounded to a whole number in [-112, 127], and what that leaves of z
 * enters as (the rest) * sum_c xq; integer sums are exact, groups are added in fp32.
 *
 *  codes, scales_f16, zeros_f16   as for gptq_quantized_linear: bits 3, 4 or 8,
 *             group_size 32, 64, 128, 0 (per row) or -1 (per tensor, as 0).
 *  xq         n_tokens x d_col int8 (values -128 .. 127), pitch ldx >= d_col.
 *  x_scale    n_tokens fp32.
 *  y          n_tokens x d_row, pitch d_row, dtype y_dtype; written, not read.
 * Errors: as gptq_quantized_linear; another group_size, or more than 2^36 outputs ->
 * GPTQ_ERR_UNSUPPORTED.
 */
gptq_status gptqs_linear_int8(const uint8_t* codes, const uint16_t* scales_f16, const uint16_t* zeros_f16,
                              int64_t d_row, int64_t d_col, int32_t bits, int32_t group_size,
                              const int8_t* xq, int64_t ldx, const float* x_scale, int64_t n_tokens,
                              void* y, gptq_dtype y_dtype, void* stream);

/*
 * A projection on stored codes, shared by all tokens, with a low-rank adapter per token
 * beside it:
 *   y[t] = What x[t] + scaling[a] B[a] (A[a] x[t]),  a = adapter_ids[t];
 * a token whose id is outside 0 .. n_adapters - 1 (by convention -1) takes What x[t]
 * alone.  Tokens may come in any order; runs of tokens with one adapter are cheapest.
 * A x is summed in fp32 and scaling A x enters the second product in fp32, whatever the
 * batch (in large ones as three bfloat16 parts).  An infinite x gives infinities with the weights' signs (NaN where
 * a code is its zero), for every token count where zeros are whole numbers in -240 .. 240;
 * no other token's outputs change.
 *
 *  codes, scales_f16, zeros_f16, d_row, d_col, bits, group_size   as gptqs_linear_int8.
 *  x            n_tokens x d_col, pitch ldx >= d_col, dtype x_dtype: GPTQ_BF16 or GPTQ_F16
 *  A            n_adapters x rank x d_col, dtype x_dtype
 *  B            n_adapters x d_row x rank, dtype x_dtype
 *  adapter_ids  n_tokens int32
 *  scaling      n_adapters fp32, or NULL for 1
 *  y            n_tokens x d_row, pitch d_row, dtype y_dtype
 *  ws           at least gptqs_linear_lora_workspace_size(n_tokens, d_col, rank) bytes,
 *               4-byte aligned; contents on entry are ignored.  The size does not fall as
 *               n_tokens grows: one workspace for the largest batch serves all smaller ones.
 * Errors: as gptqs_linear_int8; x_dtype GPTQ_F32 -> GPTQ_ERR_UNSUPPORTED; rank outside
 * 1 .. 256 or n_adapters < 0 -> GPTQ_ERR_INVALID_ARG; a missing, misaligned or short
 * workspace -> GPTQ_ERR_WORKSPACE.  n_adapters == 0: A, B and ws may be NULL.
 */
size_t gptqs_linear_lora_workspace_size(int64_t n_tokens, int64_t d_col, int32_t rank);
gptq_status gptqs_linear_lora(const uint8_t* codes, const uint16_t* scales_f16, const uint16_t* zeros_f16,
                              int64_t d_row, int64_t d_col, int32_t bits, int32_t group_size,
                              const void* x, gptq_dtype x_dtype, int64_t n_tokens, int64_t ldx,
                              const void* A, const void* B, int32_t n_adapters, int32_t rank,
                              const int32_t* adapter_ids, const float* scaling,
                              void* y, gptq_dtype y_dtype, void* ws, size_t ws_bytes, void* stream);

/*
 * A mixture-of-experts layer for a few tokens, the experts held as stored layers:
 *   l = router x[t];  the top_k experts of largest l (equal ones: the lower index first;
 *   a NaN counts as -infinity), in falling order;
 *   w = softmax of l over all experts at the chosen ones, or with renormalize over the
 *   chosen ones alone;
 *   h_j = silu(G_e x[t]) * (U_e x[t]),  e = the j-th chosen expert;
 *   y[t] = sum_j w_j D_e h_j.
 * Logits, softmax and sums in fp32; w_j h_j enters the last product as it is (fp32, in
 * three bfloat16 parts) where y is fp32, and to 2^-17 of each value (two parts) where y has
 * 16 bits.
 *
 *  x            n_tokens x d, pitch ldx >= d, dtype x_dtype: GPTQ_BF16 or GPTQ_F16
 *  router       n_experts x d, dtype x_dtype
 *  up_*         the gate and up projections as one stored matrix of n_experts * 2 f rows
 *               and d columns: expert e's gate rows 2 f e .. 2 f e + f - 1, then its up rows
 *  down_*       the down projections as one of n_experts * d rows and f columns
 *  bits, group_size   of both, as gptqs_linear_int8 (the group divides d and f)
 *  y            n_tokens x d, pitch d, dtype y_dtype
 *  topk_ids     n_tokens x top_k int32: the chosen experts, in falling order of l
 *  topk_weights n_tokens x top_k fp32: w
 *  ws           at least gptqs_moe_workspace_size(...) bytes, 16-byte aligned; contents on
 *               entry are ignored
 * Errors: negative sizes, top_k outside 1 .. n_experts, a pitch below d, a group that
 * divides d or f not, odd d or f with 4-bit codes (3-bit: not multiples of 8), a bad
 * dtype, a NULL pointer -> GPTQ_ERR_INVALID_ARG; x_dtype GPTQ_F32, bits or group_size not
 * listed, n_tokens > 256, n_experts > 512, top_k > 32, d or f > 2^20 ->
 * GPTQ_ERR_UNSUPPORTED; a missing, misaligned or short workspace -> GPTQ_ERR_WORKSPACE.
 * n_tokens == 0 is a no-op.
 */
size_t gptqs_moe_workspace_size(int64_t n_tokens, int64_t d, int64_t f, int32_t n_experts, int32_t top_k);
gptq_status gptqs_moe(const void* x, gptq_dtype x_dtype, int64_t n_tokens, int64_t d, int64_t ldx,
                      const void* router, int32_t n_experts, int32_t top_k, int32_t renormalize, int64_t f,
                      const uint8_t* up_codes, const uint16_t* up_scales_f16, const uint16_t* up_zeros_f16,
                      const uint8_t* down_codes, const uint16_t* down_scales_f16, const uint16_t* down_zeros_f16,
                      int32_t bits, int32_t group_size, void* y, gptq_dtype y_dtype,
                      int32_t* topk_ids, float* topk_weights, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* GPTQ_SERVING_MI355X_H */
