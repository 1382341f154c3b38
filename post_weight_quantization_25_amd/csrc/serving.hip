// C ABI of the serving operators: argument validation, workspace sizing and dispatch.
// See include/gptq_serving.h for the contract.

#include "common.h"
#include "serving.h"

using namespace gptq;

static bool valid_dtype(gptq_dtype t) { return t == GPTQ_F32 || t == GPTQ_BF16 || t == GPTQ_F16; }

// Settings of a stored layer that the serving products take; group -1 (per tensor) becomes 0.
static gptq_status check_stored(int64_t d_col, int32_t bits, int32_t& group) {
    if (group == -1) group = 0;
    if (group < 0) return GPTQ_ERR_INVALID_ARG;
    if (bits != 3 && bits != 4 && bits != 8) return GPTQ_ERR_UNSUPPORTED;
    if (group > 0 && d_col % group != 0) return GPTQ_ERR_INVALID_ARG;
    if (group != 0 && group != 32 && group != 64 && group != 128) return GPTQ_ERR_UNSUPPORTED;
    if (bits <= 4 && (d_col & 1)) return GPTQ_ERR_INVALID_ARG;
    if (bits == 3 && (d_col & 7)) return GPTQ_ERR_INVALID_ARG;
    return GPTQ_OK;
}

#pragma GCC visibility push(default)
extern "C" {

gptq_status gptqs_rmsnorm_int8(const void* x, gptq_dtype x_dtype, int64_t ldx, const void* residual,
                               int64_t ld_residual, const void* weight, gptq_dtype w_dtype, float eps,
                               int64_t n_tokens, int64_t d, void* residual_out, int64_t ld_residual_out,
                               void* normed, int64_t ld_normed, int8_t* q, int64_t ldq, float* scale, void* stream) {
    if (n_tokens < 0 || d < 0 || !(eps >= 0.f)) return GPTQ_ERR_INVALID_ARG;
    if (!valid_dtype(x_dtype) || (w_dtype != x_dtype && w_dtype != GPTQ_F32)) return GPTQ_ERR_INVALID_ARG;
    if (n_tokens == 0 || d == 0) return GPTQ_OK;
    if (!x || !weight || !q || !scale || ldx < d || ldq < d) return GPTQ_ERR_INVALID_ARG;
    if ((residual && ld_residual < d) || (residual_out && ld_residual_out < d) || (normed && ld_normed < d))
        return GPTQ_ERR_INVALID_ARG;
    if (residual_out && residual_out == normed) return GPTQ_ERR_INVALID_ARG;
    if (n_tokens > SERVE_MAX_TOKENS || d > ((int64_t)1 << 30)) return GPTQ_ERR_UNSUPPORTED;
    NormArgs a;
    a.x = x; a.ldx = ldx; a.r = residual; a.ldr = ld_residual; a.w = weight; a.eps = eps;
    a.n = n_tokens; a.d = d; a.h = residual_out; a.ldh = ld_residual_out; a.y = normed; a.ldy = ld_normed;
    a.q = q; a.ldq = ldq; a.scale = scale;
    return norm_launch(a, x_dtype, w_dtype, (hipStream_t)stream);
}

gptq_status gptqs_linear_int8(const uint8_t* codes, const uint16_t* scales_f16, const uint16_t* zeros_f16,
                              int64_t d_row, int64_t d_col, int32_t bits, int32_t group_size, const int8_t* xq,
                              int64_t ldx, const float* x_scale, int64_t n_tokens, void* y, gptq_dtype y_dtype,
                              void* stream) {
    if (d_row < 0 || d_col < 0 || n_tokens < 0 || !valid_dtype(y_dtype)) return GPTQ_ERR_INVALID_ARG;
    const gptq_status st = check_stored(d_col, bits, group_size);
    if (st != GPTQ_OK) return st;
    if (d_row == 0 || d_col == 0 || n_tokens == 0) return GPTQ_OK;
    if (!codes || !scales_f16 || !zeros_f16 || !xq || !x_scale || !y || ldx < d_col) return GPTQ_ERR_INVALID_ARG;
    if (d_row > 2147483647LL / 64 || d_col > 2147483647LL / 64 || n_tokens > SERVE_MAX_TOKENS ||
        d_row > SERVE_MAX_OUTPUTS / n_tokens)
        return GPTQ_ERR_UNSUPPORTED;
    return linear_int8_launch(codes, scales_f16, zeros_f16, d_row, d_col, bits, group_size, xq, ldx, x_scale, n_tokens,
                              y, y_dtype, (hipStream_t)stream);
}

size_t gptqs_linear_lora_workspace_size(int64_t n_tokens, int64_t d_col, int32_t rank) {
    if (n_tokens <= 0 || d_col <= 0 || rank < 1 || rank > LORA_MAX_RANK) return 0;
    return lora_ws_bytes(n_tokens, d_col, rank);
}

gptq_status gptqs_linear_lora(const uint8_t* codes, const uint16_t* scales_f16, const uint16_t* zeros_f16,
                              int64_t d_row, int64_t d_col, int32_t bits, int32_t group_size, const void* x,
                              gptq_dtype x_dtype, int64_t n_tokens, int64_t ldx, const void* A, const void* B,
                              int32_t n_adapters, int32_t rank, const int32_t* adapter_ids, const float* scaling,
                              void* y, gptq_dtype y_dtype, void* ws, size_t ws_bytes, void* stream) {
    if (d_row < 0 || d_col < 0 || n_tokens < 0 || !valid_dtype(x_dtype) || !valid_dtype(y_dtype))
        return GPTQ_ERR_INVALID_ARG;
    if (n_adapters < 0 || (n_adapters > 0 && (rank < 1 || rank > LORA_MAX_RANK))) return GPTQ_ERR_INVALID_ARG;
    const gptq_status st = check_stored(d_col, bits, group_size);
    if (st != GPTQ_OK) return st;
    if (x_dtype == GPTQ_F32) return GPTQ_ERR_UNSUPPORTED;
    if (d_row == 0 || d_col == 0 || n_tokens == 0) return GPTQ_OK;
    if (!codes || !scales_f16 || !zeros_f16 || !x || !y || ldx < d_col) return GPTQ_ERR_INVALID_ARG;
    if (n_adapters > 0 && (!A || !B || !adapter_ids)) return GPTQ_ERR_INVALID_ARG;
    if (d_row > 2147483647LL / 64 || d_col > 2147483647LL / 64 || n_tokens > SERVE_MAX_TOKENS ||
        d_row > SERVE_MAX_OUTPUTS / n_tokens)
        return GPTQ_ERR_UNSUPPORTED;
    if (n_adapters > 0 && (!ws || (reinterpret_cast<uintptr_t>(ws) & 3) || ws_bytes < lora_ws_bytes(n_tokens, d_col, rank)))
        return GPTQ_ERR_WORKSPACE;
    return linear_lora_launch(codes, scales_f16, zeros_f16, d_row, d_col, bits, group_size, x, x_dtype, n_tokens, ldx,
                              A, B, n_adapters, rank, adapter_ids, scaling, y, y_dtype, ws, (hipStream_t)stream);
}

size_t gptqs_moe_workspace_size(int64_t n_tokens, int64_t d, int64_t f, int32_t n_experts, int32_t top_k) {
    if (n_tokens <= 0 || d <= 0 || f <= 0 || n_experts < 1 || top_k < 1 || top_k > n_experts) return 0;
    if (n_tokens > MOE_MAX_TOKENS || n_experts > MOE_MAX_EXPERTS || top_k > MOE_MAX_TOPK || d > MOE_MAX_WIDTH ||
        f > MOE_MAX_WIDTH)
        return 0;
    return moe_ws_bytes(n_tokens, d, f, n_experts, top_k);
}

gptq_status gptqs_moe(const void* x, gptq_dtype x_dtype, int64_t n_tokens, int64_t d, int64_t ldx, const void* router,
                      int32_t n_experts, int32_t top_k, int32_t renormalize, int64_t f, const uint8_t* up_codes,
                      const uint16_t* up_scales_f16, const uint16_t* up_zeros_f16, const uint8_t* down_codes,
                      const uint16_t* down_scales_f16, const uint16_t* down_zeros_f16, int32_t bits,
                      int32_t group_size, void* y, gptq_dtype y_dtype, int32_t* topk_ids, float* topk_weights, void* ws,
                      size_t ws_bytes, void* stream) {
    if (n_tokens < 0 || d < 1 || f < 1 || !valid_dtype(x_dtype) || !valid_dtype(y_dtype)) return GPTQ_ERR_INVALID_ARG;
    if (n_experts < 1 || top_k < 1 || top_k > n_experts || ldx < d) return GPTQ_ERR_INVALID_ARG;
    int32_t group = group_size;
    gptq_status st = check_stored(d, bits, group);
    if (st == GPTQ_OK) st = check_stored(f, bits, group);
    if (st != GPTQ_OK) return st;
    if (x_dtype == GPTQ_F32 || n_tokens > MOE_MAX_TOKENS || n_experts > MOE_MAX_EXPERTS || top_k > MOE_MAX_TOPK ||
        d > MOE_MAX_WIDTH || f > MOE_MAX_WIDTH)
        return GPTQ_ERR_UNSUPPORTED;
    if (n_tokens == 0) return GPTQ_OK;
    if (!x || !router || !up_codes || !up_scales_f16 || !up_zeros_f16 || !down_codes || !down_scales_f16 ||
        !down_zeros_f16 || !y || !topk_ids || !topk_weights)
        return GPTQ_ERR_INVALID_ARG;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 15) || ws_bytes < moe_ws_bytes(n_tokens, d, f, n_experts, top_k))
        return GPTQ_ERR_WORKSPACE;
    MoeCall c;
    c.x = x; c.xt = x_dtype; c.n = n_tokens; c.d = d; c.ldx = ldx; c.f = f;
    c.router = router; c.E = n_experts; c.k = top_k; c.renormalize = renormalize;
    c.up_codes = up_codes; c.up_scales = up_scales_f16; c.up_zeros = up_zeros_f16;
    c.down_codes = down_codes; c.down_scales = down_scales_f16; c.down_zeros = down_zeros_f16;
    c.bits = bits; c.group = group; c.y = y; c.yt = y_dtype; c.ids = topk_ids; c.weights = topk_weights; c.ws = ws;
    return moe_launch(c, (hipStream_t)stream);
}

}  // extern "C"
#pragma GCC visibility pop
