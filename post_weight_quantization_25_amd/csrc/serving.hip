// C ABI of the serving operators: argument validation, workspace sizing and dispatch.
// See include/gptq_serving.h for the contract.

#include "common.h"
#include "serving.h"

using namespace gptq;

static bool valid_dtype(gptq_dtype t) { return t == GPTQ_F32 || t == GPTQ_BF16 || t == GPTQ_F16; }

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

}  // extern "C"
#pragma GCC visibility pop
