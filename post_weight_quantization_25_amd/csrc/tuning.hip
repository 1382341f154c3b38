// C ABI of the tuning operators: argument validation, workspace sizing and dispatch.
// See include/gptq_tuning.h for the contract.

#include "common.h"
#include "tuning.h"

using namespace gptq;

static bool valid_dtype(gptq_dtype t) { return t == GPTQ_F32 || t == GPTQ_BF16 || t == GPTQ_F16; }
static bool misfit(const void* ws, size_t have, size_t need) {
    return !ws || (reinterpret_cast<uintptr_t>(ws) & 15) || have < need;
}

// What the operators ask of a stored layer of n_experts * d_row rows and of n rows of
// activations; group -1 (per tensor) becomes 0.
static gptq_status check_layer(int64_t E, int64_t d_row, int64_t d_col, int32_t bits, int32_t& group, int64_t n) {
    if (E < 1 || d_row < 1 || d_col < 1 || n < 0) return GPTQ_ERR_INVALID_ARG;
    if (group == -1) group = 0;
    if (group < 0) return GPTQ_ERR_INVALID_ARG;
    if (bits != 3 && bits != 4 && bits != 8) return GPTQ_ERR_UNSUPPORTED;
    if (group > 0 && d_col % group != 0) return GPTQ_ERR_INVALID_ARG;
    if (group != 0 && group != 32 && group != 64 && group != 128) return GPTQ_ERR_UNSUPPORTED;
    if (bits <= 4 && (d_col & 1)) return GPTQ_ERR_INVALID_ARG;
    if (bits == 3 && (d_col & 7)) return GPTQ_ERR_INVALID_ARG;
    if (E > TUNE_MAX_EXPERTS || d_col > TUNE_MAX_WIDTH || d_row > ((int64_t)1 << 25) || E * d_row > ((int64_t)1 << 26) ||
        n > SERVE_MAX_TOKENS)
        return GPTQ_ERR_UNSUPPORTED;
    return GPTQ_OK;
}

// The smallest tiles of many rows, `per` x 128 outputs, are one launch extent (of less than 2^32 threads).
static bool many_tiles(int64_t n, int64_t E, int64_t width, int per) {
    return (n / per + (E < n ? E : n) + 1) * ((width + 127) / 128) > ((int64_t)1 << 24);
}

static gptq_status check_grouped(int64_t E, int64_t d_row, int64_t d_col, int32_t bits, int32_t& group, int64_t n,
                                 gptq_dtype in, gptq_dtype out, int64_t ld, int64_t in_width, int64_t out_width,
                                 const int32_t* offsets, int tile) {
    if (!valid_dtype(in) || !valid_dtype(out)) return GPTQ_ERR_INVALID_ARG;
    const gptq_status st = check_layer(E, d_row, d_col, bits, group, n);
    if (st != GPTQ_OK) return st;
    if (ld < in_width || (!offsets && E != 1)) return GPTQ_ERR_INVALID_ARG;
    if (in == GPTQ_F32 || many_tiles(n, E, out_width, tile)) return GPTQ_ERR_UNSUPPORTED;
    return GPTQ_OK;
}

static gptq_status head(const uint8_t* codes, const uint16_t* scales, const uint16_t* zeros, int64_t vocab, int64_t d,
                        int32_t bits, int32_t group, const void* x, gptq_dtype xt, int64_t n, int64_t ldx,
                        const int32_t* ids, const void* top, gptq_dtype topt, int32_t k, float T, const float* weights,
                        float* loss, void* dx, gptq_dtype dxt, void* ws, size_t ws_bytes, void* stream) {
    if (!valid_dtype(xt) || (dx && !valid_dtype(dxt))) return GPTQ_ERR_INVALID_ARG;
    const gptq_status st = check_layer(1, vocab, d, bits, group, n);
    if (st != GPTQ_OK) return st;
    if (ldx < d) return GPTQ_ERR_INVALID_ARG;
    if (xt == GPTQ_F32 || ldx > TUNE_MAX_PITCH || k > TUNE_MAX_TOP) return GPTQ_ERR_UNSUPPORTED;
    if (n == 0) return GPTQ_OK;
    if (!codes || !scales || !zeros || !x || !ids || !loss) return GPTQ_ERR_INVALID_ARG;
    if (misfit(ws, ws_bytes, head_ws_bytes(n, d, vocab, group, k, dx != nullptr))) return GPTQ_ERR_WORKSPACE;
    HeadCall c;
    c.L = stored_layer(codes, scales, zeros, d, bits, group);
    c.vocab = vocab; c.bits = bits; c.group = group;
    c.x = x; c.xt = xt; c.ldx = ldx; c.n = n;
    c.ids = ids; c.k = k; c.top = top; c.topt = topt; c.temperature = T; c.weights = weights;
    c.loss = loss; c.dx = dx; c.dxt = dxt; c.ws = ws;
    return head_launch(c, (hipStream_t)stream);
}

#pragma GCC visibility push(default)
extern "C" {

gptq_status gptqt_linear_grouped(const uint8_t* codes, const uint16_t* scales_f16, const uint16_t* zeros_f16,
                                 int32_t n_experts, int64_t d_row, int64_t d_col, int32_t bits, int32_t group_size,
                                 const void* x, gptq_dtype x_dtype, int64_t n_rows, int64_t ldx,
                                 const int32_t* offsets, void* y, gptq_dtype y_dtype, void* ws, size_t ws_bytes, void* stream) {
    const gptq_status st = check_grouped(n_experts, d_row, d_col, bits, group_size, n_rows, x_dtype, y_dtype, ldx, d_col,
                                         d_row, offsets, 64);
    if (st != GPTQ_OK) return st;
    if (ldx > TUNE_MAX_PITCH) return GPTQ_ERR_UNSUPPORTED;
    if (n_rows == 0) return GPTQ_OK;
    if (!codes || !scales_f16 || !zeros_f16 || !x || !y) return GPTQ_ERR_INVALID_ARG;
    const size_t need = grouped_ws_bytes(n_rows, n_experts, d_row, d_col, group_size);
    if (need && misfit(ws, ws_bytes, need)) return GPTQ_ERR_WORKSPACE;
    GroupedArgs a = {};
    a.L = stored_layer(codes, scales_f16, zeros_f16, d_col, bits, group_size);
    a.d_row = d_row; a.x = (const uint16_t*)x; a.ldx = ldx; a.n = n_rows; a.offsets = offsets; a.E = n_experts;
    a.y = y; a.yt = y_dtype; a.ldy = d_row;
    const bool large = grouped_large(a, d_row);
    const gptq_status ready = large ? grouped_prepare(a, x_dtype, bits, group_size, ws, (hipStream_t)stream) : GPTQ_OK;
    return ready != GPTQ_OK ? ready : grouped_launch(a, x_dtype, bits, group_size, large, ws, d_row, 0, (hipStream_t)stream);
}

static bool layer_sized(int64_t n, int64_t E, int64_t d_row, int64_t d_col, int32_t& group) {
    int32_t g = group;
    const bool ok = check_layer(E, d_row, d_col, 8, g, n) == GPTQ_OK && n > 0;
    group = g;
    return ok;
}

size_t gptqt_linear_grouped_workspace_size(int64_t n_rows, int32_t n_experts, int64_t d_row, int64_t d_col, int32_t group_size) {
    return layer_sized(n_rows, n_experts, d_row, d_col, group_size) ? grouped_ws_bytes(n_rows, n_experts, d_row, d_col, group_size) : 0;
}

size_t gptqt_linear_grouped_backward_workspace_size(int64_t n_rows, int32_t n_experts, int64_t d_row, int64_t d_col,
                                                    int32_t group_size) {
    return layer_sized(n_rows, n_experts, d_row, d_col, group_size) ? back_ws_bytes(n_rows, n_experts, d_row, d_col, group_size) : 0;
}

gptq_status gptqt_linear_grouped_backward(const uint8_t* codes, const uint16_t* scales_f16, const uint16_t* zeros_f16,
                                          int32_t n_experts, int64_t d_row, int64_t d_col, int32_t bits,
                                          int32_t group_size, const void* dy, gptq_dtype dy_dtype, int64_t n_rows,
                                          int64_t ld_dy, const int32_t* offsets, void* dx, gptq_dtype dx_dtype,
                                          void* ws, size_t ws_bytes, void* stream) {
    const gptq_status st = check_grouped(n_experts, d_row, d_col, bits, group_size, n_rows, dy_dtype, dx_dtype, ld_dy,
                                         d_row, d_col, offsets, 32);
    if (st != GPTQ_OK) return st;
    if (n_rows == 0) return GPTQ_OK;
    if (!codes || !scales_f16 || !zeros_f16 || !dy || !dx) return GPTQ_ERR_INVALID_ARG;
    if (misfit(ws, ws_bytes, back_ws_bytes(n_rows, n_experts, d_row, d_col, group_size))) return GPTQ_ERR_WORKSPACE;
    BackCall c;
    c.L = stored_layer(codes, scales_f16, zeros_f16, d_col, bits, group_size);
    c.d_row = d_row; c.bits = bits; c.dy = dy; c.dyt = dy_dtype; c.ldy = ld_dy; c.n = n_rows;
    c.offsets = offsets; c.E = n_experts; c.dx = dx; c.dxt = dx_dtype; c.ws = ws;
    return back_launch(c, (hipStream_t)stream);
}

size_t gptqt_cross_entropy_workspace_size(int64_t n_tokens, int64_t d, int64_t vocab, int32_t group_size, int32_t with_grad) {
    return layer_sized(n_tokens, 1, vocab, d, group_size) ? head_ws_bytes(n_tokens, d, vocab, group_size, 1, with_grad != 0) : 0;
}

gptq_status gptqt_cross_entropy(const uint8_t* codes, const uint16_t* scales_f16, const uint16_t* zeros_f16,
                                int64_t vocab, int64_t d, int32_t bits, int32_t group_size, const void* x,
                                gptq_dtype x_dtype, int64_t n_tokens, int64_t ldx, const int32_t* targets,
                                const float* weights, float* loss, void* dx, gptq_dtype dx_dtype, void* ws,
                                size_t ws_bytes, void* stream) {
    return head(codes, scales_f16, zeros_f16, vocab, d, bits, group_size, x, x_dtype, n_tokens, ldx, targets, nullptr,
                GPTQ_F32, 1, 1.f, weights, loss, dx, dx_dtype, ws, ws_bytes, stream);
}

size_t gptqt_distill_workspace_size(int64_t n_tokens, int64_t d, int64_t vocab, int32_t group_size, int32_t top_k,
                                    int32_t with_grad) {
    return layer_sized(n_tokens, 1, vocab, d, group_size) && top_k >= 1 && top_k <= TUNE_MAX_TOP
               ? head_ws_bytes(n_tokens, d, vocab, group_size, top_k, with_grad != 0) : 0;
}

gptq_status gptqt_distill(const uint8_t* codes, const uint16_t* scales_f16, const uint16_t* zeros_f16, int64_t vocab,
                          int64_t d, int32_t bits, int32_t group_size, const void* x, gptq_dtype x_dtype,
                          int64_t n_tokens, int64_t ldx, const int32_t* ids, const void* top, gptq_dtype top_dtype,
                          int32_t top_k, float temperature, const float* weights, float* loss, void* dx,
                          gptq_dtype dx_dtype, void* ws, size_t ws_bytes, void* stream) {
    if (top_k < 1 || !valid_dtype(top_dtype) || !(temperature > 0.f && temperature < INFINITY)) return GPTQ_ERR_INVALID_ARG;
    if (n_tokens > 0 && !top) return GPTQ_ERR_INVALID_ARG;
    return head(codes, scales_f16, zeros_f16, vocab, d, bits, group_size, x, x_dtype, n_tokens, ldx, ids, top, top_dtype,
                top_k, temperature, weights, loss, dx, dx_dtype, ws, ws_bytes, stream);
}

}  // extern "C"
#pragma GCC visibility pop
