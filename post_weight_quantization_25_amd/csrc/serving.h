// Host-side launchers of the serving operators (internal to the library).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gptq_serving.h"

namespace gptq {

// Most tokens of a call: their tiles are on the grid's y extent (at most 65535 tiles of 64),
// and one 1024-thread workgroup per token stays below 2^32 threads.
constexpr int64_t SERVE_MAX_TOKENS = (int64_t)65535 * 64;
// Most outputs of a product: its 128 x 128 tiles are one launch extent (below 2^24).
constexpr int64_t SERVE_MAX_OUTPUTS = (int64_t)1 << 36;

struct NormArgs {
    const void* x; int64_t ldx;
    const void* r; int64_t ldr;          // residual, or nullptr
    const void* w;
    float eps;
    int64_t n, d;
    void* h; int64_t ldh;                // T(x + r), or nullptr
    void* y; int64_t ldy;                // T(p rstd), or nullptr
    int8_t* q; int64_t ldq;
    float* scale;
};
gptq_status norm_launch(const NormArgs& a, gptq_dtype xt, gptq_dtype wt, hipStream_t s);

gptq_status linear_int8_launch(const uint8_t* codes, const uint16_t* scales, const uint16_t* zeros, int64_t d_row,
                               int64_t d_col, int bits, int group, const int8_t* x, int64_t ldx, const float* xs,
                               int64_t n, void* y, gptq_dtype yt, hipStream_t s);

constexpr int LORA_MAX_RANK = 256;
size_t lora_ws_bytes(int64_t n, int64_t d_col, int rank);
gptq_status linear_lora_launch(const uint8_t* codes, const uint16_t* scales, const uint16_t* zeros, int64_t d_row,
                               int64_t d_col, int bits, int group, const void* x, gptq_dtype xt, int64_t n, int64_t ldx,
                               const void* A, const void* B, int n_adapters, int rank, const int32_t* ids,
                               const float* scaling, void* y, gptq_dtype yt, void* ws, hipStream_t s);

struct MoeCall {
    const void* x; gptq_dtype xt; int64_t n, d, ldx, f;
    const void* router; int E, k, renormalize;
    const uint8_t* up_codes; const uint16_t* up_scales; const uint16_t* up_zeros;
    const uint8_t* down_codes; const uint16_t* down_scales; const uint16_t* down_zeros;
    int bits, group;
    void* y; gptq_dtype yt; int32_t* ids; float* weights; void* ws;
};
constexpr int MOE_MAX_TOKENS = 256, MOE_MAX_EXPERTS = 512, MOE_MAX_TOPK = 32;
constexpr int64_t MOE_MAX_WIDTH = (int64_t)1 << 20;   // d and f
size_t moe_ws_bytes(int64_t n, int64_t d, int64_t f, int E, int k);
gptq_status moe_launch(const MoeCall& c, hipStream_t s);

}  // namespace gptq
