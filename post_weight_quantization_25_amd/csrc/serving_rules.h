// Which kernel of the serving products takes a call: rules on sizes alone, host code.
#pragma once
#include <stdint.h>

namespace gptq {

// What a large-batch tile's 32-bit offsets and a row's 32-bit integer sums take.  An 8-bit
// activation and an operand u - 128 can both be -128, so a row's sum reaches 2^14 d_col and
// has to stay below 2^31.
constexpr bool gemm_fits(int64_t d_col, int64_t ldx_bytes) {
    return d_col < ((int64_t)1 << 17) && ldx_bytes <= ((int64_t)1 << 24);
}

}  // namespace gptq
