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

// Kernel of a batch: the tile kernels for few outputs, else the LDS kernel with 64 or 128
// tokens per workgroup.
constexpr int TILES = 0;

// Tokens per workgroup of the LDS kernel: 128 once that leaves more than 320 workgroups, and
// never for 64 tokens or fewer, which would multiply empty rows.  Both sides measured, int4
// g128, us, 64 / 128 tokens per workgroup:
//  - 8-bit rows.  Rows x 4096, tokens (workgroups of 128): 4096, 1024 (256): 42.1 / 43.1, 1536
//    (384): 63.8 / 60.5, 2048 (512): 80.5 / 62.9; 11008, 320 (258): 41.7 / 57.5, 512 (344): 63.1
//    / 60.2; 131072, 16 (1024): 82.2 / 113.9, 64: 89.0 / 118.4, 96: 160 / 121; 32768, 64 (256):
//    32.8 / 43.4, 128: 43.5 / 44.7.
//  - adapters (bf16, rank 16): 4096, 1024 (256): 78 / 112, 1536 (384): 130 / 114, 2048 (512): 135
//    / 111; 11008, 512 (344): 136 / 117, 2048 (1376): 356 / 307; 131072, 16 (1024): 126 / 172,
//    64: 149 / 191, 96: 278 / 206.  Where the last round of workgroups is nearly empty 128 can
//    lose 5% (11008, 1024 (688): 213 / 222).
constexpr int lds_tokens(int64_t n, int64_t d_row) {
    return n > 64 && (n + 127) / 128 * ((d_row + 127) / 128) > 320 ? 128 : 64;
}

// 8-bit rows.  The two kernels meet at about 2^21 outputs, from 65536 rows on at 2^20.  Both
// sides measured, int4 g128, us, tiles / LDS kernel (64 tokens per workgroup below 65), rows x
// columns, tokens:
//  4096 x 4096, 384: 26.3 / 29.4, 512: 33.9 / 30.1; 11008 x 4096, 128: 27.0 / 29.7, 192: 42.4 /
//  40.2; 4096 x 11008, 384: 60.7 / 72.2, 512: 78.7 / 73.9; 2048 x 1408, 768: 15.5 / 17.5, 1024:
//  19.5 / 17.6; 32768 x 4096, 48: 28.3 / 32.5, 64: 36.0 / 32.8; 49152 x 4096, 32: 39.3 / 41.7;
//  65536 x 4096, 8: 41.3 / 41.7, 16: 48.9 / 41.7; 131072 x 4096, 8: 80.2 / 81.5, 16: 100 / 81.7;
//  131072 x 2048, 4: 40.5 / 43.0, 8: 45.8 / 42.9.  Groups of 32 meet a little later (11008 x
//  4096, 192: 67.0 / 80.4, 256: 84.9 / 83.1), one scale per row earlier (int8, 4096 x 4096, 256:
//  21.8 / 27.2, 384: 31.7 / 27.7; 11008 x 4096, 64: 22.1 / 27.6, 96: 31.3 / 28.2).
constexpr int int8_kernel(int64_t n, int64_t d_row, int64_t d_col, int64_t ldx_bytes) {
    const int64_t least = (int64_t)1 << (d_row >= 65536 ? 20 : 21);
    return n * d_row >= least && gemm_fits(d_col, ldx_bytes) ? lds_tokens(n, d_row) : TILES;
}

// Adapters.  The two kernels meet at about 2^20 outputs; at 2^19 from 32768 rows on, where 128
// rows per workgroup fill the device, and for groups of 32 from 49 tokens on, whose tiles hold
// too much for their registers.  Both sides measured, bf16, rank 16, us, tiles / LDS kernel:
//  int4 g128: 4096 x 4096, 256: 61.5 / 67.2, 320: 78.0 / 63.4; 11008 x 4096, 64: 44.5 / 63, 96:
//  77.3 / 62.9; 4096 x 11008, 256: 137 / 165, 320: 170 / 157; 2048 x 1408, 384: 27.6 / 31.0, 512:
//  35.0 / 32.2; 16384 x 4096, 64: 57.7 / 64.5, 96: 99.9 / 64.6; 32768 x 4096, 8: 41.4 / 50.9, 16:
//  52.1 / 53.8, 17: 68.8 / 55.0, 32: 74.1 / 58.2; 49152 x 4096, 8: 59.0 / 63.7, 12: 66.7 / 64.5;
//  65536 x 4096, 4: 64.8 / 63.6, 8: 76.0 / 63.9; 131072 x 4096, 2: 123 / 121, 4: 132 / 122;
//  40000 x 8192, 16: 114 / 118, 17: 143 / 120.
//  int4 g32: 4096 x 4096, 64: 47.3 / 84.5, 96: 77.6 / 84.8, 128: 87.9 / 85.7, 256: 170 / 89.1;
//  11008 x 4096, 48: 44.5 / 81.9, 64: 128 / 85.6; 32768 x 2048, 17: 56.1 / 42.7, 48: 72.2 / 47.5.
constexpr int lora_kernel(int64_t n, int64_t d_row, int64_t d_col, int64_t ldx_bytes, int group) {
    const bool early = d_row >= 32768 || (group == 32 && n > 48);
    const bool many = early ? n * d_row >= ((int64_t)1 << 19) : n * d_row > ((int64_t)1 << 20);
    return many && gemm_fits(d_col, ldx_bytes) ? lds_tokens(n, d_row) : TILES;
}

}  // namespace gptq
