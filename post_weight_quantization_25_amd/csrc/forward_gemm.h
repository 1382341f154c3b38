// Products with a stored layer on the matrix cores for many tokens: y[t][r] = sum_g S[r][g] sum_c
// x[t][c] (u[r][c] - z[r][g]), exact products of fp16 numbers added in fp32.
//
// Activations come as fp16 rows (forward_pack_kernel): fp16 as they are, bfloat16 with a power of
// two per token multiplied in, which brings the largest to 2^14 .. 2^15, so that elements down to
// 2^-28 of it are themselves.  u - z is exact for whole z in -1024 .. 1024.  A row's sums run on
// through its groups in the matrix cores' accumulators: they are kept in units of the current
// group's scale, so where a group begins they are multiplied by S[g - 1] / S[g] (two fp32
// roundings a group), which costs one instruction per sum and group and no second set of sums.
// A layer with another zero, or with a scale that is zero or no number, raises a flag
// (forward_rows_kernel) and is left to the kernel of stored_gemm.h, which takes any.
//
// A workgroup of eight waves owns 256 tokens x 256 rows in slabs of 32 columns, a wave 128 x 64.
// Both operands go through LDS: activations four slabs ahead, codes in chunks of 64 bytes a row
// (whole cache lines' worth over a few slabs), straight from memory; the codes of the next slab
// are decoded, once per workgroup, between the products of this one.  A thread decodes 16
// columns of a row; 3- and 4-bit codes come out as columns 0, 4, 1, 5, 2, 6, 3, 7 of every 8, the
// order in which the activations are packed.
//
// Measured: 4096 tokens x 8192 x 4096 8-bit g128 268 us (1025 Tflop/s), the matrix unit busy 43% of the
// cycles, the vector unit 32%; a dense product of 8192^3 bfloat16 reaches 1286.  The matrix
// instructions alone would take 0.7 of it; decoding, LDS reads and issuing loads add to them
// rather than hide, since a CU holds one workgroup.  The weight fragments of the next slab are
// read into a second set during the step (16 experts of 11008 x 4096, 8192 rows: 1120 to 1190 us).  The
// 128 x 128 tiles, two workgroups per CU, took 368 for the 4096 tokens.
#pragma once
#include "back_gemm.h"

namespace gptq {

struct ForwardArgs {
    Stored L; int64_t d_row;                                    // rows of each expert (or of the span)
    const uint16_t* A;                                          // [slab][token][32 columns]
    const int32_t* shift;                                       // tokens' powers of two
    const float* rho; const uint32_t* zz; const float* S_last;  // [group][row] of all rows; of the row's last group
    int64_t pitch, expert_pitch;                                // rows from a group to the next; values from an expert to the next
    const int32_t* odd;                                         // not 0: nothing is done here
    int64_t n;
    const int32_t* offsets; int E;
    void* y; gptq_dtype yt; int64_t ldy;
};

inline int64_t forward_columns(int64_t d_col) { return (d_col + 127) / 128 * 128; }   // whole turns of four slabs

// GPT: groups per turn of four slabs (forward_turn_groups); 0: one scale per row.
template <int CB, int GPT>
struct ForwardGemm {
    static constexpr int BM = 256, BN = 256, THREADS = 512, WAVES = 8, MT = 8, NI = 4;
    static constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2;
    static constexpr int ROW = CB == 3 ? 48 : 64, SPC = CB == 8 ? 2 : 4;      // bytes of a row in a chunk; slabs of a chunk
    static constexpr int C_BYTES = BN * ROW, PIECES = ROW / 16, C_LOADS = BN * PIECES / 64;   // 16 or 12 loads of a wave
    static constexpr int SETS = GPT ? GPT : 1, T_BYTES = 2048 * SETS;         // a turn's rho and zz, 1 KB each per group
    static constexpr int LDS_BYTES = 4 * A_BYTES + 2 * B_BYTES + 2 * C_BYTES + 2 * T_BYTES;
    static constexpr int SPG = GPT ? 4 / GPT : 4;                             // slabs of a group

    // acc[i][j]: lane l's value v is row 64 (wave % 4) + 16 i + l % 16, token 128 (wave / 4) + 16 j + 4 (l / 16) + v.
    static GPTQ_DEV void run(f32x4_t (&acc)[NI][MT], const ForwardArgs& a, const Stored& L, const float* rho, const uint32_t* zzs,
                             int64_t tok0, int64_t end, int64_t row0, uint8_t* lds) {
        const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n16 = lane & 15, q = lane >> 4;
        const int wr = 64 * (wave & 3), wt = 128 * (wave >> 2);
        uint8_t* bb = lds + 4 * A_BYTES;
        uint8_t* cc = bb + 2 * B_BYTES;
        uint8_t* tt = cc + 2 * C_BYTES;
        const int slabs = (int)((L.d_col + BK - 1) / BK), turns = (slabs + 3) / 4;

        uint32_t aoff[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int line = 4 * (wave + WAVES * j) + (lane >> 4), x = (lane & 15) ^ line_swizzle(line);
            int m = 4 * line + (x >> 2);
            if (tok0 + m >= end) m = (int)(end - 1 - tok0);
            aoff[j] = (uint32_t)m * (2 * BK) + 16 * (x & 3);
        }
        const uint8_t* a_next = reinterpret_cast<const uint8_t*>(a.A + tok0 * BK);
        const int64_t a_step = a.n * (2 * BK);
        // Loads wave, wave + 8 of a chunk: 64 pieces each, in LDS [row][piece], a row's four pieces
        // XOR-swizzled by the row.  Pieces behind the row's end: its first of the chunk.
        const int chunks = (slabs + SPC - 1) / SPC;
        const int64_t row_left = L.code_ld - (int64_t)(chunks - 1) * ROW;      // bytes of a row in the last chunk
        uint32_t coff[2], coff_last[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int u = 64 * (wave + 8 * x) + lane, row = u / PIECES, piece = PIECES == 4 ? (u & 3) ^ ((row >> 2) & 3) : u % PIECES;
            const int64_t r = row0 + row < a.d_row ? row : a.d_row - 1 - row0;
            coff[x] = (uint32_t)r * (uint32_t)L.code_ld + 16 * piece;
            coff_last[x] = (uint32_t)r * (uint32_t)L.code_ld + (16 * piece < row_left ? 16 * piece : 0);
        }
        const uint8_t* c_next = L.codes + row0 * L.code_ld;
        // Load w of a turn's tables: group (w / 2) % SETS, rho or zz.
        const float* t_rho = rho + row0 + (int64_t)((wave >> 1) % SETS) * a.pitch;
        const uint32_t* t_zz = zzs + row0 + (int64_t)((wave >> 1) % SETS) * a.pitch;
        const uint8_t* t_next = (wave & 1) ? reinterpret_cast<const uint8_t*>(t_zz) : reinterpret_cast<const uint8_t*>(t_rho);
        const int64_t t_step = GPT ? a.pitch * (4 * GPT) : 0;

        const uint32_t m_lds = lds_addr(reinterpret_cast<const uint16_t*>(lds));
        const uint32_t m_a = m_lds + wave * 1024, m_c = m_lds + (uint32_t)(cc - lds) + wave * 1024;
        const uint32_t m_t = m_lds + (uint32_t)(tt - lds) + ((wave >> 1) % SETS) * 2048 + (wave & 1) * 1024;

        // Behind the last chunk and turn those are loaded again; A has zeros up to whole turns.
        int a_left = 4 * turns - 1, c_left = chunks - 1, t_left = turns - 1;
        auto load_a = [&](int buf) {
#pragma unroll
            for (int j = 0; j < 2; ++j) dma16<0>(aoff[j], a_next, m_a + buf * A_BYTES + j * (WAVES * 1024));
            a_next += a_left > 0 ? a_step : 0;
            --a_left;
        };
        auto load_c = [&](int place) {
            const bool more = c_left > 0;                        // uniform
            dma16<0>(more ? coff[0] : coff_last[0], c_next, m_c + place * C_BYTES);
            if (C_LOADS == 16 || wave < C_LOADS - 8) dma16<0>(more ? coff[1] : coff_last[1], c_next, m_c + place * C_BYTES + 8 * 1024);
            c_next += more ? ROW : 0;
            --c_left;
        };
        auto load_t = [&](int turn) {
            dma16<0>(16 * lane, t_next, m_t + (turn & 1) * T_BYTES);
            t_next += t_left > 0 ? t_step : 0;
            --t_left;
        };

        // The thread's codes: row tid % 256, columns 16 half .. of a slab.
        const int crow = tid & 255, half = tid >> 8;
        struct Codes { uint32_t w[4]; uint32_t zz; };
        auto read_codes = [&](Codes& r, int place, int sub, int set, int turn) {   // slab `sub` of its chunk, group `set` of its turn
            r.zz = *reinterpret_cast<const uint32_t*>(tt + (turn & 1) * T_BYTES + set * 2048 + 1024 + 4 * crow);
            const uint8_t* row = cc + place * C_BYTES + crow * ROW;
            if constexpr (CB == 8) {
                const u32x4_t v = *reinterpret_cast<const u32x4_t*>(row + 16 * ((2 * sub + half) ^ ((crow >> 2) & 3)));
#pragma unroll
                for (int e = 0; e < 4; ++e) r.w[e] = v[e];
            } else if constexpr (CB == 4) {
                const uint2 v = *reinterpret_cast<const uint2*>(row + 16 * (sub ^ ((crow >> 2) & 3)) + 8 * half);
                r.w[0] = v.x; r.w[1] = v.y;
            } else {
                const uint32_t* w = reinterpret_cast<const uint32_t*>(row + 12 * sub + 4 * half);
                const uint64_t v = (((uint64_t)w[1] << 32) | w[0]) >> (16 * half);
                r.w[0] = (uint32_t)v & 0xFFFFFFu; r.w[1] = (uint32_t)(v >> 24) & 0xFFFFFFu;
            }
        };
        struct Decoded { uint32_t o[8]; };
        auto decode_one = [&](Decoded& d, const Codes& r, int p) {       // pair p of 8
            uint32_t u;
            if constexpr (CB == 8) u = __builtin_amdgcn_perm(0x64646464u, r.w[p >> 1], p & 1 ? 0x04030402u : 0x04010400u);
            else {
                const uint32_t w = CB == 4 ? r.w[p >> 2] : (r.w[p >> 2] & 0xFFFu) | ((r.w[p >> 2] & 0xFFF000u) << 4);
                u = ((w >> (CB * (p & 3))) & (CB == 4 ? 0x000F000Fu : 0x00070007u)) | 0x64006400u;
            }
            d.o[p] = as_u32(as_f16x2(u) - as_f16x2(r.zz));
            asm volatile("" : "+v"(d.o[p]));                             // here, between the products
        };
        auto store = [&](const Decoded& d, int buf) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<u32x4_t*>(bb + buf * B_BYTES + slab_at(crow, 2 * half + h)) =
                    u32x4_t{d.o[4 * h], d.o[4 * h + 1], d.o[4 * h + 2], d.o[4 * h + 3]};
        };

#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

        u32x4_t bf[2][NI], af[4];
        auto read_a = [&](int buf, int j) { af[j & 3] = *reinterpret_cast<const u32x4_t*>(lds + buf * A_BYTES + slab_at(wt + 16 * j + n16, q)); };
        auto read_b = [&](int buf, int i) { bf[buf][i] = *reinterpret_cast<const u32x4_t*>(bb + buf * B_BYTES + slab_at(wr + 16 * i + n16, q)); };

        // As in BackGemm: step s multiplies slab s, decodes slab s + 2 and sends for A of slab s + 3;
        // a chunk as soon as the one in its place is decoded, two or four steps before its first slab
        // is; the next turn's tables at a turn's first step.
        Codes r;
        Decoded d;
        auto step = [&](auto K, int turn) {
            constexpr int k = decltype(K)::value, ahead = (k + 2) & 3;
            wait_vm_lgkm0<2>();
            barrier_only();
            constexpr bool begins = GPT != 0 && k % SPG == 0;    // a group (rho of the first one is 1)
            float scale[NI];
            if constexpr (begins)
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    scale[i] = *reinterpret_cast<const float*>(tt + (turn & 1) * T_BYTES + (k / SPG) * 2048 + 4 * (wr + 16 * i + n16));
            const int other = turn + (k >= 2);                   // turn of slab s + 2
            read_codes(r, SPC == 4 ? other & 1 : ahead / 2, ahead % SPC, GPT ? ahead / SPG : 0, other);
            load_a((k + 3) & 3);
            if (SPC == 4 && k == 2) load_c(turn & 1);            // chunk turn + 2; slab 4 turn + 3 was decoded a step ago
            if (SPC == 2 && k % 2 == 0) load_c(k / 2);           // chunk of slabs s + 4, s + 5; slab s + 1 was decoded a step ago
            if (k == 0) load_t(turn + 1);
            __builtin_amdgcn_sched_barrier(0);
            auto rescale = [&](int j) {
                if constexpr (begins)
#pragma unroll
                    for (int i = 0; i < NI; ++i)
#pragma unroll
                        for (int v = 0; v < 4; ++v) acc[i][j][v] *= scale[i];
            };
            rescale(0);
            __builtin_amdgcn_s_setprio(1);                       // as in BackGemm
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                read_a(j + 2 < MT ? k : (k + 1) & 3, (j + 2) % MT);
#pragma unroll
                for (int i = 0; i < NI; ++i) acc[i][j] = mfma16<X_F16>(af[j & 3], bf[k & 1][i], acc[i][j]);
                if (j >= MT - NI) read_b((k + 1) & 1, j - (MT - NI));   // slab s + 1's
                if (j + 1 < MT) rescale(j + 1);
                if (j >= 1)
#pragma unroll
                    for (int u = 8 * (j - 1) / (MT - 1); u < 8 * j / (MT - 1); ++u) decode_one(d, r, u);
                __builtin_amdgcn_sched_barrier(0);
            }
            __builtin_amdgcn_s_setprio(0);
            store(d, k & 1);                                     // (behind the last slab: not used)
        };
        load_t(0);
        load_c(0);
        load_c(1);
#pragma unroll
        for (int k = 0; k < 3; ++k) load_a(k);
        wait_vm_lgkm0<0>();
        barrier_only();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            read_codes(r, 0, k, GPT ? k / SPG : 0, 0);
#pragma unroll
            for (int p = 0; p < 8; ++p) decode_one(d, r, p);
            store(d, k);
        }
        wait_vm_lgkm0<0>();
        barrier_only();
#pragma unroll
        for (int i = 0; i < NI; ++i) read_b(0, i);
        read_a(0, 0);
        read_a(0, 1);
        for (int turn = 0; turn < turns; ++turn) {
            step(std::integral_constant<int, 0>{}, turn);
            step(std::integral_constant<int, 1>{}, turn);
            step(std::integral_constant<int, 2>{}, turn);
            step(std::integral_constant<int, 3>{}, turn);
        }
        wait_vm_lgkm0<0>();                                      // no load into LDS outlives the workgroup
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) settle(acc[i][j]);
    }
};

// What a product of many tokens keeps in the workspace (grouped.hip): the arrays of ForwardArgs, `groups`
// groups of `pitch` rows of each expert.
struct ForwardBuffers {
    uint16_t* A; int32_t* shift; float* rho; uint32_t* zz; float* S_last; int32_t* odd;
    int64_t pitch, groups;
};

}  // namespace gptq
