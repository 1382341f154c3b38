// Products with a stored layer's transpose on the matrix cores: out[t][c] = sum_r A[t][r]
// What[r][c].
//
// The sum runs over the rows, whose scales differ, so a scale cannot be taken out of it: the
// weights enter as numbers.  A row is taken times 2^-e_r (group_exponent, rows_kernel), which brings
// its largest scale to 16 .. 32 for zeros up to 1024, and which fp16 then holds to 2^-11 of each
// weight and 2^-25: in one part (PB = 1, for bfloat16 outputs, whose own rounding is 2^-8) or in
// two (PB = 2: 2^-23, and 2^-25).  A comes as fp16 planes (PA parts) with 2^e_r and a power of two per
// token multiplied in, zeros behind the last row.
//
// A workgroup owns BM tokens x BN columns in slabs of 32 rows; a wave MT x 4 tiles of 16 x 16.
// Both operands go through LDS as fp16 with a slab's rows together, the codes decoded once per
// workgroup: a thread takes 4 rows x 4 columns, pairs two rows' codes in a register (1024 + u
// as fp16 is 0x6400 | u, so u - z and its product with the scale are one packed instruction
// each) and so writes them transposed.  One barrier per slab.
//
// Measured: 2048 tokens x 11008 x 4096 int4 g128, one part, 180 us (1030 Tflop/s), the matrix unit busy
// 47% of the cycles, the vector unit 34%; 4096 x 8192 x 4096 8-bit 240 to 265 (1040 to 1150).  Of 246
// us for 256 slabs the matrix instructions and barriers alone take 174, with the LDS reads 180,
// without the loads 220; the loads alone 117.  A second set of weight fragments spills (510 us).
// Decoding per wave from registers, without LDS, took 461 for the 8-bit case.
#pragma once
#include "stored_gemm.h"
#include "tuning.h"

namespace gptq {

constexpr int BK = 32;                                          // rows per slab

// Four rows' scales times 2^-e_r and 1024 + their zeros, fp16, as the product takes them.  A
// zero that is no whole number in -1024 .. 1024 has the sign bit of its 1024 + z set: such
// rows' zeros are read from the layer (decode_any).
struct Quad { uint32_t S01, zz01, S23, zz23; };

struct BackArgs {
    Stored L; int64_t d_row;                                    // rows of each expert
    const Quad* T; int64_t quads;                               // per expert and group: `quads` for its rows, zeros behind the last
    const uint16_t* A[2]; int64_t a0;                           // [slab][token][32 rows] each, from row a0 on
    int64_t n;
    const int32_t* offsets; int E;
    // rounded outputs: out = acc 2^-shift[t]
    void* y; gptq_dtype yt;
    const int32_t* shift;
    // or sums in fp32, a buffer per share of the rows: out = acc, or from the second round on out f[t] + acc
    float* sums; int64_t share; const float* f; int first;
};

// log2 of the power of two below |v|: of a subnormal too; a zero or no number: -1000.
GPTQ_DEV int exponent_of(float v) {
    return v == 0.f || !(fabsf(v) < INFINITY) ? -1000 : __builtin_amdgcn_frexp_expf(v) - 1;
}

// v 2^k in fp16 parts: the nearest, and the nearest to what it leaves.
GPTQ_DEV void f16_parts(float v, uint16_t& hi, uint16_t& lo) {
    hi = f32_to_f16_bits(v);
    const float r = v - f16_bits_to_f32(hi);
    lo = f32_to_f16_bits(fabsf(v) < INFINITY ? r : 0.f);
}

GPTQ_DEV f16x2_t as_f16x2(uint32_t v) { return __builtin_bit_cast(f16x2_t, v); }
GPTQ_DEV uint32_t as_u32(f16x2_t v) { return __builtin_bit_cast(uint32_t, v); }

// LDS holds a slab as 256-byte lines of four columns (or tokens), 16 bytes for 8 of the slab's 32
// rows, a line's 16 pieces XOR-swizzled.  A read of 16 columns by a wave serves columns 0 - 3
// and 12 - 15 of one lane group and the other 8 of the next at a time: with these swizzles
// they lie in 16 places.  The writes of every fourth column's two halves of a piece do, too.
GPTQ_DEV int line_swizzle(int line) { return (line & 12) | (((line ^ (line >> 1)) & 1) << 1) | ((line >> 1) & 1); }
GPTQ_DEV int slab_at(int c, int piece) { return (c >> 2) * 256 + 16 * ((((c & 3) << 2) | piece) ^ line_swizzle(c >> 2)); }

// The barrier of a workgroup whose waves have waited for what the others read; loads stay in flight.
GPTQ_DEV void barrier_only() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// DIRECT: the codes' rows are whole and aligned 16 bytes (direct_codes) and go straight to LDS.
inline bool direct_codes(const Stored& L) { return ((reinterpret_cast<uintptr_t>(L.codes) | (uintptr_t)L.code_ld) & 15) == 0; }

template <int CB, int PA, int PB, int MT, int WT, int WC, bool DIRECT>
struct BackGemm {
    static constexpr int BM = 16 * MT * WT, BN = 64 * WC, THREADS = 64 * WT * WC, WAVES = WT * WC, NI = 4;
    static constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2;
    static constexpr int ROW = BN * CB / 8, PIECES = ROW / 16, C_BYTES = BK * ROW, T_BYTES = 1024;   // codes of a slab; its Quads
    static constexpr int BUFS = 4;
    static constexpr int LDS_BYTES = BUFS * (PA * A_BYTES + C_BYTES + 2 * T_BYTES) + 2 * PB * B_BYTES;
    static constexpr int AP = BM / 16 / WAVES > 0 ? BM / 16 / WAVES : 1;   // loads of a plane's slab per wave: 16 tokens each
    static constexpr bool ALL_C = BK * PIECES == THREADS;       // every wave loads codes
    static_assert(WT == 2 && BK * PIECES <= THREADS, "a thread decodes one patch of 4 rows x 4 columns and copies at most one piece");

    // acc[i][j]: lane l's value v is column 64 (wave % WC) + 16 i + 4 (l / 16) + v, token 16 MT (wave / WC) + 16 j + l % 16.
    // Rows k0 .. k1 - 1 of the layer enter; k0 and k0 - a.a0 are multiples of 32, and k1 is one or d_row.
    // T: the layer's Quads.
    static GPTQ_DEV void run(f32x4_t (&acc)[NI][MT], const BackArgs& a, const Stored& L, const Quad* T, int64_t tok0, int64_t end,
                             int64_t c0, int64_t k0, int64_t k1, uint8_t* lds) {
        const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n16 = lane & 15, q = lane >> 4;
        const int wc = 64 * (wave % WC), wt = 16 * MT * (wave / WC);
        const int gs = L.n_groups == 1 ? 30 : L.gshift;          // one scale per row: every column in group 0
        const int slabs = (int)((k1 - k0 + BK - 1) / BK);
        uint8_t* bb = lds + BUFS * PA * A_BYTES;
        uint8_t* cc = bb + 2 * PB * B_BYTES;
        uint8_t* tt = cc + BUFS * C_BYTES;                       // two turns of four slabs
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        if (slabs <= 0) return;

        // Wave w loads tokens 16 (w + WAVES j) .. + 15 of A: 4 lines of slab_at, lane l the line's
        // piece l % 16.  (Few tokens: several waves the same ones, so that all count alike.)
        const int block = BM / 16 < WAVES ? wave % (BM / 16) : wave;
        uint32_t aoff[AP];
#pragma unroll
        for (int j = 0; j < AP; ++j) {
            const int line = 4 * (block + WAVES * j) + (lane >> 4), x = (lane & 15) ^ line_swizzle(line);
            int m = 4 * line + (x >> 2);
            if (tok0 + m >= end) m = (int)(end - 1 - tok0);
            aoff[j] = (uint32_t)m * (2 * BK) + 16 * (x & 3);
        }
        const uint8_t* a_next[PA];
#pragma unroll
        for (int p = 0; p < PA; ++p) a_next[p] = reinterpret_cast<const uint8_t*>(a.A[p] + ((k0 - a.a0) / BK * a.n + tok0) * BK);

        // Piece `tid` of a slab's codes: row tid / PIECES.  Pieces behind the columns: the row's first.
        const uint32_t ld = (uint32_t)L.code_ld;
        const int64_t row_left = L.code_ld - c0 * CB / 8;        // bytes of the row from the tile's first column on
        const int crow = tid / PIECES, ccol = 16 * (tid % PIECES) < row_left ? 16 * (tid % PIECES) : 0;
        const bool has_piece = tid < BK * PIECES;
        const bool loads_c = DIRECT && wave * 64 < BK * PIECES;
        const int tail = (int)(a.d_row - k0 - (int64_t)(slabs - 1) * BK < BK ? a.d_row - k0 - (int64_t)(slabs - 1) * BK : BK);   // rows of the last slab
        const uint32_t coff = (uint32_t)crow * ld + ccol, coff_last = (uint32_t)(crow < tail ? crow : tail - 1) * ld + ccol;
        const uint8_t* c_next = L.codes + k0 * L.code_ld + c0 * CB / 8;
        const uint8_t* c_end = L.codes + a.d_row * L.code_ld;

        // Quads: lane 8 g + quad, group g of the tile's; wave w those of slab w % 4 of a turn.  Behind
        // the last slab the zeros that end a group's, so that turns are whole.
        const int64_t tg = (c0 >> gs) + (lane >> 3) < L.n_groups ? lane >> 3 : L.n_groups - 1 - (c0 >> gs);
        const uint32_t toff = (uint32_t)(((gs >= 30 ? 0 : tg) * a.quads + (lane & 7)) * (int64_t)sizeof(Quad));
        const Quad* t_first = T + (c0 >> gs) * a.quads;

        const uint32_t m_lds = lds_addr(reinterpret_cast<const uint16_t*>(lds));
        const uint32_t m_a = m_lds + block * 1024, m_c = m_lds + (uint32_t)(cc - lds) + wave * 1024, m_t = m_lds + (uint32_t)(tt - lds) + (wave & 3) * T_BYTES;
        const int64_t a_step = a.n * (2 * BK), c_step = BK * L.code_ld;

        // Behind the last slab that one is loaded again.
        int a_left = slabs - 1, c_left = slabs - 1;
        auto load_a = [&](int buf) {
#pragma unroll
            for (int p = 0; p < PA; ++p)
#pragma unroll
                for (int j = 0; j < AP; ++j) dma16<0>(aoff[j], a_next[p], m_a + (buf * PA + p) * A_BYTES + j * (WAVES * 1024));
            const int64_t by = a_left > 0 ? a_step : 0;
            --a_left;
#pragma unroll
            for (int p = 0; p < PA; ++p) a_next[p] += by;
        };
        u32x4_t piece = {0u, 0u, 0u, 0u};                        // codes on their way through registers
        auto load_c = [&](int buf) {
            const bool more = c_left > 0;                        // uniform
            const uint32_t off = more ? coff : coff_last;
            if constexpr (DIRECT) {
                if (ALL_C || (loads_c && has_piece)) dma16<0>(off, c_next, m_c + buf * C_BYTES);
            } else if (has_piece) {
                const uint8_t* src = c_next + off;
                if (c_end - src >= 16) {
                    __builtin_memcpy(&piece, src, 16);
                } else {                                         // the layer ends in the piece
                    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int i = 0; i < 15; ++i)
                        if (src + i < c_end) w[i >> 2] |= (uint32_t)src[i] << (8 * (i & 3));
                    piece = u32x4_t{w[0], w[1], w[2], w[3]};
                }
            }
            --c_left;
            c_next += more ? c_step : 0;
        };
        auto load_t = [&](int turn) {                            // slabs 4 turn ..
            const int s = 4 * turn + (wave & 3);
            dma16<0>(toff, t_first + (s < slabs ? k0 / 4 + (int64_t)s * (BK / 4) : a.quads - 16), m_t + (turn & 1) * (4 * T_BYTES));
        };
        auto put_piece = [&](int buf) {
            if (!DIRECT && has_piece) *reinterpret_cast<u32x4_t*>(cc + buf * C_BYTES + 16 * tid) = piece;
        };

        // The thread's patch: columns 4 cp .. of rows 4 rp .. of a slab.
        const int cp = (tid >> 1) % (BN / 4), rp = 2 * (tid / (BN / 2)) + (tid & 1);
        const int pg = gs >= 30 ? 0 : (4 * cp) >> gs;            // the patch's group (a tile starts a group)
        const uint8_t* patch = cc + 4 * rp * ROW + (CB == 3 ? (12 * cp / 32) * 4 : 4 * cp * CB / 8);
        struct Ahead { uint32_t b[4]; u32x4_t t; };              // codes of 4 columns of 4 rows, their Quad
        auto read_patch = [&](Ahead& r, int buf, int turn) {
            r.t = *reinterpret_cast<const u32x4_t*>(tt + ((turn & 1) * 4 + buf) * T_BYTES + (8 * pg + rp) * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint8_t* at = patch + buf * C_BYTES + j * ROW;
                if constexpr (CB == 8) r.b[j] = *reinterpret_cast<const uint32_t*>(at);
                else if constexpr (CB == 4) r.b[j] = *reinterpret_cast<const uint16_t*>(at);
                else {                                           // 12 bits of two words (behind the last row: whatever LDS holds)
                    const uint32_t lo = reinterpret_cast<const uint32_t*>(at)[0], hi = reinterpret_cast<const uint32_t*>(at)[1];
                    r.b[j] = (uint32_t)((((uint64_t)hi << 32) | lo) >> (12 * cp & 31)) & 0xFFFu;
                }
            }
        };
        struct Decoded { uint32_t o[PB][4][2]; };                // [part][column][rows 0, 1 or 2, 3]
        // 1024 + u and 1024 + z are fp16 numbers, and so is their difference.
        auto decode_one = [&](Decoded& d, const Ahead& r, int h, int i) {
            uint32_t u;
            if constexpr (CB == 8) u = __builtin_amdgcn_perm(r.b[2 * h + 1], r.b[2 * h], 0x0C000C00u | i | ((4 + i) << 16));
            else u = ((r.b[2 * h] | (r.b[2 * h + 1] << 16)) >> (CB * i)) & (CB == 4 ? 0x000F000Fu : 0x00070007u);
            const f16x2_t v = as_f16x2(u | 0x64006400u) - as_f16x2(r.t[2 * h + 1]), S = as_f16x2(r.t[2 * h]);
            const f16x2_t hi = v * S;
            d.o[0][i][h] = as_u32(hi);
            asm volatile("" : "+v"(d.o[0][i][h]));               // here, between the products
            if constexpr (PB == 2) {
                d.o[1][i][h] = as_u32(__builtin_elementwise_fma(v, S, -hi));
                asm volatile("" : "+v"(d.o[1][i][h]));
            }
        };
        auto odd = [&](const Ahead& r) { return ((r.t[1] | r.t[3]) & 0x80008000u) != 0; };
        // Any zeros, in fp32.
        auto decode_any = [&](Decoded& d, const Ahead& r, int s) {
            int64_t g = (c0 >> gs) + pg;
            g = g < L.n_groups ? g : L.n_groups - 1;             // columns that are not there
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                const int64_t row = k0 + (int64_t)s * BK + 4 * rp + j;
                const float z = f16_bits_to_f32(L.zeros[(row < a.d_row ? row : a.d_row - 1) * L.n_groups + g]);
                const uint32_t word = j == 0 ? r.b[0] : j == 1 ? r.b[1] : j == 2 ? r.b[2] : r.b[3];
                const float S = f16_bits_to_f32((uint16_t)((j < 2 ? r.t[0] : r.t[2]) >> (16 * (j & 1))));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t u = (word >> (CB * i)) & ((1u << CB) - 1);
                    uint16_t part[2];
                    f16_parts(S * ((float)u - z), part[0], part[1]);
#pragma unroll
                    for (int p = 0; p < PB; ++p)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (h == j >> 1)
                                d.o[p][i][h] = j & 1 ? (d.o[p][i][h] & 0xFFFFu) | ((uint32_t)part[p] << 16) : (d.o[p][i][h] & 0xFFFF0000u) | part[p];
                }
            }
        };
        auto store = [&](const Decoded& d, int buf) {
#pragma unroll
            for (int p = 0; p < PB; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint2 v;
                    v.x = d.o[p][i][0]; v.y = d.o[p][i][1];
                    *reinterpret_cast<uint2*>(bb + (buf * PB + p) * B_BYTES + slab_at(4 * cp + i, rp >> 1) + 8 * (rp & 1)) = v;
                }
        };
        // The products of a slab, a token tile after the other, and in between the next slab's
        // codes: fragments are read two tiles ahead, and a tile's products are issued with a share
        // of the decoding, so that both units are fed.
        auto multiply = [&](int abuf, int bbuf, int next, int turn, Decoded& d, Ahead& r, auto&& loads) {
            constexpr int RING = MT < 3 ? MT : 3;
            u32x4_t bf[PB][NI], af[RING][PA];
            auto read_a = [&](int j) {
#pragma unroll
                for (int p = 0; p < PA; ++p)
                    af[j % RING][p] = *reinterpret_cast<const u32x4_t*>(lds + (abuf * PA + p) * A_BYTES + slab_at(wt + 16 * j + n16, q));
            };
#pragma unroll
            for (int p = 0; p < PB; ++p)
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    bf[p][i] = *reinterpret_cast<const u32x4_t*>(bb + (bbuf * PB + p) * B_BYTES + slab_at(wc + 16 * i + n16, q));
#pragma unroll
            for (int j = 0; j < RING - 1; ++j) read_a(j);
            read_patch(r, next, turn);
            __builtin_amdgcn_sched_barrier(0);
            loads();
            __builtin_amdgcn_sched_barrier(0);
            // A wave that multiplies goes before one that still loads or already stores (16 experts of
            // 4096 x 5504, two parts: 912 -> 876 us; 2048 tokens x 11008 x 4096: 244 -> 236).
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                if (j + RING - 1 < MT || RING == 1) read_a(j + RING - 1);
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const u32x4_t (&x)[PA] = af[j % RING];
                    if constexpr (PA == 2) acc[i][j] = mfma16<X_F16>(bf[0][i], x[1], acc[i][j]);
                    if constexpr (PB == 2) acc[i][j] = mfma16<X_F16>(bf[1][i], x[0], acc[i][j]);
                    acc[i][j] = mfma16<X_F16>(bf[0][i], x[0], acc[i][j]);
                }
#pragma unroll
                for (int u = 8 * j / MT; u < 8 * (j + 1) / MT; ++u) decode_one(d, r, u & 1, u >> 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            __builtin_amdgcn_s_setprio(0);
        };

        // Step s multiplies slab s, decodes slab s + 1 into LDS and sends for A of slab s + 3 and
        // the codes of slab s + 4 (Quads: a turn of four slabs at its first step).  At its barrier
        // the loads of the last two steps may be in flight: A of slab s and the codes of slab s + 1
        // are in LDS, and nobody reads the buffers any more that this step's loads and stores fill.
        // Codes that go through registers reach LDS a step later.  A step has no branch but those
        // for odd zeros and for waves without codes: with 8 waves in step a taken branch costs all.
        Ahead r;
        Decoded d = {};
        load_t(0);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k < 3) load_a(k);
            load_c(k);
            put_piece(k);
        }
        wait_vm_lgkm0<0>();
        barrier_only();
        read_patch(r, 0, 0);
        decode_any(d, r, 0);
        store(d, 0);
        const int turns = (slabs + 3) / 4;
        auto step = [&](auto K, int turn) {
            constexpr int k = decltype(K)::value;
            wait_vm_lgkm0<2 * PA * AP>();
            barrier_only();
            multiply(k, k & 1, (k + 1) & 3, turn + (k == 3), d, r, [&] {
                if (k != 0 || turn > 0) put_piece((k + 3) & 3);
                load_a((k + 3) & 3);
                load_c(k);
                if (k == 0) load_t(turn + 1);
            });
            if (__builtin_expect(__ballot(odd(r)) != 0, 0)) decode_any(d, r, 4 * turn + k + 1);   // wave-uniform
            store(d, (k + 1) & 1);                               // (behind the last slab: not used)
        };
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

    // f(column, token of the call, the lane's 4 values from that column on, how many exist)
    template <typename F>
    static GPTQ_DEV void each(const f32x4_t (&acc)[NI][MT], int64_t tok0, int64_t end, int64_t c0, int64_t d_col, F&& f) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n16 = lane & 15, q = lane >> 4;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int64_t t = tok0 + 16 * MT * (wave / WC) + 16 * j + n16;
            if (t >= end) continue;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int64_t c = c0 + 64 * (wave % WC) + 16 * i + 4 * q;
                const int have = (int)(d_col - c < 4 ? d_col - c : 4);
                if (have > 0) f(c, t, acc[i][j], have);
            }
        }
    }
};

// Four outputs, or those of them that exist, from element idx on.
template <gptq_dtype T>
GPTQ_DEV void store_four(void* y, int64_t idx, f32x4_t v, int have) {
    if (have == 4 && T != GPTQ_F32) {
        uint16_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) store_as<T>(h, i, v[i]);
        __builtin_memcpy(reinterpret_cast<uint16_t*>(y) + idx, h, 8);
    } else if (have == 4) {
        __builtin_memcpy(reinterpret_cast<float*>(y) + idx, &v, 16);
    } else {
        for (int i = 0; i < have; ++i) store_as<T>(y, idx + i, v[i]);
    }
}

// The power of two that a group with scale S and zero z asks of its row: the least with which S (u - z)
// 2^-e is an fp16 number, so that the row's other scales lie as far above fp16's subnormals as
// they can.  S 2^-e is below 32 with zeros up to 1024 (32 x 1279 = 40928), 2 up to 32000 (2 x
// 32255 = 64510), 1/2 with any.  In rows whose scales are below 32 (e <= 0) every one keeps all its
// bits; with 2 as the limit for all zeros, scales below 2^-11 next to one of 8 lost some.
GPTQ_DEV int group_exponent(float S, float z) { return exponent_of(S) - (fabsf(z) <= 1024.f ? 4 : fabsf(z) <= 32000.f ? 0 : -2); }

// e_r, the largest of the row's groups, and the layer's Quads.  A workgroup takes 16 rows of an
// expert (blockIdx.y), 16 threads a row; rows behind the last have zeros.
struct RowsArgs {
    const uint16_t* scales; const uint16_t* zeros;
    int64_t d_row; int n_groups;
    int8_t* e; Quad* T; int64_t quads;
};
static __global__ __launch_bounds__(256) void rows_kernel(RowsArgs a) {
    __shared__ int es[16];
    const int tid = threadIdx.x;
    const int64_t row0 = (int64_t)blockIdx.x * 16, base = blockIdx.y * a.d_row;
    const int64_t r = row0 + (tid >> 4);
    int m = -1000;
    if (r < a.d_row)
        for (int g = tid & 15; g < a.n_groups; g += 16) {
            const int64_t at = (base + r) * a.n_groups + g;
            const int v = group_exponent(f16_bits_to_f32(a.scales[at]), f16_bits_to_f32(a.zeros[at]));
            m = v > m ? v : m;
        }
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) {
        const int v = __shfl_xor(m, o);
        m = v > m ? v : m;
    }
    if (m < -900) m = 0;                                         // no scale but zeros
    if ((tid & 15) == 0) {
        es[tid >> 4] = m;
        if (r < a.d_row) a.e[base + r] = (int8_t)m;
    }
    __syncthreads();
    for (int i = tid; i < 4 * a.n_groups; i += 256) {
        const int quad = i & 3, g = i >> 2;
        uint32_t S[4], z4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t row = row0 + 4 * quad + j;
            S[j] = 0;
            z4[j] = 0x6400u;
            if (row < a.d_row) {
                const int64_t at = (base + row) * a.n_groups + g;
                S[j] = f32_to_f16_bits(ldexpf(f16_bits_to_f32(a.scales[at]), -es[4 * quad + j]));
                const float z = f16_bits_to_f32(a.zeros[at]);
                const bool plain = z >= -1024.f && z <= 1024.f && rintf(z) == z;
                z4[j] = plain ? f32_to_f16_bits(1024.f + z) : 0x8000u;
            }
        }
        a.T[((int64_t)blockIdx.y * a.n_groups + g) * a.quads + row0 / 4 + quad] =
            Quad{S[0] | (S[1] << 16), z4[0] | (z4[1] << 16), S[2] | (S[3] << 16), z4[2] | (z4[3] << 16)};
    }
}

// A group's Quads: of rows up to whole 64, and 64 rows of zeros.
inline int64_t quads_of(int64_t d_row) { return (d_row + 63) / 64 * 16 + 16; }
inline size_t quads_bytes(int64_t E, int64_t d_row, int64_t n_groups) { return (size_t)(E * n_groups * quads_of(d_row)) * sizeof(Quad); }

inline void rows_launch(const Stored& L, int64_t E, int64_t d_row, int8_t* e, Quad* T, hipStream_t s) {
    const RowsArgs a = {L.scales, L.zeros, d_row, L.n_groups, e, T, quads_of(d_row)};
    rows_kernel<<<dim3((unsigned)(((d_row + 63) / 64 + 1) * 4), (unsigned)E), 256, 0, s>>>(a);
}

}  // namespace gptq
