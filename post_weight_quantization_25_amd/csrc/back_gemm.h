// Products with a stored layer's transpose on the matrix cores: out[t][c] = sum_r A[t][r]
// What[r][c].
//
// The sum runs over the rows, whose scales differ, so a scale cannot be taken out of it: the
// weights enter as numbers.  A row is taken times 2^-e_r, its largest scale's power of two
// (row_exponents_kernel), which fp16 then holds to 2^-12 of each weight, down to 2^-25 of the
// row's largest: in one part (PB = 1, for bfloat16 outputs, whose own rounding is 2^-9) or in
// two (PB = 2: 2^-23).  A comes as fp16 planes (PA parts) with 2^e_r and a power of two per
// token multiplied in, zeros behind the last row.
//
// A workgroup of four waves owns BM x BN outputs, a wave a quarter of them.  Slabs of 64 rows:
// A's pieces and the codes of the next slab are on their way into registers while this one is
// multiplied; codes are decoded where they lie transposed, 4 rows x 8 columns per thread, and
// written to LDS by column.  Two buffers, one barrier per slab.
#pragma once
#include "tuning.h"

namespace gptq {

constexpr int BK = 64;                                          // rows per slab

struct BackArgs {
    Stored L; int64_t d_row;                                    // rows of each expert
    const int8_t* e;                                            // e_r of every row
    const uint16_t* A[2]; int64_t lda, a0;                      // n x lda each, lda a multiple of 64: rows a0 .. a0 + lda - 1
    int64_t n;
    const int32_t* offsets; int E;
    // rounded outputs: out = acc 2^-shift[t]
    void* y; gptq_dtype yt;
    const int32_t* shift;
    // or running sums in fp32, one buffer per share of the rows: out = out f[t] + acc
    float* acc; const float* f; int64_t share; int first;
};

// log2 of the power of two below |v|: of a subnormal too; a zero or no number: -1000.
GPTQ_DEV int exponent_of(float v) {
    return v == 0.f || !(fabsf(v) < INFINITY) ? -1000 : ilogbf(v);
}

// v 2^k in fp16 parts: the nearest, and the nearest to what it leaves.
GPTQ_DEV void f16_parts(float v, uint16_t& hi, uint16_t& lo) {
    hi = f32_to_f16_bits(v);
    const float r = v - f16_bits_to_f32(hi);
    lo = f32_to_f16_bits(fabsf(v) < INFINITY ? r : 0.f);
}

GPTQ_DEV f32x4_t mfma_f16(u32x4_t a, u32x4_t b, f32x4_t c) { return mfma16<X_F16>(a, b, c); }

template <int CB, int PA, int PB>
struct BackGemm {
    static constexpr int BM = 128, BN = 128;
    static constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2;
    static constexpr int BUF = PA * A_BYTES + PB * B_BYTES;
    static constexpr int MAXG = BN / 32;                        // groups of a tile's columns
    static constexpr int TAB = BK * MAXG * 8;                   // scale 2^-e and zero of a slab
    static constexpr int LDS_BYTES = 2 * BUF + 2 * TAB;
    static constexpr int NI = 4, NJ = 4;                        // 16 x 16 tiles of a wave: columns, tokens
    struct Entry { float S, z; };

    // Byte of 16-byte piece `piece` (8 of the slab's 64 rows) of column or token `at`.  Reads of
    // 16 consecutive columns and writes of every eighth one spread over the banks.
    static GPTQ_DEV int at(int row, int piece) { return row * 128 + 16 * (piece ^ ((row ^ (row >> 3)) & 7)); }

    // acc[i][j]: lane l's value v is column 64 (wave / 2) + 16 i + 4 (l / 16) + v, token 64 (wave % 2) + 16 j + l % 16.
    // Rows k0 .. k1 - 1 of the layer enter.
    static GPTQ_DEV void run(f32x4_t (&acc)[NI][NJ], const BackArgs& a, const Stored& L, const int8_t* e, int64_t tok0, int64_t end,
                             int64_t c0, int64_t k0, int64_t k1, uint8_t* lds) {
        const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n16 = lane & 15, q = lane >> 4;
        const int wc = 64 * (wave >> 1), wt = 64 * (wave & 1);
        const int gs = L.n_groups == 1 ? 30 : L.gshift;          // one scale per row: every column in group 0
        const int g0 = (int)(c0 >> gs), ngr = L.n_groups - g0;   // the tile's first group; groups from it on
        const int tile_groups = gs >= 7 ? 1 : BN >> gs;
        Entry* tab = reinterpret_cast<Entry*>(lds + 2 * BUF);

        const int64_t left_c = L.d_col - c0;
        const int cp = tid & 15, rp = tid >> 4;                  // the thread's patch: columns 8 cp .., rows 4 rp ..
        const int pc = (int)(left_c - 8 * cp < 8 ? left_c - 8 * cp : 8);   // its columns that exist
        const uint8_t* ct = L.codes + (c0 + 8 * cp) / 8 * CB;

        u32x4_t av[PA][4];
        auto load_a = [&](int64_t k) {
#pragma unroll
            for (int p = 0; p < PA; ++p)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int u = tid + 256 * j, m = u >> 3, piece = u & 7;
                    const int64_t t = tok0 + m < end ? tok0 + m : end - 1;
                    av[p][j] = *reinterpret_cast<const u32x4_t*>(a.A[p] + t * a.lda + (k - a.a0) + 8 * piece);
                }
        };
        auto store_a = [&](uint8_t* buf) {
#pragma unroll
            for (int p = 0; p < PA; ++p)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int u = tid + 256 * j;
                    *reinterpret_cast<u32x4_t*>(buf + p * A_BYTES + at(u >> 3, u & 7)) = av[p][j];
                }
        };
        Raw<CB, 8> cv[4];
        auto load_b = [&](int64_t k) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t r = k + 4 * rp + j, rr = r < k1 ? r : k1 - 1;
                const uint8_t* src = ct + rr * L.code_ld;
                cv[j] = pc == 8 ? load_raw<CB, 8>(src) : load_raw_tail<CB, 8>(src, pc);
            }
        };
        auto load_tab = [&](int64_t k) {                          // the thread's entry: row tid % 64, group tid / 64
            Entry t = {0.f, 0.f};
            const int64_t r = k + (tid & 63);
            const int g = tid >> 6;
            if (g < tile_groups && g < ngr && r < k1) {
                const int64_t i = r * L.n_groups + g0 + g;
                t.S = ldexpf(f16_bits_to_f32(L.scales[i]), -(int)e[r]);
                t.z = f16_bits_to_f32(L.zeros[i]);
            }
            return t;
        };
        auto decode = [&](const Entry* tb, uint8_t* buf) {
            const Entry* te = tb + (gs >= 7 ? 0 : ((8 * cp) >> gs)) * BK + 4 * rp;
            Entry en[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) en[j] = te[j];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                float w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float u = (float)((code_bytes4<CB, 8>(cv[j], c >> 2) >> (8 * (c & 3))) & 0xFFu);
                    w[j] = en[j].S * (u - en[j].z);
                }
                uint16_t hi[4], lo[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) f16_parts(w[j], hi[j], lo[j]);
                uint8_t* dst = buf + PA * A_BYTES + at(8 * cp + c, rp >> 1) + 8 * (rp & 1);
                uint2 v;
                v.x = hi[0] | ((uint32_t)hi[1] << 16); v.y = hi[2] | ((uint32_t)hi[3] << 16);
                *reinterpret_cast<uint2*>(dst) = v;
                if constexpr (PB == 2) {
                    v.x = lo[0] | ((uint32_t)lo[1] << 16); v.y = lo[2] | ((uint32_t)lo[3] << 16);
                    *reinterpret_cast<uint2*>(dst + B_BYTES) = v;
                }
            }
        };

#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        const int slabs = (int)((k1 - k0 + BK - 1) / BK);
        if (slabs == 0) return;
        load_a(k0);
        load_b(k0);
        tab[tid] = load_tab(k0);
        tab[BK * MAXG + tid] = load_tab(k0 + BK);
        __syncthreads();
        store_a(lds);
        decode(tab, lds);
        for (int s = 0; s < slabs; ++s) {
            __syncthreads();
            const int64_t k = k0 + (int64_t)(s + 1) * BK;
            const bool more = s + 1 < slabs;
            Entry next = {0.f, 0.f};
            if (more) {
                load_a(k);
                load_b(k);
                next = load_tab(k + BK);
            }
            uint8_t* buf = lds + (s & 1) * BUF;
#pragma unroll
            for (int h = 0; h < 2; ++h) {                         // 32 rows each
                u32x4_t bf[PB][NI], af[PA][NJ];
#pragma unroll
                for (int i = 0; i < NI; ++i)
#pragma unroll
                    for (int p = 0; p < PB; ++p)
                        bf[p][i] = *reinterpret_cast<const u32x4_t*>(buf + PA * A_BYTES + p * B_BYTES + at(wc + 16 * i + n16, 4 * h + q));
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int p = 0; p < PA; ++p)
                        af[p][j] = *reinterpret_cast<const u32x4_t*>(buf + p * A_BYTES + at(wt + 16 * j + n16, 4 * h + q));
#pragma unroll
                for (int i = 0; i < NI; ++i)
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        acc[i][j] = mfma_f16(bf[0][i], af[0][j], acc[i][j]);
                        if constexpr (PB == 2) acc[i][j] = mfma_f16(bf[1][i], af[0][j], acc[i][j]);
                        if constexpr (PA == 2) acc[i][j] = mfma_f16(bf[0][i], af[1][j], acc[i][j]);
                    }
            }
            if (more) {
                uint8_t* to = lds + ((s + 1) & 1) * BUF;
                store_a(to);
                decode(tab + ((s + 1) & 1) * BK * MAXG, to);
                tab[(s & 1) * BK * MAXG + tid] = next;
            }
        }
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) settle(acc[i][j]);
    }

    // f(column, token of the call, the lane's 4 values from that column on, how many exist)
    template <typename F>
    static GPTQ_DEV void each(const f32x4_t (&acc)[NI][NJ], int64_t tok0, int64_t end, int64_t c0, int64_t d_col, F&& f) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n16 = lane & 15, q = lane >> 4;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int64_t t = tok0 + 64 * (wave & 1) + 16 * j + n16;
            if (t >= end) continue;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int64_t c = c0 + 64 * (wave >> 1) + 16 * i + 4 * q;
                const int have = (int)(d_col - c < 4 ? d_col - c : 4);
                if (have > 0) f(c, t, acc[i][j], have);
            }
        }
    }
};

static_assert(BackGemm<4, 1, 1>::MAXG * BK == 256, "a thread holds one entry of a slab's scales");

// e_r: the exponent of the row's largest scale.  A wave per row.
static __global__ __launch_bounds__(256) void row_exponents_kernel(const uint16_t* scales, int64_t rows, int n_groups, int8_t* e) {
    const int lane = threadIdx.x & 63;
    const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (r >= rows) return;
    int m = -1000;
    for (int g = lane; g < n_groups; g += 64) {
        const int v = exponent_of(f16_bits_to_f32(scales[r * n_groups + g]));
        m = v > m ? v : m;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
        const int v = __shfl_xor(m, o);
        m = v > m ? v : m;
    }
    if (lane == 0) e[r] = (int8_t)(m == -1000 ? 0 : m);
}

inline void row_exponents(const Stored& L, int64_t rows, int8_t* e, hipStream_t s) {
    row_exponents_kernel<<<(unsigned)((rows + 3) / 4), 256, 0, s>>>(L.scales, rows, L.n_groups, e);
}

}  // namespace gptq
