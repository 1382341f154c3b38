// Large batches: tokens x d_col activations (8- or 16-bit) with a stored layer on the
// matrix cores.
//
// A workgroup of four waves owns BM tokens x 128 weight rows; a wave takes all BM tokens
// and 32 of the rows.  So every code is loaded, by the lane that needs it, from memory
// straight into registers and decoded once per workgroup (u - zc in the operand's type, see
// stored_tile.h), and only the activations, which all four waves need, go through LDS: in
// slabs of a token's row, two buffers, one
// barrier per slab.  While slab s is multiplied, slab s + 1 is on its way into registers.
// 16-byte pieces of a slab's row are XOR-swizzled by the row, which spreads a fragment's
// 16 rows over all banks.
//
// Measured on the way (8-bit, 4096 tokens x 4096 x 4096 int4 g128, under the profiler): both
// operands through LDS 200 us, codes straight to registers 145, scales through LDS too (a
// cache line per row for 4 bytes otherwise) 137; 114 replayed without the profiler.  256
// registers and 80 KB of LDS leave two waves per SIMD, whose issue slots and waits are what
// is left; the matrix unit is busy a fifth of the time.
//
// As in stored_tile.h, a piece is the columns of one scale (128, 64 or 32), of which lane
// l holds the RUN = piece / 4 columns from RUN (l / 16) on, on both sides.  PIECE 0 is one
// scale per row: pieces of 128 columns whose sums run on through the row.
#pragma once
#include "serving_rules.h"
#include "stored_tile.h"

namespace gptq {

constexpr int GEMM_ROWS = 128;

// Workgroup -> tile: XCD k (workgroups k, k + 8, ..) takes a contiguous run of tiles, and
// within it token tiles run fastest in stripes of 8, so that the rows and the activations
// in flight on one XCD stay in its L2.
GPTQ_DEV void tile_of(int gm, int gn, int& tm, int& tn) {
    const int total = gm * gn, lin = blockIdx.x;
    const int base = total / 8, rest = total % 8, xcd = lin % 8;
    const int id = xcd * base + (xcd < rest ? xcd : rest) + lin / 8;
    const int stripe = id / (8 * gn), in = id % (8 * gn);
    const int high = gm - 8 * stripe < 8 ? gm - 8 * stripe : 8;
    tm = 8 * stripe + in % high;
    tn = in / high;
}

template <int X, int CB, int PIECE, int BM, int SLAB>   // SLAB: bytes of a token's row in LDS (128 or 256)
struct StoredGemm {
    static constexpr int XB = xbytes<X>();
    static constexpr int KS = SLAB / XB;                       // columns per slab
    static constexpr int MT = BM / 16, NT = 2;                 // 16 x 16 tiles per wave
    static constexpr int PC = PIECE ? PIECE : KS < 128 ? KS : 128;             // columns per piece
    static constexpr int PP = KS / PC;                         // pieces per slab
    static constexpr int RUN = PC / 4;
    static constexpr int KB = X == X_I8 && RUN == 8 ? 8 : 16;  // bytes of a lane's operand per product
    static constexpr int STEPS = RUN * XB / KB;                // products per piece
    static constexpr int AU = BM * (SLAB / 16) / 256;          // 16-byte activation pieces per thread
    static constexpr int LDS_BYTES = 2 * BM * SLAB + (PIECE ? 16 * GEMM_ROWS * 8 : 0);
    typedef typename Acc<X>::t sum_t;

    // A fragment read serves 16 lanes at a time: rows 0 - 3 and 12 - 15 of one lane group and
    // the other 8 rows of the next, whose pieces are RUN XB / 16 further on.  The swizzle
    // spreads them over the 16 16-byte columns of the 64 banks.
    static GPTQ_DEV int slab_at(int row, int piece16) {
        constexpr bool EVEN = RUN * XB % 32 == 0;              // the lane groups' pieces differ in bits above the lowest
        int f = row & 15;
        if constexpr (SLAB == 128) {
            const int g = f >> 1;
            f = EVEN ? ((g & 1) << 1) | (g & 4) | (((g >> 1) ^ (g >> 2)) & 1) : g;
        } else if constexpr (EVEN) {
            f = ((f & 3) << 1) | (f & 8) | (((f >> 2) ^ (f >> 3)) & 1);
        }
        return row * SLAB + 16 * (piece16 ^ f);
    }

    // With 64 tokens per workgroup codes are half the cache accesses: lane l then loads row l /
    // 4's piece l % 4 (contiguous over four lanes, an access per 64 bytes instead of one per
    // lane) and decode hands it to the lane that multiplies it (777 tokens x 4001 x 11008 int3:
    // 61.8 us against 65.9).  With 128 the lanes' own loads are as good (4096 tokens x 4096 x
    // 4096 int4: 114 us against 116).
    static constexpr bool SPREAD = BM == 64;
    struct Codes { Raw<CB, RUN> c[NT][PP]; };                  // a slab's codes of the lane's rows
    struct Frag { uint32_t w[KB / 4]; };
    struct Operand {                                           // the same, decoded
        Frag f[PP][NT][STEPS];
        float S[PP][NT], rz[PP][NT];
    };
    // Scales and zeros of the tile's rows for TG groups, in LDS as [group][row]: read from
    // memory slab by slab they would cost a cache line per row for every 4 bytes used.
    static constexpr int TG = 16;
    struct Entry { float S; uint32_t z; };                     // z: fp16 zero | its part in the operand's form << 16
    static GPTQ_DEV Entry entry(uint16_t S, uint16_t z) {
        const float zc = zero_part<X, CB>(f16_bits_to_f32(z));
        uint32_t form;
        if constexpr (X == X_I8) form = (uint32_t)(int)zc & 0xFFu;                                    // the byte
        else if constexpr (X == X_F16) form = __builtin_bit_cast(uint16_t, (_Float16)(1024.f + zc));  // fp16(1024 + zc)
        else form = f32_to_bf16_bits(zc);                                                             // bfloat16(zc), exact
        return Entry{f16_bits_to_f32(S), z | (form << 16)};
    }
    static GPTQ_DEV float part_of(uint32_t form) {             // zc from its form
        if constexpr (X == X_I8) return CB == 8 ? 128.f : (float)(int)(int8_t)(form & 0xFFu);
        else if constexpr (X == X_F16) return f16_bits_to_f32((uint16_t)form) - 1024.f;
        else return bf16_bits_to_f32((uint16_t)form);
    }

    // acc[mt][nt]: lane l's value i is token 16 mt + 4 (l / 16) + i, weight row 32 wave + 16 nt
    // + l % 16 of the tile.
    static GPTQ_DEV void run(f32x4_t (&acc)[MT][NT], const Stored& L, int64_t d_row, const uint8_t* x, int64_t ldx_bytes,
                             int64_t n, int64_t tok0, int64_t row0, uint8_t* lds) {
        const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n16 = lane & 15, q = lane >> 4;
        const int nslab = (int)((L.d_col + KS - 1) / KS), nfull = (int)(L.d_col / KS);

        // tile-relative offsets fit 32 bits (gemm_fits); rows past the end re-read the last
        const uint8_t* xt = x + tok0 * ldx_bytes;
        const uint8_t* ct = L.codes + row0 * L.code_ld;
        const uint16_t* st = L.scales + row0 * L.n_groups;
        const uint16_t* zt = L.zeros + row0 * L.n_groups;
        const int toks = (int)(n - tok0 < BM ? n - tok0 : BM);
        const int rows = (int)(d_row - row0 < GEMM_ROWS ? d_row - row0 : GEMM_ROWS);
        uint32_t aoff[AU];
#pragma unroll
        for (int j = 0; j < AU; ++j) {
            const int u = tid + 256 * j, r = u / (SLAB / 16);
            aoff[j] = (uint32_t)(r < toks ? r : toks - 1) * (uint32_t)ldx_bytes + 16 * (u % (SLAB / 16));
        }
        const int crow = SPREAD ? lane >> 2 : n16, cpart = SPREAD ? lane & 3 : q;
        uint32_t boff[NT], soff[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = 32 * wave + 16 * nt + n16, c = 32 * wave + 16 * nt + crow;
            boff[nt] = (uint32_t)(c < rows ? c : rows - 1) * (uint32_t)L.code_ld + cpart * (RUN * CB / 8);
            soff[nt] = (uint32_t)(r < rows ? r : rows - 1) * (uint32_t)L.n_groups;
        }

        auto load_a = [&](u32x4_t (&a)[AU], int s) {
            const uint8_t* xs = xt + (int64_t)s * SLAB;
#pragma unroll
            for (int j = 0; j < AU; ++j) __builtin_memcpy(&a[j], xs + aoff[j], 16);
        };
        auto store_a = [&](const u32x4_t (&a)[AU], int s) {
            uint8_t* buf = lds + (s & 1) * BM * SLAB;
#pragma unroll
            for (int j = 0; j < AU; ++j) {
                const int u = tid + 256 * j;
                *reinterpret_cast<u32x4_t*>(buf + slab_at(u / (SLAB / 16), u % (SLAB / 16))) = a[j];
            }
        };
        auto load_b = [&](Codes& b, int s) {
            const uint8_t* cs = ct + (int64_t)s * (KS / 8 * CB);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int p = 0; p < PP; ++p) {
                    b.c[nt][p] = load_raw<CB, RUN>(cs + boff[nt] + p * (PC / 8 * CB));
                }
        };
        Entry* tab = reinterpret_cast<Entry*>(lds + 2 * BM * SLAB);
        auto fill = [&](int g0) {                              // groups g0 .. g0 + TG - 1
            for (int e = tid; e < GEMM_ROWS * TG; e += 256) {
                const int r = e / TG, g = g0 + e % TG;
                const uint32_t at = (uint32_t)(r < rows ? r : rows - 1) * (uint32_t)L.n_groups + g;
                if (g < L.n_groups) tab[(e % TG) * GEMM_ROWS + r] = entry(st[at], zt[at]);
            }
        };
        // the slab in which the rows end: zeros behind them
        const int last = (int)(L.d_col - (int64_t)nfull * KS);  // its columns
        auto tail_a = [&]() {
            const uint8_t* xs = xt + (int64_t)nfull * SLAB;
            uint8_t* buf = lds + (nfull & 1) * BM * SLAB;
#pragma unroll
            for (int j = 0; j < AU; ++j) {
                const int u = tid + 256 * j, c = u % (SLAB / 16), have = last * XB - 16 * c;
                u32x4_t v = {0u, 0u, 0u, 0u};
                if (have >= 16) __builtin_memcpy(&v, xs + aoff[j], 16);
                uint8_t* dst = buf + slab_at(u / (SLAB / 16), c);
                *reinterpret_cast<u32x4_t*>(dst) = v;
                for (int e = 0; e < have && have < 16; e += XB) {   // the piece in which they end
                    if constexpr (XB == 1) dst[e] = xs[aoff[j] + e];
                    else __builtin_memcpy(dst + e, xs + aoff[j] + e, 2);
                }
            }
        };
        auto tail_b = [&](Codes& b) {
            const uint8_t* cs = ct + (int64_t)nfull * (KS / 8 * CB);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int p = 0; p < PP; ++p) {
                    const int left = last - p * PC - cpart * RUN;
                    b.c[nt][p] = load_raw_tail<CB, RUN>(cs + boff[nt] + p * (PC / 8 * CB), left < RUN ? left : RUN);
                }
        };

        Entry rowE[NT];                                        // PIECE 0: the row's scale and zero
        bool row_rest = false;
        if constexpr (PIECE == 0) {
            bool r = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                rowE[nt] = entry(st[soff[nt]], zt[soff[nt]]);
                r = r || !(f16_bits_to_f32((uint16_t)(rowE[nt].z & 0xFFFFu)) - part_of(rowE[nt].z >> 16) == 0.f);
            }
            row_rest = __ballot(r) != 0;
        }
        sum_t cs[PIECE == 0 ? MT : 1][NT], xs[PIECE == 0 ? MT : 1];   // PIECE 0: the row's running sums
        if constexpr (PIECE == 0) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                xs[mt] = sum_t{0, 0, 0, 0};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) cs[mt][nt] = sum_t{0, 0, 0, 0};
            }
        } else {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }

        auto decode = [&](Operand& o, const Codes& b, int s) {
#pragma unroll
            for (int p = 0; p < PP; ++p) {
                int g = PIECE ? (s * KS + p * PC) >> L.gshift : 0;
                g = g < L.n_groups ? g : L.n_groups - 1;       // pieces behind the row
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    Entry e;
                    if constexpr (PIECE != 0) e = tab[(g % TG) * GEMM_ROWS + 32 * wave + 16 * nt + n16];
                    else e = rowE[nt];
                    o.S[p][nt] = e.S;
                    Raw<CB, RUN> codes = b.c[nt][p];
#pragma unroll
                    for (int w = 0; w < (SPREAD ? (CB * RUN + 31) / 32 : 0); ++w)
                        codes.w[w] = (uint32_t)__builtin_amdgcn_ds_bpermute(4 * (4 * n16 + q), (int)codes.w[w]);
                    o.rz[p][nt] = f16_bits_to_f32((uint16_t)(e.z & 0xFFFFu)) - part_of(e.z >> 16);
#pragma unroll
                    for (int t = 0; t < STEPS; ++t) o.f[p][nt][t] = frag_b(codes, t, e.z);
                }
            }
        };
        auto step = [&](const Operand& o, int s) {
            const uint8_t* buf = lds + (s & 1) * BM * SLAB;
#pragma unroll
            for (int p = 0; p < PP; ++p) {
                if constexpr (PIECE == 0) {
                    row_products(cs, o.f[p], buf, p);
                } else {
                    products(acc, o.f[p], buf, p, o.S[p]);
                    bool r = false;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) r = r || !(o.rz[p][nt] == 0.f);
                    if (__ballot(r) != 0) rests(acc, buf, p, o.S[p], o.rz[p]);
                }
            }
            if (PIECE == 0 && row_rest) piece_sums(xs, buf);
        };

        // Whole slabs: slab s + 1 is on its way into registers while slab s is multiplied.
        u32x4_t a[AU];
        Codes b;
        Operand o;
        if constexpr (PIECE != 0) fill(0);
        if (nfull > 0) { load_a(a, 0); load_b(b, 0); store_a(a, 0); }
        auto begin = [&](int s) {
            __syncthreads();
            const int g = PIECE ? (s * KS) >> L.gshift : 0;
            const int before = PIECE && s ? ((s - 1) * KS) >> L.gshift : 0;
            if (PIECE && g / TG != before / TG) { fill(g); __syncthreads(); }
        };
        int s = 0;
        for (; s < nfull; ++s) {
            begin(s);
            decode(o, b, s);
            if (s + 1 < nfull) { load_a(a, s + 1); load_b(b, s + 1); }
            __builtin_amdgcn_sched_barrier(0);                 // the loads leave before the products begin
            step(o, s);
            if (s + 1 < nfull) store_a(a, s + 1);
        }
        if (nslab > nfull) {                                   // the slab in which the rows end
            begin(s);
            tail_a();
            tail_b(b);
            __syncthreads();
            decode(o, b, s);
            step(o, s);
        }
        if constexpr (PIECE == 0) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float rz = f16_bits_to_f32((uint16_t)(rowE[nt].z & 0xFFFFu)) - part_of(rowE[nt].z >> 16);
                    settle(cs[mt][nt]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float sum = (float)cs[mt][nt][i], less = fmaf(-rz, (float)xs[mt][i], sum);
                        acc[mt][nt][i] = rowE[nt].S * (X != X_I8 && rz == 0.f ? sum : less);   // as in rests
                    }
                }
        }
    }

    // f(mt, i, token) for the lane's token rows; rows past the end are given the last token.
    template <typename F>
    static GPTQ_DEV void each_token(int64_t n, int64_t tok0, F&& f) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t t = tok0 + 16 * mt + 4 * ((threadIdx.x & 63) >> 4) + i;
                f(mt, i, t < n ? t : n - 1);
            }
    }

    template <gptq_dtype YT>
    static GPTQ_DEV void write(const f32x4_t (&acc)[MT][NT], void* y, int64_t d_row, int64_t n, int64_t tok0, int64_t row0) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t t = tok0 + 16 * mt + 4 * (lane >> 4) + i;
                if (t >= n) continue;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int64_t r = row0 + 32 * wave + 16 * nt + (lane & 15);
                    if (r < d_row) store_as<YT>(y, t * d_row + r, acc[mt][nt][i]);
                }
            }
    }

private:
    static GPTQ_DEV sum_t product(const Frag& a, const Frag& b, sum_t c) {
        if constexpr (KB == 8) return mfma8_i8(a.w[0], a.w[1], b.w[0], b.w[1], c);
        else return mfma16<X>(u32x4_t{a.w[0], a.w[1], a.w[2], a.w[3]}, u32x4_t{b.w[0], b.w[1], b.w[2], b.w[3]}, c);
    }
    // the lane's operand of product t of piece p, token row `row` of the tile
    static GPTQ_DEV Frag frag_a(const uint8_t* buf, int row, int p, int t) {
        const int q = (threadIdx.x & 63) >> 4, byte = (p * PC + q * RUN) * XB + t * KB;
        Frag f;
        __builtin_memcpy(f.w, __builtin_assume_aligned(buf + slab_at(row, byte >> 4) + (KB == 8 ? (byte & 8) : 0), KB), KB);
        return f;
    }
    static GPTQ_DEV Frag frag_b(const Raw<CB, RUN>& c, int t, uint32_t z) {   // z: an Entry's
        Frag f;
        if constexpr (X == X_I8) {
            const uint32_t zz = __builtin_amdgcn_perm(z, z, 0x02020202u);   // the byte four times
            // as whole numbers zc 0x01010101 = zz less 2^8 + 2^16 + 2^24 for a negative zc; the
            // bytes of 128 + u - zc, taken modulo 256 each, want no borrow between them
            const uint32_t zw = zz - ((zz & 0x80u) ? 0x01010100u : 0u);
#pragma unroll
            for (int e = 0; e < KB / 4; ++e) f.w[e] = minus_zero_i8<CB>(code_bytes4<CB, RUN>(c, KB / 4 * t + e), zw);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t o[2];
                const uint32_t u4 = code_bytes4<CB, RUN>(c, 2 * t + h);
                if constexpr (X == X_F16) minus_zero_f16(u4, __builtin_amdgcn_perm(z, z, 0x03020302u), o);
                else minus_zero_bf16(u4, __uint_as_float(z & 0xFFFF0000u), o);
                f.w[2 * h] = o[0];
                f.w[2 * h + 1] = o[1];
            }
        }
        return f;
    }
    static GPTQ_DEV Frag ones() {
        Frag f;
#pragma unroll
        for (int e = 0; e < KB / 4; ++e) f.w[e] = ones_word<X>();
        return f;
    }

    // Products of one piece, scaled into acc.  A token tile's products are issued before the
    // last one's sums are scaled, so that the vector unit works while the matrix unit does.
    static GPTQ_DEV void products(f32x4_t (&acc)[MT][NT], const Frag (&bf)[NT][STEPS], const uint8_t* buf, int p,
                                  const float (&S)[NT]) {
        const int n16 = threadIdx.x & 15;
        sum_t cs[2][NT];
        constexpr int AHEAD = 2;                               // token tiles whose fragments are on their way
        Frag a[AHEAD + 1][STEPS];
#pragma unroll
        for (int m = 0; m < AHEAD; ++m)
#pragma unroll
            for (int t = 0; t < STEPS; ++t) a[m][t] = frag_a(buf, 16 * m + n16, p, t);
#pragma unroll
        for (int mt = 0; mt <= MT; ++mt) {
            __builtin_amdgcn_sched_barrier(0);
            if (mt + AHEAD < MT) {
#pragma unroll
                for (int t = 0; t < STEPS; ++t) a[(mt + AHEAD) % (AHEAD + 1)][t] = frag_a(buf, 16 * (mt + AHEAD) + n16, p, t);
            }
            if (mt < MT) {
#pragma unroll
                for (int t = 0; t < STEPS; ++t)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        cs[mt & 1][nt] = product(a[mt % (AHEAD + 1)][t], bf[nt][t], t == 0 ? sum_t{0, 0, 0, 0} : cs[mt & 1][nt]);
            }
            if (mt > 0) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[mt - 1][nt][i] = fmaf(S[nt], (float)cs[(mt - 1) & 1][nt][i], acc[mt - 1][nt][i]);
            }
            // one product, then its share of the scaling, so that both units are fed
            constexpr int V = 8 * NT / (STEPS * NT);
#pragma unroll
            for (int k = 0; k < STEPS * NT; ++k) {
                if (k == 0) __builtin_amdgcn_sched_group_barrier(0x100, STEPS, 0);   // the next tile's LDS reads
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                   // MFMA
                __builtin_amdgcn_sched_group_barrier(0x002, V, 0);                   // VALU
            }
        }
    }

    // What the zeros' rests take off a piece: (z - zc) sum x.
    static GPTQ_DEV void rests(f32x4_t (&acc)[MT][NT], const uint8_t* buf, int p, const float (&S)[NT], const float (&rz)[NT]) {
        const int n16 = threadIdx.x & 15;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            sum_t xs = {0, 0, 0, 0};
#pragma unroll
            for (int t = 0; t < STEPS; ++t) xs = product(frag_a(buf, 16 * mt + n16, p, t), ones(), xs);
            settle(xs);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float less = fmaf(-S[nt] * rz[nt], (float)xs[i], acc[mt][nt][i]);
                    // no rest, no sum of x: it may be infinite
                    acc[mt][nt][i] = X != X_I8 && rz[nt] == 0.f ? acc[mt][nt][i] : less;
                }
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    static GPTQ_DEV void row_products(sum_t (&cs)[PIECE == 0 ? MT : 1][NT], const Frag (&bf)[NT][STEPS], const uint8_t* buf,
                                      int p) {
        const int n16 = threadIdx.x & 15;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int t = 0; t < STEPS; ++t) {
                const Frag a = frag_a(buf, 16 * mt + n16, p, t);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) cs[mt][nt] = product(a, bf[nt][t], cs[mt][nt]);
            }
    }

    // sum x of a slab, per token
    static GPTQ_DEV void piece_sums(sum_t (&xs)[PIECE == 0 ? MT : 1], const uint8_t* buf) {
        const int n16 = threadIdx.x & 15;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int p = 0; p < PP; ++p)
#pragma unroll
                for (int t = 0; t < STEPS; ++t) xs[mt] = product(frag_a(buf, 16 * mt + n16, p, t), ones(), xs[mt]);
            settle(xs[mt]);
        }
    }
};

}  // namespace gptq
