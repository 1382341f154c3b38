// Products of 16-token tiles with 16-row blocks of a stored layer on the matrix cores,
// shared by the serving kernels (8-bit and 16-bit activations).
//
// A chunk is 128 columns of a row.  A piece is the part of a chunk that has one scale:
// 128 columns (groups of whole chunks, or one scale per row), 64 or 32.  Lane l of a wave
// holds, of every piece, the RUN = piece / 4 columns RUN (l / 16) .. + RUN - 1 of weight
// row l % 16 and of token l % 16, so that each column of the piece enters one product
// once; which k a column has inside a product is the same on both sides and changes
// nothing else.  The sums of a piece (exact integers for 8-bit activations) are scaled by
// S and added in fp32.
//
// Zeros: the operand is u - zc with zc = z rounded to a whole number and clamped so that
// u - zc is exact in the operand's type (8 bits: u - 128 for 8-bit codes, zc in -112 ..
// 127 for narrower ones; 16 bits: |u - zc| <= 256, or zc = 0 for 3- and 4-bit codes, see
// plain_16).  What that leaves of z is taken off the piece as (z - zc) sum x, with sum x
// from a product of the same activations with ones, so every zero is served with exact
// operands.
//
// No unit is busy in these kernels (48 tokens x 11008 x 4096 int4 g64, 8-bit rows: matrix unit 4%
// of the cycles, vector unit 27%, 0.2 L1 accesses per cycle and CU; 40 tokens with adapters
// 5%, 17%, 0.16): waves wait for their loads.  From 33 tokens on a wave has one chunk in
// registers, so nothing is in flight while it multiplies, and two to four waves per SIMD are
// too few to cover it.  Fewer and wider loads shorten the wait: a lane's 16-byte load of a
// row of its own is an L1 access, four neighbouring lanes reading one row are a quarter each.
// So codes and the activations of several tiles are loaded contiguously and handed to their
// lanes across the wave or through LDS (the 48 tokens: 25 us with every lane loading its own,
// 21 with codes contiguous, 17 with both); the scales and zeros of two row blocks come in one
// load (33 -> 26 us with the rows without tokens skipped).  Whole chunks loaded two ahead cost
// registers, hence workgroups, and measured the same or slower.  With groups of 32 (and of
// 64, four tiles) the chunk's pieces do not fit the registers beside the sums, and spill.
#pragma once
#include "common.h"

namespace gptq {

constexpr int SCK = 128;                      // columns per chunk
constexpr int X_I8 = 0, X_BF16 = 1, X_F16 = 2;

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

template <int X> constexpr int xbytes() { return X == X_I8 ? 1 : 2; }

// ---- codes of RUN consecutive columns, as stored
template <int CB, int RUN>
struct Raw { uint32_t w[(CB * RUN + 31) / 32]; };

template <int CB, int RUN>
GPTQ_DEV Raw<CB, RUN> load_raw(const uint8_t* p) {    // any alignment
    Raw<CB, RUN> r;
    r.w[(CB * RUN + 31) / 32 - 1] = 0;
    __builtin_memcpy(r.w, p, CB * RUN / 8);
    return r;
}

// The first n of RUN columns (the others 0); n <= 0 reads nothing.
template <int CB, int RUN>
GPTQ_DEV Raw<CB, RUN> load_raw_tail(const uint8_t* p, int n) {
    Raw<CB, RUN> r;
#pragma unroll
    for (int i = 0; i < (CB * RUN + 31) / 32; ++i) r.w[i] = 0;
    const int nb = n > 0 ? (n * CB + 7) / 8 : 0;
#pragma unroll
    for (int i = 0; i < CB * RUN / 8; ++i)
        if (i < nb) r.w[i / 4] |= (uint32_t)p[i] << (8 * (i & 3));
    return r;
}

// Columns 4 j .. 4 j + 3 as unsigned bytes.
template <int CB, int RUN>
GPTQ_DEV uint32_t code_bytes4(const Raw<CB, RUN>& r, int j) {
    if constexpr (CB == 8) {
        return r.w[j];
    } else if constexpr (CB == 4) {
        const uint32_t w = r.w[j >> 1], lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
        return __builtin_amdgcn_perm(hi, lo, (j & 1) ? 0x07030602u : 0x05010400u);
    } else {
        const int bit = 12 * j, k = bit >> 5, sh = bit & 31;
        uint32_t x = r.w[k] >> sh;
        if (sh > 20) x |= r.w[k + 1] << (32 - sh);
        x &= 0xFFFu;
        x = (x | (x << 10)) & 0x003F003Fu;
        return (x | (x << 5)) & 0x07070707u;
    }
}

// The whole-number part of a zero that the operand takes, and as the decoders use it.
template <int X, int CB>
GPTQ_DEV float zero_part(float z) {
    if constexpr (X == X_I8) return CB == 8 ? 128.f : fminf(fmaxf(rintf(z), -112.f), 127.f);
    else return fminf(fmaxf(rintf(z), CB == 8 ? -1.f : -240.f), CB == 8 ? 255.f : 240.f);
}

// u - zc of four columns as signed bytes; zz = zc times 0x01010101.
template <int CB>
GPTQ_DEV uint32_t minus_zero_i8(uint32_t u4, uint32_t zz) {
    if constexpr (CB == 8) return u4 ^ 0x80808080u;
    else return ((u4 | 0x80808080u) - zz) ^ 0x80808080u;   // each byte 128 + u - zc in 0 .. 255: no borrow
}

// u - zc of four columns in a 16-bit type, two per word.
// fp16: 0x6400 | u is 1024 + u; zz is 1024 + zc twice; both and the difference are whole
// numbers below 2048.
GPTQ_DEV void minus_zero_f16(uint32_t u4, uint32_t zz, uint32_t (&o)[2]) {
    const f16x2_t z = __builtin_bit_cast(f16x2_t, zz);
    o[0] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm(0x64646464u, u4, 0x04010400u)) - z);
    o[1] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm(0x64646464u, u4, 0x04030402u)) - z);
}
GPTQ_DEV void minus_zero_bf16(uint32_t u4, float zc, uint32_t (&o)[2]) {
    const f32x2_t a = {(float)(u4 & 0xFFu) - zc, (float)((u4 >> 8) & 0xFFu) - zc};
    const f32x2_t b = {(float)((u4 >> 16) & 0xFFu) - zc, (float)(u4 >> 24) - zc};
    o[0] = __builtin_bit_cast(uint32_t, __builtin_convertvector(a, bf16x2_t));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_convertvector(b, bf16x2_t));
}
// u itself of four columns of 3- or 4-bit codes in a 16-bit type.  A byte below 16 read as
// an FP8 E4M3 number is u 2^-9 (u < 8: the subnormals; 8 to 15: 2^-6 (1 + (u - 8) / 8)),
// and one instruction turns two of them into 16-bit numbers times a power of two: half an
// instruction per code, where a conversion and a subtraction in fp32 take two and a half.
template <int X>
GPTQ_DEV void plain_16(uint32_t u4, uint32_t (&o)[2]) {
    if constexpr (X == X_F16) {
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(u4, 512.f, false));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(u4, 512.f, true));
    } else {
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u4, 512.f, false));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u4, 512.f, true));
    }
}

template <int X>
GPTQ_DEV void minus_zero_16(uint32_t u4, float zc, uint32_t (&o)[2]) {
    if constexpr (X == X_F16) {
        const uint32_t h = __builtin_bit_cast(uint16_t, (_Float16)(1024.f + zc));
        minus_zero_f16(u4, h | (h << 16), o);
    } else {
        minus_zero_bf16(u4, zc, o);
    }
}

// ---- one product: 16-byte operands (8 bytes for 8-bit activations with 32-column pieces)
template <int X> struct Acc { typedef f32x4_t t; };
template <> struct Acc<X_I8> { typedef i32x4_t t; };

template <int X>
GPTQ_DEV typename Acc<X>::t mfma16(u32x4_t a, u32x4_t b, typename Acc<X>::t c) {
    if constexpr (X == X_I8)
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0, 0, 0);
    else if constexpr (X == X_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

GPTQ_DEV i32x4_t mfma8_i8(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1, i32x4_t c) {
    const long a = (long)(((uint64_t)a1 << 32) | a0), b = (long)(((uint64_t)b1 << 32) | b0);
    return __builtin_amdgcn_mfma_i32_16x16x32_i8(a, b, c, 0, 0, 0);
}

template <int X>
GPTQ_DEV constexpr uint32_t ones_word() { return X == X_I8 ? 0x01010101u : X == X_BF16 ? 0x3F803F80u : 0x3C003C00u; }

// Ends a conditional block of products: their results are settled behind it.  This compiler
// (clang 22) counts the wait between a product and a later use of its registers along only
// one of the paths that meet behind a branch, so results that leave the block are waited
// for here: 16 wait states, more than any of these products needs (12).
template <typename V>
GPTQ_DEV void settle(V& v) { asm volatile("s_nop 7\n\ts_nop 7" : "+v"(v)); }

// Orders LDS accesses before it, by any lane of the wave, with those after it: a release and
// an acquire at the wave's scope.  A wave's LDS operations execute in order, so neither costs
// an instruction; they keep the compiler from moving or forwarding accesses across.
GPTQ_DEV void lds_handover() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// ---- activations of RUN columns
template <int X, int RUN>
struct XRun { uint32_t w[RUN * xbytes<X>() / 4]; };

template <int X, int RUN>
GPTQ_DEV XRun<X, RUN> load_x(const uint8_t* p) {
    XRun<X, RUN> r;
    __builtin_memcpy(r.w, p, RUN * xbytes<X>());
    return r;
}

template <int X, int RUN>
GPTQ_DEV XRun<X, RUN> load_x_tail(const uint8_t* p, int n) {   // zeros from column n on
    XRun<X, RUN> r;
#pragma unroll
    for (int i = 0; i < RUN * xbytes<X>() / 4; ++i) r.w[i] = 0;
    if constexpr (X == X_I8) {
#pragma unroll
        for (int i = 0; i < RUN; ++i)
            if (i < n) r.w[i / 4] |= (uint32_t)p[i] << (8 * (i & 3));
    } else {
#pragma unroll
        for (int i = 0; i < RUN; ++i)
            if (i < n) r.w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
    }
    return r;
}

// The stored layer as the kernels take it.
struct Stored {
    const uint8_t* codes; int64_t code_ld;             // bytes per row
    const uint16_t* scales; const uint16_t* zeros;     // fp16, rows x n_groups
    int64_t d_col;
    int n_groups;
    int gshift;                                        // log2 of the group's columns (groups)
};

// The activation rows of NTT tiles of 16 tokens.  Scattered: a pointer per lane to the token
// of row l % 16 of each tile, nullptr for a row without one.
template <int NTT>
struct XScattered {
    const uint8_t* row[NTT];
};
// Consecutive: `live` rows from base on, pitch bytes apart, loaded in contiguous pieces (64
// lanes read 4 or 8 whole rows of a chunk) and put in order through the wave's own `stage`
// in LDS (a tile's chunk: 16 rows x 128 columns).
struct XConsecutive {
    const uint8_t* base; int64_t pitch; int live;
    uint8_t* stage;
};

// What one chunk of RB row blocks and NTT token tiles needs, in registers.
template <int X, int CB, int RUN, int NTT, int RB>
struct Chunk {
    static constexpr int P = 32 / RUN;        // pieces
    static constexpr int SZ = (RB + 1) / 2;
    Raw<CB, RUN> c[RB][P];
    XRun<X, RUN> x[NTT][P];
    // one load fetches the scales and zeros of two row blocks: lane group q holds the scale (q
    // even) or the zero (odd) of block 2 k + q / 2
    uint16_t sz[SZ][P];

    // Codes are loaded by lane l for row l / 4 and lane group l % 4, so that four neighbouring
    // lanes read one contiguous piece of a row (a cache access each 64 bytes instead of one
    // per lane), and handed to the lane that multiplies them (arrange).
    //
    // row[rb]: the row that the lane multiplies; crow[rb]: the row whose codes it loads.  A
    // row of a tile without a token is zeros, and nothing is read for it.  TAIL: the chunk in
    // which the rows end
    template <bool TAIL, typename XR>
    GPTQ_DEV void load(const Stored& L, const int64_t (&row)[RB], const int64_t (&crow)[RB], const XR& xr, int c0) {
        const int q = (threadIdx.x & 63) >> 4, cq = threadIdx.x & 3;
        const uint16_t* tab = (q & 1) ? L.zeros : L.scales;
        int64_t szrow[SZ];
#pragma unroll
        for (int k = 0; k < SZ; ++k) szrow[k] = row[2 * k + 1 < RB && q >= 2 ? 2 * k + 1 : 2 * k] * L.n_groups;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int64_t col = (int64_t)c0 * SCK + p * 4 * RUN + cq * RUN;
            const int left = (int)(L.d_col - col < RUN ? L.d_col - col : RUN);
            int g = RUN == 32 && L.n_groups == 1 ? 0 : c0 * P + p;
            if (TAIL) g = g < L.n_groups ? g : L.n_groups - 1;
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                const uint8_t* src = L.codes + crow[rb] * L.code_ld + col / 8 * CB;
                c[rb][p] = !TAIL ? load_raw<CB, RUN>(src) : load_raw_tail<CB, RUN>(src, left);
            }
#pragma unroll
            for (int k = 0; k < SZ; ++k) sz[k][p] = tab[szrow[k] + g];
        }
        load_x_rows<TAIL>(L, xr, c0);
    }

    template <bool TAIL>
    GPTQ_DEV void load_x_rows(const Stored& L, const XScattered<NTT>& xr, int c0) {
        const int q = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int tt = 0; tt < NTT; ++tt) {
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int e = 0; e < RUN * xbytes<X>() / 4; ++e) x[tt][p].w[e] = 0;
            if (xr.row[tt] != nullptr) {
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const int64_t col = (int64_t)c0 * SCK + p * 4 * RUN + q * RUN;
                    const int left = (int)(L.d_col - col < RUN ? L.d_col - col : RUN);
                    const uint8_t* src = xr.row[tt] + col * xbytes<X>();
                    x[tt][p] = !TAIL ? load_x<X, RUN>(src) : load_x_tail<X, RUN>(src, left);
                }
            }
        }
    }

    static constexpr int PPR = SCK * xbytes<X>() / 16;      // 16-byte pieces of a row's chunk
    static constexpr int XL = 16 * PPR / 64;                // loads per tile

    // piece k of the wave's XL loads of a tile, kept where x is until it is put in order
    GPTQ_DEV uint32_t& x_word(int tt, int w) { return x[tt][w / (RUN * xbytes<X>() / 4)].w[w % (RUN * xbytes<X>() / 4)]; }

    template <bool TAIL>
    GPTQ_DEV void load_x_rows(const Stored& L, const XConsecutive& xr, int c0) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int tt = 0; tt < NTT; ++tt)
#pragma unroll
            for (int k = 0; k < XL; ++k) {
                const int r = 16 * tt + (64 * k + lane) / PPR, piece = (64 * k + lane) % PPR;
                uint32_t v[4] = {0u, 0u, 0u, 0u};
                if (r < xr.live) {
                    const uint8_t* src = xr.base + r * xr.pitch + (int64_t)c0 * SCK * xbytes<X>() + 16 * piece;
                    if constexpr (!TAIL) {
                        __builtin_memcpy(v, src, 16);
                    } else {
                        const int64_t left = L.d_col - (int64_t)c0 * SCK - piece * (16 / xbytes<X>());
                        const XRun<X, 16 / xbytes<X>()> t = load_x_tail<X, 16 / xbytes<X>()>(src, (int)(left < 16 ? left : 16));
                        __builtin_memcpy(v, t.w, 16);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) x_word(tt, 4 * k + e) = v[e];
            }
    }

    GPTQ_DEV void arrange_x(const XScattered<NTT>&) {}
    GPTQ_DEV void arrange_x(const XConsecutive& xr) {
        const int lane = threadIdx.x & 63, n16 = lane & 15, q = lane >> 4;
        constexpr int B = RUN * xbytes<X>();                // bytes of a lane's run
        auto at = [&](int r, int piece) { return xr.stage + (r * PPR + (piece ^ (r & (PPR - 1)))) * 16; };
#pragma unroll
        for (int tt = 0; tt < NTT; ++tt) {
            lds_handover();                                 // the last tile is read
#pragma unroll
            for (int k = 0; k < XL; ++k)
                *reinterpret_cast<u32x4_t*>(at((64 * k + lane) / PPR, (64 * k + lane) % PPR)) =
                    u32x4_t{x_word(tt, 4 * k), x_word(tt, 4 * k + 1), x_word(tt, 4 * k + 2), x_word(tt, 4 * k + 3)};
            lds_handover();
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int byte = p * 4 * B + q * B;
                if constexpr (B >= 16) {
#pragma unroll
                    for (int e = 0; e < B / 16; ++e) {
                        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(at(n16, byte / 16 + e));
#pragma unroll
                        for (int w = 0; w < 4; ++w) x[tt][p].w[4 * e + w] = v[w];
                    }
                } else {
                    __builtin_memcpy(x[tt][p].w, __builtin_assume_aligned(at(n16, byte / 16) + byte % 16, 8), 8);
                }
            }
        }
        lds_handover();
    }

    // lane (row n, group q) takes the codes that lane 4 n + q loaded
    GPTQ_DEV void arrange() {
        const int from = 4 * (4 * (int)(threadIdx.x & 15) + (int)((threadIdx.x & 63) >> 4));
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int e = 0; e < (CB * RUN + 31) / 32; ++e)
                    c[rb][p].w[e] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)c[rb][p].w[e]);
    }

    // scale (which 0) or zero (1) of the lane's row in block rb
    GPTQ_DEV float scale_of(int rb, int p, int which) const {
        const int v = __shfl((int)sz[rb / 2][p], (int)(threadIdx.x & 15) + 16 * (2 * (rb & 1) + which));
        return f16_bits_to_f32((uint16_t)v);
    }

    // 3- and 4-bit codes with 16-bit activations enter as they are (see plain_16); the whole
    // zero is then a rest, taken off with sum x, which all the row blocks share.  The fp32 sums
    // of u x and z x are larger than that of (u - z) x, by up to 2.7 for uniform codes: 1.2e-7
    // of y in the norm in place of 7e-8
    static constexpr bool PLAIN = X != X_I8 && CB != 8;
    typedef typename Acc<X>::t sum_t;

    // sum x of piece p, per token
    GPTQ_DEV void x_sums(float (&xs)[NTT][4], int p) const {
        const uint32_t w1 = ones_word<X>();
#pragma unroll
        for (int tt = 0; tt < NTT; ++tt) {
            sum_t s = {0, 0, 0, 0};
            const uint32_t* a = x[tt][p].w;
            if constexpr (X == X_I8 && RUN == 8) {
                s = mfma8_i8(a[0], a[1], w1, w1, s);
            } else {
#pragma unroll
                for (int t = 0; t < RUN * xbytes<X>() / 16; ++t)
                    s = mfma16<X>(u32x4_t{a[4 * t], a[4 * t + 1], a[4 * t + 2], a[4 * t + 3]}, u32x4_t{w1, w1, w1, w1}, s);
            }
            if constexpr (!PLAIN) settle(s);
#pragma unroll
            for (int i = 0; i < 4; ++i) xs[tt][i] = (float)s[i];
        }
    }

    // acc[tt][rb] += the chunk's sums: lane l's value i the output of weight row l % 16 and
    // token 4 (l / 16) + i
    GPTQ_DEV void multiply(f32x4_t (&acc)[NTT][RB]) const {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            float xs[NTT][4];
            if constexpr (PLAIN) x_sums(xs, p);
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                const float S = scale_of(rb, p, 0), z = scale_of(rb, p, 1);
                const float zc = PLAIN ? 0.f : zero_part<X, CB>(z), rz = z - zc;
                sum_t cs[NTT];
#pragma unroll
                for (int tt = 0; tt < NTT; ++tt) cs[tt] = sum_t{0, 0, 0, 0};
                if constexpr (X == X_I8 && RUN == 8) {
                    const uint32_t zz = (uint32_t)((int)zc * 0x01010101);
                    const uint32_t b0 = minus_zero_i8<CB>(code_bytes4<CB, RUN>(c[rb][p], 0), zz);
                    const uint32_t b1 = minus_zero_i8<CB>(code_bytes4<CB, RUN>(c[rb][p], 1), zz);
#pragma unroll
                    for (int tt = 0; tt < NTT; ++tt) cs[tt] = mfma8_i8(x[tt][p].w[0], x[tt][p].w[1], b0, b1, cs[tt]);
                } else {
#pragma unroll
                    for (int t = 0; t < RUN * xbytes<X>() / 16; ++t) {
                        u32x4_t b;
                        if constexpr (X == X_I8) {
                            const uint32_t zz = (uint32_t)((int)zc * 0x01010101);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                b[e] = minus_zero_i8<CB>(code_bytes4<CB, RUN>(c[rb][p], 4 * t + e), zz);
                        } else {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t o[2];
                                const uint32_t u4 = code_bytes4<CB, RUN>(c[rb][p], 2 * t + h);
                                if constexpr (PLAIN) plain_16<X>(u4, o);
                                else minus_zero_16<X>(u4, zc, o);
                                b[2 * h] = o[0];
                                b[2 * h + 1] = o[1];
                            }
                        }
#pragma unroll
                        for (int tt = 0; tt < NTT; ++tt) {
                            const uint32_t* a = x[tt][p].w + 4 * t;
                            cs[tt] = mfma16<X>(u32x4_t{a[0], a[1], a[2], a[3]}, b, cs[tt]);
                        }
                    }
                }
#pragma unroll
                for (int tt = 0; tt < NTT; ++tt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[tt][rb][i] = fmaf(S, (float)cs[tt][i], acc[tt][rb][i]);
                        if constexpr (PLAIN) acc[tt][rb][i] = fmaf(-S * rz, xs[tt][i], acc[tt][rb][i]);
                    }
                if constexpr (!PLAIN) {
                    if (__ballot(!(rz == 0.f)) != 0) {         // some zero leaves a rest: rz sum x off the piece
                        x_sums(xs, p);
#pragma unroll
                        for (int tt = 0; tt < NTT; ++tt)
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[tt][rb][i] = fmaf(-S * rz, xs[tt][i], acc[tt][rb][i]);
                    }
                }
            }
        }
    }
};

// Sums of RB blocks of 16 weight rows with NTT tiles of 16 tokens over the chunks c0, c0 +
// step, .. of a row.  DEEP chunks are in registers at a time: with two, one is multiplied
// while the other is on its way; with one, only other waves' work covers its round trip.
template <int X, int CB, int RUN, int NTT, int RB, int DEEP, typename XR>
GPTQ_DEV void stored_accumulate(f32x4_t (&acc)[NTT][RB], const Stored& L, const int64_t (&row)[RB], const XR& xr, int c0,
                                int step) {
    const int nfull = (int)(L.d_col / SCK);
    // the rows whose codes the lane loads: those that lane l / 4 of the wave multiplies
    int64_t crow[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) crow[rb] = __shfl(row[rb], (int)(threadIdx.x & 63) >> 2);
    Chunk<X, CB, RUN, NTT, RB> ch[DEEP];
#pragma unroll
    for (int j = 0; j < DEEP; ++j)
        if (c0 + j * step < nfull) ch[j].template load<false>(L, row, crow, xr, c0 + j * step);
    __builtin_amdgcn_sched_barrier(0);         // every load above the arithmetic
    for (int c = c0; c < nfull; c += DEEP * step) {
#pragma unroll
        for (int j = 0; j < DEEP; ++j) {
            const int at = c + j * step, next = at + DEEP * step;
            if (at < nfull) {                  // wave-uniform
                ch[j].arrange();
                ch[j].arrange_x(xr);
                ch[j].multiply(acc);
                if (next < nfull) ch[j].template load<false>(L, row, crow, xr, next);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    if (L.d_col % SCK && nfull >= c0 && (nfull - c0) % step == 0) {
        ch[0].template load<true>(L, row, crow, xr, nfull);
        ch[0].arrange();
        ch[0].arrange_x(xr);
        ch[0].multiply(acc);
    }
}

// What[r] x by a whole wave as the definition has it, sum S (u - z) x: for sums that came out
// as no number (see finite_sum).  x8(c, m, v) gives the m elements of x from column c on, m <=
// 8.  8 columns per lane and step.
template <int CB, typename F>
GPTQ_DEV float wave_sum(const Stored& L, int64_t r, F&& x8) {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));             // addresses are formed here, not carried through the kernel
    float s = 0.f;
#pragma unroll 1
    for (int64_t c0 = 0; c0 < L.d_col && __ballot(s != s) == 0; c0 += 512) {   // a NaN stays one
        const int64_t c = c0 + 8 * lane;
        if (c < L.d_col) {
            const int m = L.d_col - c < 8 ? (int)(L.d_col - c) : 8;
            const uint8_t* src = L.codes + r * L.code_ld + c / 8 * CB;
            const Raw<CB, 8> u = m == 8 ? load_raw<CB, 8>(src) : load_raw_tail<CB, 8>(src, m);
            const int64_t at = r * L.n_groups + (L.n_groups == 1 ? 0 : c >> L.gshift);   // a group is whole steps
            const float S = f16_bits_to_f32(L.scales[at]), z = f16_bits_to_f32(L.zeros[at]);
            float x[8];
            x8(c, m, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float w = S * ((float)((code_bytes4<CB, 8>(u, e >> 2) >> (8 * (e & 3))) & 0xFFu) - z);
                if (e < m) s = fmaf(w, x[e], s);
            }
        }
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o);
    return s;
}

// v, the lane's sum, or where that is not finite the sum taken again with wave_sum.  The
// kernels' products can lose it: u x - z x, of codes that enter as they are, is infinity -
// infinity for an infinite x, and so is what a zero's rest takes off; and sums of u x may
// overflow where those of S (u - z) x do not.  The others keep their bits.  row_of(i) and
// x8(i, ..) give thread i's row and its token's data.  The whole wave calls it; lanes
// without an output pass live = false.
template <int CB, typename R, typename F>
GPTQ_DEV float finite_sum(float v, bool live, const Stored& L, R&& row_of, F&& x8) {
    uint64_t todo = __ballot(live && !(fabsf(v) < INFINITY));
    while (todo) {                                                 // wave-uniform, rare
        const int l = __builtin_ctzll(todo), i = __builtin_amdgcn_readfirstlane((int)threadIdx.x & ~63) + l;
        todo &= todo - 1;
        const float s = wave_sum<CB>(L, row_of(i), [&](int64_t c, int m, float (&x)[8]) { x8(i, c, m, x); });
        if ((int)(threadIdx.x & 63) == l) v = s;
    }
    return v;
}

// Eight 16-bit elements from p on, the first m of which exist.
template <int X>
GPTQ_DEV void load_x8(const uint16_t* p, int m, float (&v)[8]) {
    const uint8_t* b = reinterpret_cast<const uint8_t*>(p);
    const XRun<X, 8> r = m == 8 ? load_x<X, 8>(b) : load_x_tail<X, 8>(b, m);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint16_t h = (uint16_t)(r.w[e / 2] >> (16 * (e & 1)));
        v[e] = X == X_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h);
    }
}

// An fp32 number as bfloat16 parts: each the nearest to what the ones before leave (toward
// zero where the nearest is infinite).  The first two leave at most 2^-17 of it (it is in 2^e
// .. 2^(e+1), the first leaves at most 2^(e-8), and the second half a step of that at most,
// 2^(e-17)); with the third they are the number itself (what the second leaves is a multiple
// of 2^(e-23) of at most 2^(e-16): 8 bits).  An infinity or a NaN is its first part alone.
GPTQ_DEV void bf16_parts(float v, uint16_t (&p)[3]) {
    const uint32_t u = __float_as_uint(v);
    const bool fin = (u & 0x7f800000u) != 0x7f800000u;
    p[0] = f32_to_bf16_bits(v);
    if (fin && (p[0] & 0x7fffu) == 0x7f80u) p[0] = (uint16_t)(u >> 16);
    const float r = fin ? v - bf16_bits_to_f32(p[0]) : 0.f;
    p[1] = f32_to_bf16_bits(r);
    p[2] = f32_to_bf16_bits(r - bf16_bits_to_f32(p[1]));
}

// One output, rounded once (to nearest even) by the hardware's conversions.
template <gptq_dtype YT>
GPTQ_DEV void store_as(void* y, int64_t idx, float v) {
    if constexpr (YT == GPTQ_F32) reinterpret_cast<float*>(y)[idx] = v;
    else if constexpr (YT == GPTQ_BF16) reinterpret_cast<__bf16*>(y)[idx] = (__bf16)v;
    else reinterpret_cast<_Float16*>(y)[idx] = (_Float16)v;
}

GPTQ_DEV void store_out(void* y, gptq_dtype t, int64_t idx, float v) {
    if (t == GPTQ_F32) store_as<GPTQ_F32>(y, idx, v);
    else if (t == GPTQ_BF16) store_as<GPTQ_BF16>(y, idx, v);
    else store_as<GPTQ_F16>(y, idx, v);
}

// Host: the stored layer's layout; group 0 = one scale per row.
inline Stored stored_layer(const uint8_t* codes, const uint16_t* scales, const uint16_t* zeros, int64_t d_col, int bits,
                           int group) {
    Stored L;
    L.codes = codes; L.code_ld = bits == 3 ? d_col / 8 * 3 : bits == 4 ? d_col / 2 : d_col;
    L.scales = scales; L.zeros = zeros; L.d_col = d_col;
    L.gshift = group == 32 ? 5 : group == 64 ? 6 : 7;
    L.n_groups = group > 0 ? (int)(d_col / group) : 1;
    return L;
}

}  // namespace gptq
