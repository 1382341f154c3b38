// The gradient through products grouped by expert (gptqt_linear_grouped_backward):
//   dx[t] = What_e^T dy[t] for the rows t of expert e.
//
// Launches: the rows' exponents and Quads; dy as fp16 rows (back_pack_kernel), each element times
// its weight row's power of two and all of a token's times one, which brings the largest to
// 2^14 .. 2^15: bfloat16 and fp16 elements down to 2^-28 of it are themselves, smaller ones are
// off by 2^-39 of it at most; the product (back_gemm.h).  Where its tiles would leave CUs
// without work, the weight rows are split among workgroups, whose fp32 sums back_join_kernel
// adds in order.
//
// The product has no place for a row of dy with an infinity or a NaN: a second part of a weight may
// be zero or of the other sign than the first, and the slabs that end a turn multiply the last
// rows of dy by zeros.  back_pack_kernel writes dx of such a row itself and marks it, and the
// kernels behind it leave the marked rows alone.

#include "back_gemm.h"

namespace gptq {

struct PackArgs {
    const void* dy; int64_t ldy, n, d_row;
    const int8_t* e;
    const int32_t* offsets; int E;
    uint16_t* A; int64_t lda; int32_t* shift;
    Stored L; int bits;
    void* dx; gptq_dtype dxt;
};

constexpr int NOT_FINITE = 2000;                                // the exponent of an infinity or a NaN, and the mark of its row

// dx of a row with infinities or NaNs, by the whole workgroup: those elements alone decide it, the
// sum of their products (an infinity with the weights' sign; NaN of a zero weight, of both signs or
// of a NaN).  A column per thread; mask: which of 2048 elements of dy count; open: whether a wave has
// a sum that is not NaN, behind which nothing changes.  Kept small: with 8 columns per thread its
// registers cost the rows without any (2048 x 11008: 26 -> 29.5 us).  2048 rows x 11008 x 4096, 210 us:
// 430 with an infinity in one row, 510 in each, 280 with nothing but NaNs.
template <int X>
GPTQ_DEV void not_finite_row(const PackArgs& a, const uint16_t* row, const Segment& s, uint64_t* mask, int* open) {
    const Stored L = expert_of(a.L, a.d_row, s.e);
    const int tid = threadIdx.x;
    for (int64_t c0 = 0; c0 < L.d_col; c0 += 256) {
        const int64_t c = c0 + tid < L.d_col ? c0 + tid : L.d_col - 1;
        float sum = 0.f;
        for (int64_t r0 = 0; r0 < a.d_row; r0 += 2048) {
            const int64_t r = r0 + 8 * tid;
            reinterpret_cast<uint8_t*>(mask)[tid] = (uint8_t)(r < a.d_row ? not_finite8<X>(row + r, (int)(a.d_row - r < 8 ? a.d_row - r : 8)) : 0);
            __syncthreads();
#pragma unroll 1
            for (int w = 0; w < 32; ++w)
#pragma unroll 1
                for (uint64_t left = mask[w]; left != 0 && __ballot(sum == sum) != 0; left &= left - 1) {
                    const int64_t at = r0 + 64 * w + __builtin_ctzll(left);
                    const float v = X == X_BF16 ? bf16_bits_to_f32(row[at]) : f16_bits_to_f32(row[at]);
                    sum = fmaf(v, weight_at(L, a.bits, at, c), sum);
                }
            const int any = __ballot(sum == sum) != 0;
            if ((tid & 63) == 0) open[tid >> 6] = any;
            __syncthreads();                                     // and the reading of the mask is over
            if ((open[0] | open[1] | open[2] | open[3]) == 0) break;
        }
        if (c0 + tid < L.d_col) store_out(a.dx, a.dxt, s.tok0 * L.d_col + c, sum);
    }
}

// A workgroup per row, 8 elements per thread and step.  2048 x 11008 bfloat16, 90 MB, 26 us: memory, and
// the maximum's round trip before the second reading.
template <gptq_dtype T>
__global__ __launch_bounds__(256) void back_pack_kernel(PackArgs a) {
    constexpr int X = T == GPTQ_BF16 ? X_BF16 : X_F16;
    __shared__ int red[4];
    __shared__ uint64_t mask[32];
    Segment s;
    if (!segment_of(a.offsets, a.E, a.n, 1, (int)blockIdx.x, s)) return;   // tiles of one row: rows of experts alone
    const int64_t t = s.tok0;
    const int8_t* e = a.e + (int64_t)s.e * a.d_row;
    const uint16_t* row = reinterpret_cast<const uint16_t*>(a.dy) + t * a.ldy;
    auto eight = [&](int64_t r, float (&v)[8], int (&ev)[8]) {
        const int have = (int)(a.d_row - r < 8 ? a.d_row - r : 8);
        load_x8<X>(row + r, have, v);
        if (have == 8) {
            int8_t b[8];
            __builtin_memcpy(b, e + r, 8);
#pragma unroll
            for (int i = 0; i < 8; ++i) ev[i] = b[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) ev[i] = i < have ? e[r + i] : 0;
        }
    };
    int m = -1000;
    float none = 0.f;                                            // NaN behind an infinity or a NaN
    for (int64_t r = 8 * threadIdx.x; r < a.d_row; r += 2048) {
        float v[8];
        int ev[8];
        eight(r, v, ev);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int k = v[i] == 0.f ? -1000 : __builtin_amdgcn_frexp_expf(v[i]) - 1 + ev[i];
            m = k > m ? k : m;
            none = fmaf(v[i], 0.f, none);
        }
    }
    if (none != 0.f) m = NOT_FINITE;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
        const int v = __shfl_xor(m, o);
        m = v > m ? v : m;
    }
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) m = red[w] > m ? red[w] : m;
    const int k = m < -900 || m == NOT_FINITE ? 0 : 14 - m;      // nothing but zeros, or no matter
    if (threadIdx.x == 0) a.shift[t] = m == NOT_FINITE ? NOT_FINITE : k;
    for (int64_t r = 8 * threadIdx.x; r < a.lda; r += 2048) {
        u32x4_t o = {0u, 0u, 0u, 0u};
        if (r < a.d_row) {
            float v[8];
            int ev[8];
            eight(r, v, ev);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = f32_to_f16_bits(__builtin_amdgcn_ldexpf(v[2 * i], ev[2 * i] + k)) |
                       ((uint32_t)f32_to_f16_bits(__builtin_amdgcn_ldexpf(v[2 * i + 1], ev[2 * i + 1] + k)) << 16);
        }
        *reinterpret_cast<u32x4_t*>(a.A + ((r / BK) * a.n + t) * BK + r % BK) = o;
    }
    if (m == NOT_FINITE) not_finite_row<X>(a, row, s, mask, red);   // the whole workgroup
}

GPTQ_DEV void store_scaled(const BackArgs& a, int64_t at, f32x4_t v, int shift, int have) {
    if (shift == NOT_FINITE) return;                             // back_pack_kernel wrote the row
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ldexpf(v[i], -shift);
    if (a.yt == GPTQ_F32) store_four<GPTQ_F32>(a.y, at, v, have);
    else if (a.yt == GPTQ_BF16) store_four<GPTQ_BF16>(a.y, at, v, have);
    else store_four<GPTQ_F16>(a.y, at, v, have);
}

// (8-bit codes with two parts: LDS holds one workgroup of 128 x 128)
template <int CB, int PB, int MT, int WC, bool DIRECT>
__global__ __launch_bounds__(128 * WC, CB != 8 || PB == 1 || MT == 1 ? 2 : 1) void back_gemm_kernel(BackArgs a, int gm, int gn) {
    typedef BackGemm<CB, 1, PB, MT, 2, WC, DIRECT> G;
    __shared__ __align__(16) uint8_t lds[G::LDS_BYTES];
    int tm, tn;
    tile_of(gm, gn, tm, tn);
    Segment s;
    if (!segment_of(a.offsets, a.E, a.n, G::BM, tm, s)) return;
    const int64_t c0 = (int64_t)tn * G::BN, k0 = blockIdx.y * a.share, k1 = k0 + a.share < a.d_row ? k0 + a.share : a.d_row;
    f32x4_t acc[G::NI][MT];
    G::run(acc, a, expert_of(a.L, a.d_row, s.e), a.T + s.e * a.quads * a.L.n_groups, s.tok0, s.end, c0, k0, k1, lds);
    float* sums = a.sums ? a.sums + blockIdx.y * a.n * a.L.d_col : nullptr;
    G::each(acc, s.tok0, s.end, c0, a.L.d_col, [&](int64_t c, int64_t t, f32x4_t v, int have) {
        const int64_t at = t * a.L.d_col + c;
        if (sums) store_four<GPTQ_F32>(sums, at, v, have);
        else store_scaled(a, at, v, a.shift[t], have);
    });
}

// The shares' sums of one row of an expert, in order.  2048 x 4096, two shares, 84 MB: 18 us (4.6 TB/s).
__global__ __launch_bounds__(256) void back_join_kernel(BackArgs a, int shares) {
    Segment s;
    if (!segment_of(a.offsets, a.E, a.n, 1, (int)blockIdx.x, s)) return;
    const int64_t t = s.tok0, c = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 4;
    const int have = (int)(a.L.d_col - c < 4 ? a.L.d_col - c : 4);
    if (have <= 0) return;
    const float* p = a.sums + t * a.L.d_col + c;
    const int64_t step = a.n * a.L.d_col;
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    if (have == 4) {
#pragma unroll 4
        for (int i = 0; i < shares; ++i) {
            f32x4_t w;
            __builtin_memcpy(&w, p + i * step, 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] += w[j];
        }
    } else {
        for (int i = 0; i < shares; ++i)
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (j < have) v[j] += p[i * step + j];
    }
    store_scaled(a, t * a.L.d_col + c, v, a.shift[t], have);
}

template <int CB, int PB, int MT, int WC>
static void launch_tiles(BackArgs a, int places, hipStream_t s) {
    typedef BackGemm<CB, 1, PB, MT, 2, WC, true> G;
    const int gm = (int)most_tiles(a.offsets, a.E, a.n, G::BM), gn = (int)((a.L.d_col + G::BN - 1) / G::BN);
    int shares = (int)shares_of((int64_t)gm * gn, places, a.d_row, a.n * a.L.d_col * 4);
    a.share = ((a.d_row + shares - 1) / shares + 63) / 64 * 64;
    shares = (int)((a.d_row + a.share - 1) / a.share);
    if (shares == 1) a.sums = nullptr;
    const dim3 grid((unsigned)(gm * gn), (unsigned)shares);
    if (direct_codes(a.L)) back_gemm_kernel<CB, PB, MT, WC, true><<<grid, G::THREADS, 0, s>>>(a, gm, gn);
    else back_gemm_kernel<CB, PB, MT, WC, false><<<grid, G::THREADS, 0, s>>>(a, gm, gn);
    if (shares > 1) back_join_kernel<<<dim3((unsigned)a.n, (unsigned)((a.L.d_col + 1023) / 1024)), 256, 0, s>>>(a, shares);
}

template <int CB, int PB>
static void launch_parts(const BackArgs& a, hipStream_t s) {
    const SumTile t = sum_tile(ceil_div(a.n, a.E), PB, CB);
    if constexpr (PB == 1) if (t.bm == 256) return launch_tiles<CB, PB, 8, 4>(a, t.places, s);
    if (t.bm == 128) launch_tiles<CB, PB, 4, 2>(a, t.places, s);
    else launch_tiles<CB, PB, 1, 2>(a, t.places, s);
}

template <int CB>
static void launch_gemm(const BackArgs& a, hipStream_t s) {
    if (a.yt == GPTQ_BF16) launch_parts<CB, 1>(a, s);
    else launch_parts<CB, 2>(a, s);
}

static int64_t padded(int64_t d_row) { return (d_row + 63) / 64 * 64; }

// Sums: as many shares as there may be, and no more than MOST_SUMS.
size_t back_ws_bytes(int64_t n, int64_t E, int64_t d_row, int64_t d_col, int group) {
    const int64_t shares = (d_row + 255) / 256, sums = n * d_col * 4;
    const int64_t all = shares == 1 ? 0 : sums > MOST_SUMS / shares ? MOST_SUMS : sums * shares;
    return up256((size_t)(n * padded(d_row)) * 2) + up256((size_t)n * 4) + up256((size_t)(E * d_row)) +
           up256(quads_bytes(E, d_row, group ? d_col / group : 1)) + up256((size_t)all);
}

gptq_status back_launch(const BackCall& c, hipStream_t s) {
    const int64_t lda = padded(c.d_row);
    uint8_t* w = (uint8_t*)c.ws;
    auto take = [&](size_t bytes) { uint8_t* at = w; w += up256(bytes); return at; };
    uint16_t* A = (uint16_t*)take((size_t)(c.n * lda) * 2);
    int32_t* shift = (int32_t*)take((size_t)c.n * 4);
    int8_t* e = (int8_t*)take((size_t)(c.E * c.d_row));
    Quad* T = (Quad*)take(quads_bytes(c.E, c.d_row, c.L.n_groups));
    BackArgs a = {};
    a.L = c.L; a.d_row = c.d_row; a.n = c.n; a.offsets = c.offsets; a.E = c.E;
    a.A[0] = A; a.shift = shift; a.T = T; a.quads = quads_of(c.d_row);
    a.sums = (float*)w;
    a.y = c.dx; a.yt = c.dxt;
    rows_launch(c.L, c.E, c.d_row, e, T, s);
    GPTQ_LAUNCH_CHECK();
    const PackArgs p = {c.dy, c.ldy, c.n, c.d_row, e, c.offsets, c.E, A, lda, shift, c.L, c.bits, c.dx, c.dxt};
    if (c.dyt == GPTQ_BF16) back_pack_kernel<GPTQ_BF16><<<(unsigned)c.n, 256, 0, s>>>(p);
    else back_pack_kernel<GPTQ_F16><<<(unsigned)c.n, 256, 0, s>>>(p);
    GPTQ_LAUNCH_CHECK();
    if (c.bits == 3) launch_gemm<3>(a, s);
    else if (c.bits == 4) launch_gemm<4>(a, s);
    else launch_gemm<8>(a, s);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

}  // namespace gptq
