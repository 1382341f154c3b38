// The gradient through products grouped by expert (gptqt_linear_grouped_backward):
//   dx[t] = What_e^T dy[t] for the rows t of expert e.
//
// Three launches: the rows' exponents; dy as fp16 rows (back_pack_kernel), each element times
// its weight row's power of two and all of a token's times one, which brings the largest to
// 2^14 .. 2^15: bfloat16 and fp16 elements down to 2^-28 of it are themselves, smaller ones are
// off by 2^-39 of it at most; the product (back_gemm.h).

#include <stdlib.h>
#include "back_gemm.h"

namespace gptq {

struct PackArgs {
    const void* dy; int64_t ldy, n, d_row;
    const int8_t* e;
    const int32_t* offsets; int E;
    uint16_t* A; int64_t lda; int32_t* shift;
};

template <gptq_dtype T>
__global__ __launch_bounds__(256) void back_pack_kernel(PackArgs a) {
    __shared__ int red[4];
    Segment s;
    if (!segment_of(a.offsets, a.E, a.n, 1, (int)blockIdx.x, s)) return;   // tiles of one row: only rows of experts
    const int64_t t = s.tok0;
    const int8_t* e = a.e + (int64_t)s.e * a.d_row;
    int m = -1000;
    for (int64_t r = threadIdx.x; r < a.d_row; r += 256) {
        const int v = exponent_of(load_as_f32<T>(a.dy, t * a.ldy + r)) + e[r];
        m = v > m ? v : m;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
        const int v = __shfl_xor(m, o);
        m = v > m ? v : m;
    }
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int w = 1; w < 4; ++w) m = red[w] > m ? red[w] : m;
    const int k = m < -900 ? 0 : 14 - m;                         // nothing but zeros
    if (threadIdx.x == 0) a.shift[t] = k;
    for (int64_t r = threadIdx.x; r < a.lda; r += 256) {
        const float v = r < a.d_row ? ldexpf(load_as_f32<T>(a.dy, t * a.ldy + r), e[r] + k) : 0.f;
        a.A[((r / BK) * a.n + t) * BK + r % BK] = f32_to_f16_bits(v);
    }
}

template <int CB, int PB, int MT, int WC, bool DIRECT>
__global__ __launch_bounds__(128 * WC, 2) void back_gemm_kernel(BackArgs a, int gm, int gn) {
    typedef BackGemm<CB, 1, PB, MT, 2, WC, DIRECT> G;
    __shared__ __align__(16) uint8_t lds[G::LDS_BYTES];
    int tm, tn;
    tile_of(gm, gn, tm, tn);
    Segment s;
    if (!segment_of(a.offsets, a.E, a.n, G::BM, tm, s)) return;
    const int64_t c0 = (int64_t)tn * G::BN;
    f32x4_t acc[G::NI][MT];
    G::run(acc, a, expert_of(a.L, a.d_row, s.e), a.T + s.e * a.quads * a.L.n_groups, s.tok0, s.end, c0, 0, a.d_row, lds);
    G::each(acc, s.tok0, s.end, c0, a.L.d_col, [&](int64_t c, int64_t t, f32x4_t v, int have) {
        const int k = -a.shift[t];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = ldexpf(v[i], k);
        const int64_t at = t * a.L.d_col + c;
        if (a.yt == GPTQ_F32) store_four<GPTQ_F32>(a.y, at, v, have);
        else if (a.yt == GPTQ_BF16) store_four<GPTQ_BF16>(a.y, at, v, have);
        else store_four<GPTQ_F16>(a.y, at, v, have);
    });
}

template <int CB, int PB, int MT, int WC>
static void launch_tiles(const BackArgs& a, hipStream_t s) {
    typedef BackGemm<CB, 1, PB, MT, 2, WC, true> G;
    const int gm = (int)most_tiles(a.offsets, a.E, a.n, G::BM), gn = (int)((a.L.d_col + G::BN - 1) / G::BN);
    if (direct_codes(a.L)) back_gemm_kernel<CB, PB, MT, WC, true><<<(unsigned)(gm * gn), G::THREADS, 0, s>>>(a, gm, gn);
    else back_gemm_kernel<CB, PB, MT, WC, false><<<(unsigned)(gm * gn), G::THREADS, 0, s>>>(a, gm, gn);
}

template <int CB, int PB>
static void launch_parts(const BackArgs& a, hipStream_t s) {
    const int64_t each = (a.n + a.E - 1) / a.E;
    const char* force = getenv("BACK_TILE");
    const int f = force ? atoi(force) : 0;
    if constexpr (PB == 1) if (f == 256 || (!f && each > 128)) return launch_tiles<CB, PB, 8, 4>(a, s);
    if (f == 128 || (!f && each > 64)) launch_tiles<CB, PB, 4, 4>(a, s);
    else if (f == 64 || (!f && each > 32)) launch_tiles<CB, PB, 4, 2>(a, s);
    else launch_tiles<CB, PB, 1, 2>(a, s);
}

template <int CB>
static void launch_gemm(const BackArgs& a, hipStream_t s) {
    if (a.yt == GPTQ_BF16) launch_parts<CB, 1>(a, s);
    else launch_parts<CB, 2>(a, s);
}

static int64_t padded(int64_t d_row) { return (d_row + 63) / 64 * 64; }

// A scale may belong to as few columns as 32: d_col / 32 groups at most.
size_t back_ws_bytes(int64_t n, int64_t E, int64_t d_row, int64_t d_col) {
    return up256((size_t)(n * padded(d_row)) * 2) + up256((size_t)n * 4) + up256((size_t)(E * d_row)) +
           quads_bytes(E, d_row, (d_col + 31) / 32);
}

gptq_status back_launch(const BackCall& c, hipStream_t s) {
    BackArgs a = {};
    a.L = c.L; a.d_row = c.d_row; a.n = c.n; a.offsets = c.offsets; a.E = c.E;
    const int64_t lda = padded(c.d_row);
    uint8_t* w = (uint8_t*)c.ws;
    uint16_t* A = (uint16_t*)w;
    w += up256((size_t)(c.n * lda) * 2);
    int32_t* shift = (int32_t*)w;
    w += up256((size_t)c.n * 4);
    int8_t* e = (int8_t*)w;
    w += up256((size_t)(c.E * c.d_row));
    a.A[0] = A; a.A[1] = nullptr; a.shift = shift;
    a.T = (Quad*)w; a.quads = quads_of(c.d_row);
    a.y = c.dx; a.yt = c.dxt;
    rows_launch(c.L, c.E, c.d_row, e, (Quad*)w, s);
    GPTQ_LAUNCH_CHECK();
    const PackArgs p = {c.dy, c.ldy, c.n, c.d_row, e, c.offsets, c.E, A, lda, shift};
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
