// The product on stored codes with 8-bit rows (gptqs_linear_int8):
//   y[t][r] = xs[t] sum_g S[r][g] sum_{c in g} xq[t][c] (u[r][c] - z[r][g]),
// integer products on v_mfma_i32_16x16x64_i8 (exact), groups added in fp32.
//
// Small batches (int8_tile_kernel): bound by the codes' bytes and, at one token, by the
// latency of one round trip.  A workgroup of 8 waves owns 16 RB rows and 16 NTT tokens; its
// waves take the rows' 128-column chunks in turn and meet in LDS at the end.  One token,
// 4096 x 4096 int4 g128: 5.0 us; 48 tokens x 11008 x 4096 g64: 17 us (see stored_tile.h).
//
// Large ones (int8_gemm_kernel, stored_gemm.h): bound by the vector unit's issue (58% of the
// cycles, the matrix unit 23%), two instructions per four sums and 128 columns to scale them
// beside two products of the matrix unit, plus the decoding; with one scale per row (51% and
// 21%) decoding alone.  4096 tokens x 4096 x 4096 int4 g128: 114 us, 1.2 Pop/s,
// where the library's plain int8 product reaches 2.05.

#include "serving.h"
#include "stored_gemm.h"

namespace gptq {

constexpr int TW = 8;    // waves per workgroup

struct Int8Args {
    Stored L; int64_t d_row;
    const int8_t* x; int64_t ldx; int64_t n;
    const float* xs;
    void* y; gptq_dtype yt;
};

template <int CB, int RUN, int NTT, int RB>
__global__ __launch_bounds__(64 * TW, NTT * RB < 8 ? 4 : 2) void int8_tile_kernel(Int8Args a) {
    constexpr int DEEP = NTT >= 3 ? 1 : 2;
    constexpr int STAGE = 16 * SCK * xbytes<X_I8>();                   // one tile's chunk
    constexpr int RED = TW * NTT * RB * 1024, LDS = NTT > 1 && TW * STAGE > RED ? TW * STAGE : RED;
    __shared__ __align__(16) uint8_t stage[LDS];
    float (*red)[NTT * RB][4][64] = reinterpret_cast<float (*)[NTT * RB][4][64]>(stage);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n16 = lane & 15;
    const int64_t row0 = (int64_t)blockIdx.x * 16 * RB, tok0 = (int64_t)blockIdx.y * 16 * NTT;
    int64_t row[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const int64_t r = row0 + 16 * rb + n16;
        row[rb] = r < a.d_row ? r : a.d_row - 1;                 // rows past the end re-read the last
    }
    f32x4_t acc[NTT][RB];
#pragma unroll
    for (int tt = 0; tt < NTT; ++tt)
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) acc[tt][rb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // one tile of few tokens is read in place, its empty rows costing nothing; more tiles in
    // contiguous pieces
    if constexpr (NTT == 1) {
        const int64_t t = tok0 + n16;
        const XScattered<1> xr = {{t < a.n ? reinterpret_cast<const uint8_t*>(a.x) + tok0 * a.ldx + n16 * (int64_t)a.ldx : nullptr}};
        stored_accumulate<X_I8, CB, RUN, NTT, RB, DEEP>(acc, a.L, row, xr, wave, TW);
    } else {
        const XConsecutive xr = {reinterpret_cast<const uint8_t*>(a.x) + tok0 * a.ldx, a.ldx, (int)(a.n - tok0 < 16 * NTT ? a.n - tok0 : 16 * NTT), stage + STAGE * wave};
        stored_accumulate<X_I8, CB, RUN, NTT, RB, DEEP>(acc, a.L, row, xr, wave, TW);
        __syncthreads();                       // the stages give way to the sums
    }
#pragma unroll
    for (int tt = 0; tt < NTT; ++tt)
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int i = 0; i < 4; ++i) red[wave][tt * RB + rb][i][lane] = acc[tt][rb][i];
    __syncthreads();
    for (int o = threadIdx.x; o < NTT * RB * 256; o += 64 * TW) {
        const int tr = o >> 8, m = (o >> 4) & 15, n = o & 15, tt = tr / RB, rb = tr % RB;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < TW; ++w) v += red[w][tr][m & 3][n + 16 * (m >> 2)];
        const int64_t t = tok0 + 16 * tt + m, r = row0 + 16 * rb + n;
        if (t < a.n && r < a.d_row) store_out(a.y, a.yt, t * a.d_row + r, a.xs[t] * v);
    }
}

// Large batches: see stored_gemm.h.
template <int CB, int PIECE, int BM>
__global__ __launch_bounds__(256, 2) void int8_gemm_kernel(Int8Args a, int gm, int gn) {
    typedef StoredGemm<X_I8, CB, PIECE, BM, 256> G;
    __shared__ __align__(16) uint8_t lds[G::LDS_BYTES];
    int tm, tn;
    tile_of(gm, gn, tm, tn);
    const int64_t tok0 = (int64_t)tm * BM, row0 = (int64_t)tn * GEMM_ROWS;
    f32x4_t acc[G::MT][G::NT];
    G::run(acc, a.L, a.d_row, reinterpret_cast<const uint8_t*>(a.x), a.ldx, a.n, tok0, row0, lds);
    G::each_token(a.n, tok0, [&](int mt, int i, int64_t t) {
        const float xs = a.xs[t];
#pragma unroll
        for (int nt = 0; nt < G::NT; ++nt) acc[mt][nt][i] *= xs;
    });
    if (a.yt == GPTQ_F32) G::template write<GPTQ_F32>(acc, a.y, a.d_row, a.n, tok0, row0);
    else if (a.yt == GPTQ_BF16) G::template write<GPTQ_BF16>(acc, a.y, a.d_row, a.n, tok0, row0);
    else G::template write<GPTQ_F16>(acc, a.y, a.d_row, a.n, tok0, row0);
}

template <int CB, int PIECE, int BM>
static void launch_gemm(const Int8Args& a, hipStream_t s) {
    const int gm = (int)((a.n + BM - 1) / BM), gn = (int)((a.d_row + GEMM_ROWS - 1) / GEMM_ROWS);
    int8_gemm_kernel<CB, PIECE, BM><<<(unsigned)(gm * gn), 256, 0, s>>>(a, gm, gn);
}

template <int CB, int RUN, int NTT>
static void launch_tiles(const Int8Args& a, hipStream_t s) {
    constexpr int RB = RUN == 8 ? 1 : 2;
    const dim3 grid((unsigned)((a.d_row + 16 * RB - 1) / (16 * RB)), (unsigned)((a.n + 16 * NTT - 1) / (16 * NTT)));
    int8_tile_kernel<CB, RUN, NTT, RB><<<grid, 64 * TW, 0, s>>>(a);
}

template <int CB, int RUN, int PIECE>
static gptq_status launch(const Int8Args& a, hipStream_t s) {
    if (const int per = int8_kernel(a.n, a.d_row, a.L.d_col, a.ldx)) {
        if (per == 128) launch_gemm<CB, PIECE, 128>(a, s);
        else launch_gemm<CB, PIECE, 64>(a, s);
        GPTQ_LAUNCH_CHECK();
        return GPTQ_OK;
    }
    const unsigned g16 = (unsigned)((a.d_row + 15) / 16);
    if (a.n <= 16) int8_tile_kernel<CB, RUN, 1, 1><<<dim3(g16, 1), 64 * TW, 0, s>>>(a);
    else if (a.n <= 32) int8_tile_kernel<CB, RUN, 2, 1><<<dim3(g16, 1), 64 * TW, 0, s>>>(a);
    else if (a.n <= 48) launch_tiles<CB, RUN, 3>(a, s);
    else launch_tiles<CB, RUN, 4>(a, s);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

template <int CB>
static gptq_status launch_runs(const Int8Args& a, int group, hipStream_t s) {
    return group == 32 ? launch<CB, 8, 32>(a, s) : group == 64 ? launch<CB, 16, 64>(a, s)
         : group == 128 ? launch<CB, 32, 128>(a, s) : launch<CB, 32, 0>(a, s);
}

gptq_status linear_int8_launch(const uint8_t* codes, const uint16_t* scales, const uint16_t* zeros, int64_t d_row,
                               int64_t d_col, int bits, int group, const int8_t* x, int64_t ldx, const float* xs,
                               int64_t n, void* y, gptq_dtype yt, hipStream_t s) {
    Int8Args a;
    a.L = stored_layer(codes, scales, zeros, d_col, bits, group);
    a.d_row = d_row; a.x = x; a.ldx = ldx; a.n = n; a.xs = xs; a.y = y; a.yt = yt;
    return bits == 3 ? launch_runs<3>(a, group, s) : bits == 4 ? launch_runs<4>(a, group, s) : launch_runs<8>(a, group, s);
}

}  // namespace gptq
