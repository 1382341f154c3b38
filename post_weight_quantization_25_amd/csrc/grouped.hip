// Products grouped by expert (gptqt_linear_grouped): y[t] = What_e x[t] for the rows t of
// expert e, and the logits of the losses at a stored head (one expert).
//
// Workgroups find their expert and rows from the offsets on the device (segment_of), so the
// call needs no count on the host: the grid holds the most tiles that n rows of E experts can
// have, and workgroups behind the last one end.

#include "tuning.h"
#include "stored_gemm.h"

namespace gptq {

constexpr int TW = 8;         // waves per workgroup of the tile kernel

template <int X, int CB, int RUN>
__global__ __launch_bounds__(64 * TW, 4) void grouped_tile_kernel(GroupedArgs a) {
    __shared__ float red[TW][4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n16 = lane & 15;
    const int64_t row0 = (int64_t)blockIdx.x * 16;
    Segment s;
    if (!segment_of(a.offsets, a.E, a.n, 16, (int)blockIdx.y, s)) return;
    const Stored L = expert_of(a.L, a.d_row, s.e);
    const int64_t r = row0 + n16 < a.d_row ? row0 + n16 : a.d_row - 1;
    const int64_t row[1] = {r};
    const int64_t t = s.tok0 + n16;
    f32x4_t acc[1][1];
    acc[0][0] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const XScattered<1> xr = {{t < s.end ? reinterpret_cast<const uint8_t*>(a.x + t * a.ldx) : nullptr}};
    stored_accumulate<X, CB, RUN, 1, 1, 2>(acc, L, row, xr, wave, TW);
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][i][lane] = acc[0][0][i];
    __syncthreads();
    if (threadIdx.x >= 256) return;
    const int m = threadIdx.x >> 4, n = threadIdx.x & 15;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < TW; ++w) v += red[w][m & 3][n + 16 * (m >> 2)];
    const bool live = s.tok0 + m < s.end && row0 + n < a.d_row;
    v = finite_sum<CB>(v, live, L, [&](int i) { return row0 + (i & 15); },
                       [&](int i, int64_t c, int m8, float (&x)[8]) { load_x8<X>(a.x + (s.tok0 + (i >> 4)) * a.ldx + c, m8, x); });
    if (live) store_out(a.y, a.yt, (s.tok0 + m) * a.ldy + row0 + n, v);
}

template <int X, int CB, int PIECE, int BM>
__global__ __launch_bounds__(256, 2) void grouped_gemm_kernel(GroupedArgs a, int gm, int gn) {
    typedef StoredGemm<X, CB, PIECE, BM, 256> G;
    __shared__ __align__(16) uint8_t lds[G::LDS_BYTES];
    int tm, tn;
    tile_of(gm, gn, tm, tn);
    Segment s;
    if (!segment_of(a.offsets, a.E, a.n, BM, tm, s)) return;
    const int64_t row0 = (int64_t)tn * GEMM_ROWS;
    f32x4_t acc[G::MT][G::NT];
    G::run(acc, expert_of(a.L, a.d_row, s.e), a.d_row, reinterpret_cast<const uint8_t*>(a.x), 2 * a.ldx, s.end, s.tok0, row0, lds);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int mt = 0; mt < G::MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t t = s.tok0 + 16 * mt + 4 * (lane >> 4) + i;
            if (t >= s.end) continue;
#pragma unroll
            for (int nt = 0; nt < G::NT; ++nt) {
                const int64_t r = row0 + 32 * wave + 16 * nt + (lane & 15);
                if (r < a.d_row) store_out(a.y, a.yt, t * a.ldy + r, acc[mt][nt][i]);
            }
        }
}

template <int X, int CB, int PIECE, int BM>
static void launch_gemm(const GroupedArgs& a, hipStream_t s) {
    const int gm = (int)most_tiles(a.offsets, a.E, a.n, BM), gn = (int)((a.d_row + GEMM_ROWS - 1) / GEMM_ROWS);
    grouped_gemm_kernel<X, CB, PIECE, BM><<<(unsigned)(gm * gn), 256, 0, s>>>(a, gm, gn);
}

template <int X, int CB, int RUN, int PIECE>
static gptq_status launch(const GroupedArgs& a, hipStream_t s) {
    const int64_t each = a.n / a.E;
    if (each <= 16) {
        const dim3 grid((unsigned)((a.d_row + 15) / 16), (unsigned)most_tiles(a.offsets, a.E, a.n, 16));
        grouped_tile_kernel<X, CB, RUN><<<grid, 64 * TW, 0, s>>>(a);
    } else if (each <= 96) {
        launch_gemm<X, CB, PIECE, 64>(a, s);
    } else {
        launch_gemm<X, CB, PIECE, 128>(a, s);
    }
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

template <int X, int CB>
static gptq_status launch_runs(const GroupedArgs& a, int group, hipStream_t s) {
    return group == 32 ? launch<X, CB, 8, 32>(a, s) : group == 64 ? launch<X, CB, 16, 64>(a, s)
         : group == 128 ? launch<X, CB, 32, 128>(a, s) : launch<X, CB, 32, 0>(a, s);
}

template <int X>
static gptq_status launch_bits(const GroupedArgs& a, int bits, int group, hipStream_t s) {
    return bits == 3 ? launch_runs<X, 3>(a, group, s) : bits == 4 ? launch_runs<X, 4>(a, group, s) : launch_runs<X, 8>(a, group, s);
}

gptq_status grouped_launch(const GroupedArgs& a, gptq_dtype xt, int bits, int group, hipStream_t s) {
    return xt == GPTQ_BF16 ? launch_bits<X_BF16>(a, bits, group, s) : launch_bits<X_F16>(a, bits, group, s);
}

}  // namespace gptq
