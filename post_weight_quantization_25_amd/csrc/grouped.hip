// Products grouped by expert (gptqt_linear_grouped): y[t] = What_e x[t] for the rows t of
// expert e, and the logits of the losses at a stored head (one expert).
//
// Many tokens per expert: forward_gemm.h, with the activations as fp16 rows and the scales' ratios
// laid out first.  Others, and layers that it leaves: stored_gemm.h; few tokens: stored_tile.h.
//
// Workgroups find their expert and rows from the offsets on the device (segment_of), so the
// call needs no count on the host: the grid holds the most tiles that n rows of E experts can
// have, and workgroups behind the last one end.

#include "forward_gemm.h"

namespace gptq {

// Few tokens: TW waves share a row's chunks, each with one chunk in registers.  Instructions bound
// it (about 170 a chunk of 16 rows x 128 columns, most of them decoding and arranging the
// operands): 131072 x 4096 int4 g128, one token: 81 us, 3.5 TB/s, with 4 or 8 waves and 1, 2 or 3
// chunks in flight alike.  Two chunks cost registers and a workgroup's time to begin: 131072 x 2048
// int3, 3 tokens: 44 us with one, 58 with two; 64 experts of 2816 x 2048, 8 rows: 13.6 / 16.
// 4 waves for narrow rows, which have few chunks for each: 131072 x 2048 int3: 37 us with 4, 44 with
// 8; 65536 x 512: 12.6 / 14; 4096 x 11008: 15.2 / 12.6; 131072 x 4096: 88 / 81; 64 experts of 2816 x
// 2048: 13.7 / 13.6 (whole calls in a chain from Python; the kernel alone 10.5, replayed 10.9).
constexpr bool few_waves(int64_t d_col) { return d_col <= 2048; }

template <int X, int CB, int RUN, int TW>
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
    stored_accumulate<X, CB, RUN, 1, 1, 1>(acc, L, row, xr, wave, TW);
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

// The outputs of the wave's 16 NT rows and of a tile's tokens that the wave has stored and that are
// not finite, by the whole wave.  Elements of x that are not finite decide a token's outputs alone;
// with none, as finite_sum.  2048 tokens x 32000 x 4096, one odd zero (690 us): 5.3 ms with an infinity
// in each token (134 with every output summed anew), 6.3 with nothing but NaNs (29).
template <int X, int CB, int NT>
GPTQ_DEV void sums_again(const GroupedArgs& a, const Segment& s, int tokens, int64_t tile_row) {
    int tid = threadIdx.x;
    // Formed here, not carried through the kernel; and no reading of y moves above its stores, which have
    // another type (in the hardware a lane's own accesses are in order).
    asm volatile("" : "+v"(tid) : : "memory");
    const int lane = tid & 63;
    const int64_t row0 = tile_row + 16 * NT * __builtin_amdgcn_readfirstlane(tid >> 6);
    const Stored L = expert_of(a.L, a.d_row, s.e);
#pragma unroll 1
    for (int m = 0; m < tokens && s.tok0 + m < s.end; ++m) {
        const int64_t t = s.tok0 + m;
        const uint16_t* x = a.x + t * a.ldx;
        bool lost[NT];                                           // the lane's own outputs: rows row0 + 16 nt + lane % 16
        uint64_t all = 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int64_t r = row0 + 16 * nt + (lane & 15), at = t * a.ldy + r;
            lost[nt] = false;
            if ((m & 15) >> 2 == lane >> 4 && r < a.d_row)
                lost[nt] = !(fabsf(a.yt == GPTQ_F32 ? load_as_f32<GPTQ_F32>(a.y, at) : a.yt == GPTQ_BF16 ? load_as_f32<GPTQ_BF16>(a.y, at)
                                                                                                         : load_as_f32<GPTQ_F16>(a.y, at)) < INFINITY);
            all |= __ballot(lost[nt]);
        }
        if (all == 0) continue;
        float sum[NT] = {};
        bool some = false;                                       // elements that are not finite
        for (int64_t c0 = 0; c0 < L.d_col; c0 += 512) {
            const int64_t c = c0 + 8 * lane;
            const uint32_t found = c < L.d_col ? not_finite8<X>(x + c, (int)(L.d_col - c < 8 ? L.d_col - c : 8)) : 0;
            uint64_t open = __ballot(found != 0);
            some = some || open != 0;
            for (; open != 0; open &= open - 1) {
                const int l = __builtin_ctzll(open);
#pragma unroll 1
                for (uint32_t left = __builtin_amdgcn_readlane(found, l); left != 0; left &= left - 1) {
                    const int64_t col = c0 + 8 * l + __builtin_ctz(left);
                    const float v = X == X_BF16 ? bf16_bits_to_f32(x[col]) : f16_bits_to_f32(x[col]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        if (lost[nt]) sum[nt] = fmaf(v, weight_at(L, CB, row0 + 16 * nt + (lane & 15), col), sum[nt]);
                }
                bool more = false;                               // sums that are not NaN yet
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) more = more || (lost[nt] && sum[nt] == sum[nt]);
                if (__ballot(more) == 0) { c0 = L.d_col; break; }
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            uint64_t todo = some ? 0 : __ballot(lost[nt]);
            while (todo) {                                       // wave-uniform
                const int l = __builtin_ctzll(todo);
                todo &= todo - 1;
                const float v = wave_sum<CB>(L, row0 + 16 * nt + (l & 15), [&](int64_t c, int n, float (&e)[8]) { load_x8<X>(x + c, n, e); });
                if (lane == l) sum[nt] = v;
            }
            if (lost[nt]) store_out(a.y, a.yt, t * a.ldy + row0 + 16 * nt + (lane & 15), sum[nt]);
        }
    }
}

template <int X, int CB, int PIECE, int BM>
__global__ __launch_bounds__(256, 2) void grouped_gemm_kernel(GroupedArgs a, int gm, int gn) {
    typedef StoredGemm<X, CB, PIECE, BM, 256> G;
    __shared__ __align__(16) uint8_t lds[G::LDS_BYTES];
    if (a.unless_zero && *a.unless_zero == 0) return;
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
    // Outputs that are not finite, once more by the definition (a zero's rest is infinity - infinity,
    // and sums of u - z may overflow where those of S (u - z) do not).  One instruction per output
    // tells whether there is any; behind the stores, whose registers the rest would take, they are
    // found in y.
    float none = 0.f;
#pragma unroll
    for (int mt = 0; mt < G::MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < G::NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) none = fmaf(acc[mt][nt][i], 0.f, none);
    if (__ballot(none != 0.f) != 0) sums_again<X, CB, G::NT>(a, s, BM, row0);   // wave-uniform; no barrier below
}

template <int X, int CB, int PIECE, int BM>
static void launch_gemm(const GroupedArgs& a, hipStream_t s) {
    const int gm = (int)most_tiles(a.offsets, a.E, a.n, BM), gn = (int)((a.d_row + GEMM_ROWS - 1) / GEMM_ROWS);
    grouped_gemm_kernel<X, CB, PIECE, BM><<<(unsigned)(gm * gn), 256, 0, s>>>(a, gm, gn);
}

// ---- many tokens
struct ForwardPackArgs {
    const uint16_t* x; int64_t ldx, n, d_col, columns;
    uint16_t* A; int32_t* shift; int32_t* odd; int natural;     // natural: columns in order (8-bit codes)
};

// A workgroup per token, 8 elements per thread and step; the second reading of a row comes from
// the cache.  Bound by memory: 8192 x 4096 bfloat16, 134 MB, 28 us (4.7 TB/s).
template <int X>
__global__ __launch_bounds__(256) void forward_pack_kernel(ForwardPackArgs a) {
    __shared__ int red[4];
    const int64_t t = blockIdx.x;
    const uint16_t* row = a.x + t * a.ldx;
    int k = 0;
    if constexpr (X == X_BF16) {
        int m = -1000;
        for (int64_t c = 8 * threadIdx.x; c < a.d_col; c += 2048) {
            float v[8];
            load_x8<X>(row + c, (int)(a.d_col - c < 8 ? a.d_col - c : 8), v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = exponent_of(v[i]);
                m = e > m ? e : m;
            }
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) {
            const int v = __shfl_xor(m, o);
            m = v > m ? v : m;
        }
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 4; ++w) m = red[w] > m ? red[w] : m;
        k = m < -900 ? 0 : 14 - m;                               // nothing but zeros
    }
    if (threadIdx.x == 0) {
        a.shift[t] = k;
        if (t == 0) *a.odd = 0;                                  // for forward_rows_kernel, which runs next
    }
    for (int64_t c = 8 * threadIdx.x; c < a.columns; c += 2048) {
        float v[8] = {};
        if (c < a.d_col) load_x8<X>(row + c, (int)(a.d_col - c < 8 ? a.d_col - c : 8), v);
        uint16_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = f32_to_f16_bits(X == X_BF16 ? __builtin_amdgcn_ldexpf(v[i], k) : v[i]);
        u32x4_t o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = a.natural ? h[2 * i] | ((uint32_t)h[2 * i + 1] << 16) : h[i] | ((uint32_t)h[i + 4] << 16);
        *reinterpret_cast<u32x4_t*>(a.A + ((c / BK) * a.n + t) * BK + c % BK) = o;
    }
}

// Ratios of a row's scales, its zeros as fp16 pairs, its last scale; the flag where one of them is
// not for this kernel.  64 rows of an expert per workgroup, threads along the rows: the layer has a
// row's groups together, the tables a group's rows (131072 rows of 32 groups: 16 us, through LDS).
__global__ __launch_bounds__(256) void forward_rows_kernel(Stored L, int64_t d_row, ForwardBuffers b) {
    __shared__ float S[64][33];
    __shared__ uint16_t Z[64][34];
    const int64_t row0 = (int64_t)blockIdx.x * 64, base = blockIdx.y * d_row, at = blockIdx.y * b.pitch * b.groups;
    bool odd = false;
    float before = 0.f;                                          // thread r's row: the scale of the group before
    for (int g0 = 0; g0 < b.groups; g0 += 32) {
        const int take = (int)(b.groups - g0 < 32 ? b.groups - g0 : 32);
        __syncthreads();
        for (int i = threadIdx.x; i < 64 * take; i += 256) {
            const int r = i / take, g = g0 + i % take;
            float s = 1.f, z = 0.f;
            if (row0 + r < d_row) {
                const int64_t p = (base + row0 + r) * L.n_groups + (g < L.n_groups ? g : L.n_groups - 1);   // behind the last: that one
                s = f16_bits_to_f32(L.scales[p]);
                z = f16_bits_to_f32(L.zeros[p]);
                odd = odd || !(s != 0.f && fabsf(s) < INFINITY && fabsf(z) <= 1024.f && rintf(z) == z);
            }
            S[r][g - g0] = s;
            Z[r][g - g0] = f32_to_f16_bits(1024.f + z);
        }
        __syncthreads();
        const int r = threadIdx.x & 63;
        for (int g = threadIdx.x >> 6; g < take; g += 4) {
            const float s = S[r][g], was = g > 0 ? S[r][g - 1] : g0 > 0 ? before : s;
            if (row0 + r < b.pitch) {
                b.rho[at + (int64_t)(g0 + g) * b.pitch + row0 + r] = was / s;
                b.zz[at + (int64_t)(g0 + g) * b.pitch + row0 + r] = Z[r][g] * 0x10001u;
                if (g0 + g == b.groups - 1) b.S_last[blockIdx.y * b.pitch + row0 + r] = s;
            }
        }
        before = S[r][take - 1];
    }
    if (__ballot(odd) != 0 && (threadIdx.x & 63) == 0) atomicOr(b.odd, 1);
}

template <int CB, int GPT>
__global__ __launch_bounds__(512, 2) void forward_gemm_kernel(ForwardArgs a, int gm, int gn) {
    typedef ForwardGemm<CB, GPT> G;
    __shared__ __align__(16) uint8_t lds[G::LDS_BYTES];
    if (*a.odd != 0) return;
    int tm, tn;
    tile_of(gm, gn, tm, tn);
    Segment s;
    if (!segment_of(a.offsets, a.E, a.n, G::BM, tm, s)) return;
    const int64_t row0 = (int64_t)tn * G::BN, table = s.e * a.expert_pitch;
    f32x4_t acc[G::NI][G::MT];
    G::run(acc, a, expert_of(a.L, a.d_row, s.e), a.rho + table, a.zz + table, s.tok0, s.end, row0, lds);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n16 = lane & 15, q = lane >> 4;
    float last[G::NI];
#pragma unroll
    for (int i = 0; i < G::NI; ++i) {
        const int64_t r = row0 + 64 * (wave & 3) + 16 * i + n16;
        last[i] = a.S_last[s.e * a.pitch + (r < a.d_row ? r : a.d_row - 1)];
    }
#pragma unroll
    for (int j = 0; j < G::MT; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int64_t t = s.tok0 + 128 * (wave >> 2) + 16 * j + 4 * q + v;
            if (t >= s.end) continue;
            const int k = -a.shift[t];
#pragma unroll
            for (int i = 0; i < G::NI; ++i) {
                const int64_t r = row0 + 64 * (wave & 3) + 16 * i + n16;
                if (r < a.d_row) store_out(a.y, a.yt, t * a.ldy + r, ldexpf(acc[i][j][v] * last[i], k));
            }
        }
}

template <int CB, int GPT>
static void launch_forward(const ForwardArgs& a, hipStream_t s) {
    typedef ForwardGemm<CB, GPT> G;
    const int gm = (int)most_tiles(a.offsets, a.E, a.n, G::BM), gn = (int)((a.d_row + G::BN - 1) / G::BN);
    forward_gemm_kernel<CB, GPT><<<(unsigned)(gm * gn), G::THREADS, 0, s>>>(a, gm, gn);
}

template <int CB>
static void launch_forward_groups(const ForwardArgs& a, int group, hipStream_t s) {
    const int per = forward_turn_groups(a.L.n_groups, group);
    if (per == 4) launch_forward<CB, 4>(a, s);
    else if (per == 2) launch_forward<CB, 2>(a, s);
    else if (per == 1) launch_forward<CB, 1>(a, s);
    else launch_forward<CB, 0>(a, s);
}

static size_t forward_layout(ForwardBuffers* b, uint8_t* w, int64_t n, int64_t E, int64_t d_row, int64_t d_col, int group) {
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t here = at; at += up256(bytes); return w ? w + here : nullptr; };
    const Stored L = stored_layer(nullptr, nullptr, nullptr, d_col, 8, group);
    ForwardBuffers h;
    h.pitch = (d_row + 3) / 4 * 4;
    h.groups = forward_groups(L.n_groups, group);
    h.odd = (int32_t*)take(4);
    h.A = (uint16_t*)take((size_t)(n * forward_columns(d_col)) * 2);
    h.shift = (int32_t*)take((size_t)n * 4);
    // a tile's loads of 256 rows may run over a table's end
    h.rho = (float*)take((size_t)(E * h.pitch * h.groups) * 4 + 1024);
    h.zz = (uint32_t*)take((size_t)(E * h.pitch * h.groups) * 4 + 1024);
    h.S_last = (float*)take((size_t)(E * h.pitch) * 4);
    if (b) *b = h;
    return at;
}

size_t grouped_ws_bytes(int64_t n, int64_t E, int64_t d_row, int64_t d_col, int group) {
    return many_rows(n, E) ? forward_layout(nullptr, nullptr, n, E, d_row, d_col, group) : 0;
}

bool grouped_large(const GroupedArgs& a, int64_t rows) { return direct_codes(a.L) && forward_pays(a.n, a.E, rows, a.L.d_col); }

gptq_status grouped_prepare(const GroupedArgs& a, gptq_dtype xt, int bits, int group, void* ws, hipStream_t s) {
    ForwardBuffers b;
    forward_layout(&b, (uint8_t*)ws, a.n, a.E, a.d_row, a.L.d_col, group);
    const ForwardPackArgs p = {a.x, a.ldx, a.n, a.L.d_col, forward_columns(a.L.d_col), b.A, b.shift, b.odd, bits == 8};
    if (xt == GPTQ_BF16) forward_pack_kernel<X_BF16><<<(unsigned)a.n, 256, 0, s>>>(p);
    else forward_pack_kernel<X_F16><<<(unsigned)a.n, 256, 0, s>>>(p);
    forward_rows_kernel<<<dim3((unsigned)((a.d_row + 63) / 64), (unsigned)a.E), 256, 0, s>>>(a.L, a.d_row, b);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

template <int X, int CB, int RUN, int PIECE>
static gptq_status launch(const GroupedArgs& a, hipStream_t s) {
    if (!a.unless_zero && small_tiles(a.n, a.E, a.d_row)) {
        const dim3 grid((unsigned)((a.d_row + 15) / 16), (unsigned)most_tiles(a.offsets, a.E, a.n, 16));
        if (few_waves(a.L.d_col)) grouped_tile_kernel<X, CB, RUN, 4><<<grid, 256, 0, s>>>(a);
        else grouped_tile_kernel<X, CB, RUN, 8><<<grid, 512, 0, s>>>(a);
    } else if (a.n / a.E <= 96) {
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

gptq_status grouped_launch(const GroupedArgs& given, gptq_dtype xt, int bits, int group, bool large, void* ws, int64_t all_rows,
                           int64_t row0, hipStream_t s) {
    GroupedArgs a = given;
    a.unless_zero = nullptr;
    if (large) {
        ForwardBuffers b;
        forward_layout(&b, (uint8_t*)ws, a.n, a.E, all_rows, a.L.d_col, group);
        ForwardArgs f;
        f.L = a.L; f.d_row = a.d_row; f.A = b.A; f.shift = b.shift;
        f.rho = b.rho + row0; f.zz = b.zz + row0; f.S_last = b.S_last + row0;
        f.pitch = b.pitch; f.expert_pitch = b.pitch * b.groups; f.odd = b.odd;
        f.n = a.n; f.offsets = a.offsets; f.E = a.E; f.y = a.y; f.yt = a.yt; f.ldy = a.ldy;
        if (bits == 3) launch_forward_groups<3>(f, group, s);
        else if (bits == 4) launch_forward_groups<4>(f, group, s);
        else launch_forward_groups<8>(f, group, s);
        GPTQ_LAUNCH_CHECK();
        a.unless_zero = b.odd;
    }
    return xt == GPTQ_BF16 ? launch_bits<X_BF16>(a, bits, group, s) : launch_bits<X_F16>(a, bits, group, s);
}

}  // namespace gptq
