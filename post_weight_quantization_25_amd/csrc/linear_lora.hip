// A shared projection on stored codes with a low-rank adapter per token beside it
// (gptqs_linear_lora):
//   y[t] = What x[t] + s_a B_a (A_a x[t]),  a = ids[t].
//
// Two launches.  lora_shrink_kernel forms v[t] = A_a x[t] on the matrix cores: a workgroup
// takes 16 tokens and a share of the columns, and for each distinct adapter among its
// tokens (few tokens: its share of them) multiplies all 16 by that adapter's rows and
// keeps the rows of the tokens that have it (a run of tokens with one adapter costs one
// product).  v of a token without an adapter is not written, and not used.  The shares' sums go to
// the workspace, fp32, and are added in a fixed order by the readers.  Then the
// projection's kernel adds s_a B_a v to its own sums before its one rounding, so the
// adapters cost no extra pass over y.  Selecting rows, rather than multiplying by zero,
// keeps an infinity or a NaN of one adapter away from the tokens of the others.
//
// One token, 4096 x 4096 int4 g128, rank 16: 3.3 + 7.0 us; 40 tokens with up to 32 adapters
// of rank 32: 6.3 + 19 us; 2048 tokens x 11008 x 4096, rank 16, runs of 450 tokens: 308 us
// together (10 the first), 605 Tflop/s of the 1286 that the library's bf16 product on plain
// weights reaches: there the decoding to bfloat16 (a conversion, a subtraction and half a
// packing per code) shares the vector unit, 44% busy, with the scaling.  From 64 to 256
// tokens the projection alone (gptq_quantized_linear) is faster on few rows: 256 tokens x
// 4096 x 4096, 32 us against 66, x 4096 x 11008, 62 against 141.  It multiplies 64 rows per
// workgroup, the tiles here 16, so the activations are read from L2 four times as often.

#include "serving.h"
#include "stored_gemm.h"

namespace gptq {

constexpr int TW = 8;         // waves per workgroup of the projection
constexpr int SW = 4;         // waves per workgroup of the shrink product
constexpr int SHARE = 512;    // columns of one share's step: 128 per wave
constexpr int RCH = 64;       // ranks held in LDS at a time by the projection's epilogue

struct LoraArgs {
    Stored L; int64_t d_row;
    const uint16_t* x; int64_t ldx; int64_t n;
    const uint16_t* A; const uint16_t* B; int n_adapters; int rank;   // rank 0: no adapters
    const int32_t* ids; const float* scaling;
    float* v; int splits; int64_t share;   // v: splits x n x rank; share: columns per split
    int slots;                             // workgroups among which a tile's adapters are dealt
    void* y; gptq_dtype yt;
};

// The adapter of token t: -1 past the last token or outside the table.
GPTQ_DEV int adapter_of(const LoraArgs& a, int64_t t) {
    const int id = t < a.n ? a.ids[t] : -1;
    return id >= 0 && id < a.n_adapters ? id : -1;
}

template <int X>
__global__ __launch_bounds__(64 * SW) void lora_shrink_kernel(LoraArgs a) {
    __shared__ float red[SW][4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n16 = lane & 15, q = lane >> 4;
    const int64_t tok0 = (int64_t)blockIdx.x * 16;
    const int64_t t = tok0 + n16 < a.n ? tok0 + n16 : a.n - 1;
    const int id = adapter_of(a, tok0 + n16);
    const uint8_t* xrow = reinterpret_cast<const uint8_t*>(a.x + t * a.ldx);
    const int64_t col_a = (int64_t)blockIdx.y * a.share;
    const int64_t col_b = col_a + a.share < a.L.d_col ? col_a + a.share : a.L.d_col;
    const int rt = blockIdx.z / a.slots, slot = blockIdx.z % a.slots;   // 16 ranks; a share of the tile's adapters
    const int k = 16 * rt + n16 < a.rank ? 16 * rt + n16 : a.rank - 1;
    f32x4_t out = {0.f, 0.f, 0.f, 0.f};
    uint32_t todo = (uint32_t)__ballot(id >= 0) & 0xFFFFu, done = 0;
    for (int j = 0; todo; ++j) {                                 // wave-uniform
        const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
        const uint32_t mine = (uint32_t)__ballot(id == ad) & 0xFFFFu;
        todo &= ~mine;
        if (j % a.slots != slot) continue;
        done |= mine;
        const uint8_t* arow = reinterpret_cast<const uint8_t*>(a.A + ((int64_t)ad * a.rank + k) * a.L.d_col);
        f32x4_t cs = {0.f, 0.f, 0.f, 0.f};
        for (int64_t c0 = col_a + 128 * wave; c0 < col_b; c0 += SHARE) {
            u32x4_t xf[4], af[4];
            const int64_t col = c0 + 32 * q;                     // the lane's 32 columns of 128
            if (c0 + 128 <= col_b) {
                const XRun<X, 32> xr = load_x<X, 32>(xrow + 2 * col), ar = load_x<X, 32>(arow + 2 * col);
                __builtin_memcpy(xf, xr.w, 64);
                __builtin_memcpy(af, ar.w, 64);
            } else {
                const int left = (int)(col_b - col < 32 ? col_b - col : 32);
                const XRun<X, 32> xr = load_x_tail<X, 32>(xrow + 2 * col, left), ar = load_x_tail<X, 32>(arow + 2 * col, left);
                __builtin_memcpy(xf, xr.w, 64);
                __builtin_memcpy(af, ar.w, 64);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) cs = mfma16<X>(xf[e], af[e], cs);
        }
        settle(cs);                                              // products end behind the loop's branch
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = (mine >> (4 * q + i)) & 1 ? cs[i] : out[i];
    }
    if (done == 0) return;                                       // the whole workgroup: every wave sees the same ids
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][i][lane] = out[i];
    __syncthreads();
    const int m = threadIdx.x >> 4, n = threadIdx.x & 15;        // token m, rank n of the tile
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < SW; ++w) v += red[w][m & 3][n + 16 * (m >> 2)];
    if (((done >> m) & 1) && 16 * rt + n < a.rank)
        a.v[((int64_t)blockIdx.y * a.n + tok0 + m) * a.rank + 16 * rt + n] = v;
}

template <int X>
GPTQ_DEV float elem16(uint16_t b) { return X == X_BF16 ? bf16_bits_to_f32(b) : f16_bits_to_f32(b); }

template <int X, int CB, int RUN, int NTT, int RB>
__global__ __launch_bounds__(64 * TW, NTT == 1 ? 4 : 2) void lora_tile_kernel(LoraArgs a) {
    constexpr int DEEP = NTT >= 3 ? 1 : 2;
    constexpr int PER = (NTT * RB * 256 + 64 * TW - 1) / (64 * TW);   // outputs per thread
    constexpr int STAGE = 16 * SCK * xbytes<X>();                   // one tile's chunk
    constexpr int RED = TW * NTT * RB * 1024, LDS = NTT > 1 && TW * STAGE > RED ? TW * STAGE : RED;
    __shared__ __align__(16) uint8_t stage[LDS];
    float (*red)[NTT * RB][4][64] = reinterpret_cast<float (*)[NTT * RB][4][64]>(stage);
    __shared__ float vs[16 * NTT][RCH + 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n16 = lane & 15;
    const int64_t row0 = (int64_t)blockIdx.x * 16 * RB, tok0 = (int64_t)blockIdx.y * 16 * NTT;
    int64_t row[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const int64_t r = row0 + 16 * rb + n16;
        row[rb] = r < a.d_row ? r : a.d_row - 1;
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
        const XScattered<1> xr = {{t < a.n ? reinterpret_cast<const uint8_t*>(a.x + tok0 * a.ldx) + n16 * 2 * a.ldx : nullptr}};
        stored_accumulate<X, CB, RUN, NTT, RB, DEEP>(acc, a.L, row, xr, wave, TW);
    } else {
        const XConsecutive xr = {reinterpret_cast<const uint8_t*>(a.x + tok0 * a.ldx), 2 * a.ldx, (int)(a.n - tok0 < 16 * NTT ? a.n - tok0 : 16 * NTT), stage + STAGE * wave};
        stored_accumulate<X, CB, RUN, NTT, RB, DEEP>(acc, a.L, row, xr, wave, TW);
        __syncthreads();                       // the stages give way to the sums
    }
#pragma unroll
    for (int tt = 0; tt < NTT; ++tt)
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int i = 0; i < 4; ++i) red[wave][tt * RB + rb][i][lane] = acc[tt][rb][i];

    // the thread's outputs: o = threadIdx.x + 64 TW k
    float delta[PER];
    int id[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int o = threadIdx.x + 64 * TW * k, tr = o >> 8;
        delta[k] = 0.f;
        id[k] = a.rank && tr < NTT * RB ? adapter_of(a, tok0 + 16 * (tr / RB) + ((o >> 4) & 15)) : -1;
    }
    for (int k0 = 0; k0 < a.rank; k0 += RCH) {
        const int kn = a.rank - k0 < RCH ? a.rank - k0 : RCH;
        __syncthreads();
        for (int e = threadIdx.x; e < 16 * NTT * kn; e += 64 * TW) {
            const int m = e / kn, k = e % kn;
            const int64_t t = tok0 + m;
            float v = 0.f;
            if (t < a.n) {
                for (int s = 0; s < a.splits; ++s) v += a.v[((int64_t)s * a.n + t) * a.rank + k0 + k];
                const int ad = adapter_of(a, t);
                if (a.scaling && ad >= 0) v *= a.scaling[ad];
            }
            vs[m][k] = v;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int o = threadIdx.x + 64 * TW * k, tr = o >> 8, m = 16 * (tr / RB) + ((o >> 4) & 15);
            const int64_t r = row0 + 16 * (tr % RB) + (o & 15);
            if (id[k] < 0 || r >= a.d_row) continue;
            const uint16_t* b = a.B + ((int64_t)id[k] * a.d_row + r) * a.rank + k0;
            int e = 0;
            for (; e + 8 <= kn; e += 8) {
                uint16_t w[8];
                __builtin_memcpy(w, b + e, 16);
#pragma unroll
                for (int f = 0; f < 8; ++f) delta[k] = fmaf(vs[m][e + f], elem16<X>(w[f]), delta[k]);
            }
            for (; e < kn; ++e) delta[k] = fmaf(vs[m][e], elem16<X>(b[e]), delta[k]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int o = threadIdx.x + 64 * TW * k, tr = o >> 8, m = (o >> 4) & 15, n = o & 15;
        if (tr >= NTT * RB) continue;                              // whole waves
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < TW; ++w) v += red[w][tr][m & 3][n + 16 * (m >> 2)];
        const int64_t t = tok0 + 16 * (tr / RB) + m, r = row0 + 16 * (tr % RB) + n;
        v = finite_sum<CB>(
            v, t < a.n && r < a.d_row, a.L,
            [&](int i) { return row0 + 16 * (((i + 64 * TW * k) >> 8) % RB) + (i & 15); },
            [&](int i, int64_t c, int m8, float (&x)[8]) {
                load_x8<X>(a.x + (tok0 + 16 * (((i + 64 * TW * k) >> 8) / RB) + ((i >> 4) & 15)) * a.ldx + c, m8, x);
            });
        if (id[k] >= 0) v += delta[k];
        if (t < a.n && r < a.d_row) store_out(a.y, a.yt, t * a.d_row + r, v);
    }
}

// Large batches (see stored_gemm.h).  The adapters' product is added to the finished sums on
// the matrix cores, 32 ranks at a time: s_a v as its three bfloat16 parts (bf16_parts) with
// B's rows, bfloat16 as they are, fp16 as two exact bfloat16 parts (fp16's 11 bits and its
// range fit; the smallest part by the smallest, below 2^-25 of a product, is left out), for
// each distinct adapter among the wave's tokens, into the rows of the tokens that have it.
// Sums that are not finite, where a part of 0 may have met an infinity, are taken again
// from the whole numbers.
template <int X, int CB, int PIECE, int BM>
__global__ __launch_bounds__(256, 2) void lora_gemm_kernel(LoraArgs a, int gm, int gn) {
    typedef StoredGemm<X, CB, PIECE, BM, 256> G;
    __shared__ __align__(16) uint8_t lds[G::LDS_BYTES];
    int tm, tn;
    tile_of(gm, gn, tm, tn);
    const int64_t tok0 = (int64_t)tm * BM, row0 = (int64_t)tn * GEMM_ROWS;
    f32x4_t acc[G::MT][G::NT];
    G::run(acc, a.L, a.d_row, reinterpret_cast<const uint8_t*>(a.x), 2 * a.ldx, a.n, tok0, row0, lds);

    if (a.rank) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n16 = lane & 15, q = lane >> 4;
        // the tile's scaled v for 32 ranks, by bfloat16 part: [part][token][rank], in the slabs' place
        uint16_t* vp = reinterpret_cast<uint16_t*>(lds);
        int* ids = reinterpret_cast<int*>(vp + 3 * BM * 32);
        __syncthreads();                                       // the last slab is read
        for (int m = threadIdx.x; m < BM; m += 256) ids[m] = adapter_of(a, tok0 + m);
        for (int k0 = 0; k0 < a.rank; k0 += 32) {
            __syncthreads();
            for (int e = threadIdx.x; e < BM * 32; e += 256) {
                const int m = e >> 5, k = k0 + (e & 31), ad = ids[m];
                float v = 0.f;
                if (ad >= 0 && k < a.rank) {
                    for (int p = 0; p < a.splits; ++p) v += a.v[((int64_t)p * a.n + tok0 + m) * a.rank + k];
                    if (a.scaling) v *= a.scaling[ad];
                }
                uint16_t part[3];
                bf16_parts(v, part);
#pragma unroll
                for (int j = 0; j < 3; ++j) vp[j * BM * 32 + e] = part[j];
            }
            __syncthreads();
#pragma unroll 1
            for (int mt = 0; mt < G::MT; ++mt) {
                const int id = ids[16 * mt + n16];
                u32x4_t av[3];
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    av[j] = *reinterpret_cast<const u32x4_t*>(vp + j * BM * 32 + (16 * mt + n16) * 32 + 8 * q);
                f32x4_t sum[G::NT];
#pragma unroll
                for (int nt = 0; nt < G::NT; ++nt) sum[nt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
                uint32_t todo = (uint32_t)__ballot(id >= 0) & 0xFFFFu;
                while (todo) {                                 // wave-uniform
                    const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
                    const uint32_t mine = (uint32_t)__ballot(id == ad) & 0xFFFFu;
                    todo &= ~mine;
                    const bool all = mine == 0xFFFFu;
#pragma unroll
                    for (int nt = 0; nt < G::NT; ++nt) {
                        const int64_t r = row0 + 32 * wave + 16 * nt + n16;
                        const uint16_t* b = a.B + ((int64_t)ad * a.d_row + (r < a.d_row ? r : a.d_row - 1)) * a.rank + k0 + 8 * q;
                        const int left = a.rank - k0 - 8 * q;
                        uint16_t w[8];
                        if (left >= 8) __builtin_memcpy(w, b, 16);
                        else
#pragma unroll
                            for (int e = 0; e < 8; ++e) w[e] = e < left ? b[e] : 0;
                        f32x4_t c = {0.f, 0.f, 0.f, 0.f};
                        if constexpr (X == X_BF16) {
                            u32x4_t bb;
                            __builtin_memcpy(&bb, w, 16);
#pragma unroll
                            for (int j = 2; j >= 0; --j) c = mfma16<X_BF16>(av[j], bb, c);
                        } else {
                            bf16x8_t bh, bl;
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float f = f16_bits_to_f32(w[e]);
                                bh[e] = (__bf16)f;
                                bl[e] = (__bf16)(f - (float)bh[e]);   // (an infinity's: NaN, see lost)
                            }
                            const u32x4_t b0 = __builtin_bit_cast(u32x4_t, bh), b1 = __builtin_bit_cast(u32x4_t, bl);
                            c = mfma16<X_BF16>(av[2], b0, c);
                            c = mfma16<X_BF16>(av[1], b1, c);
                            c = mfma16<X_BF16>(av[1], b0, c);
                            c = mfma16<X_BF16>(av[0], b1, c);
                            c = mfma16<X_BF16>(av[0], b0, c);
                        }
                        settle(c);
                        bool lost = false;
#pragma unroll
                        for (int i = 0; i < 4; ++i) lost = lost || !(fabsf(c[i]) < INFINITY);
                        if (__ballot(lost) != 0) {             // wave-uniform, rare
                            f32x4_t again = {0.f, 0.f, 0.f, 0.f};
                            const int kn = a.rank - k0 < 32 ? a.rank - k0 : 32;
#pragma unroll 1
                            for (int k = 0; k < kn; ++k) {
                                const float bk = elem16<X>(b[k - 8 * q]);
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const uint16_t* v = vp + (16 * mt + 4 * q + i) * 32 + k;
                                    const float rest = bf16_bits_to_f32(v[BM * 32]) + bf16_bits_to_f32(v[2 * BM * 32]);
                                    again[i] = fmaf(bf16_bits_to_f32(v[0]) + rest, bk, again[i]);
                                }
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) c[i] = fabsf(c[i]) < INFINITY ? c[i] : again[i];
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) sum[nt][i] = all || ((mine >> (4 * q + i)) & 1) ? c[i] : sum[nt][i];
                    }
                }
                // acc is indexed by a constant in each arm
#pragma unroll
                for (int m = 0; m < G::MT; ++m)
                    if (m == mt)
#pragma unroll
                        for (int nt = 0; nt < G::NT; ++nt) acc[m][nt] += sum[nt];
            }
        }
    }
    if (a.yt == GPTQ_F32) G::template write<GPTQ_F32>(acc, a.y, a.d_row, a.n, tok0, row0);
    else if (a.yt == GPTQ_BF16) G::template write<GPTQ_BF16>(acc, a.y, a.d_row, a.n, tok0, row0);
    else G::template write<GPTQ_F16>(acc, a.y, a.d_row, a.n, tok0, row0);
}

template <int X, int CB, int PIECE, int BM>
static void launch_gemm(const LoraArgs& a, hipStream_t s) {
    const int gm = (int)((a.n + BM - 1) / BM), gn = (int)((a.d_row + GEMM_ROWS - 1) / GEMM_ROWS);
    lora_gemm_kernel<X, CB, PIECE, BM><<<(unsigned)(gm * gn), 256, 0, s>>>(a, gm, gn);
}

template <int X, int CB, int RUN, int PIECE>
static gptq_status launch(const LoraArgs& a, hipStream_t s) {
    if (const int per = lora_kernel(a.n, a.d_row, a.L.d_col, 2 * a.ldx, PIECE)) {
        if (per == 128) launch_gemm<X, CB, PIECE, 128>(a, s);
        else launch_gemm<X, CB, PIECE, 64>(a, s);
        GPTQ_LAUNCH_CHECK();
        return GPTQ_OK;
    }
    const unsigned g16 = (unsigned)((a.d_row + 15) / 16);
    auto tiles = [&](int per) { return (unsigned)((a.n + per - 1) / per); };
    if (a.n <= 16) lora_tile_kernel<X, CB, RUN, 1, 1><<<dim3(g16, 1), 64 * TW, 0, s>>>(a);
    else if (a.n <= 32) lora_tile_kernel<X, CB, RUN, 2, 1><<<dim3(g16, 1), 64 * TW, 0, s>>>(a);
    else if (a.n <= 48) lora_tile_kernel<X, CB, RUN, 3, 1><<<dim3(g16, tiles(48)), 64 * TW, 0, s>>>(a);
    else lora_tile_kernel<X, CB, RUN, 4, 1><<<dim3(g16, tiles(64)), 64 * TW, 0, s>>>(a);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

template <int X, int CB>
static gptq_status launch_runs(const LoraArgs& a, int group, hipStream_t s) {
    return group == 32 ? launch<X, CB, 8, 32>(a, s) : group == 64 ? launch<X, CB, 16, 64>(a, s)
         : group == 128 ? launch<X, CB, 32, 128>(a, s) : launch<X, CB, 32, 0>(a, s);
}

template <int X>
static gptq_status launch_bits(const LoraArgs& a, int bits, int group, hipStream_t s) {
    if (a.rank) {
        const dim3 grid((unsigned)((a.n + 15) / 16), (unsigned)a.splits, (unsigned)((a.rank + 15) / 16 * a.slots));
        lora_shrink_kernel<X><<<grid, 64 * SW, 0, s>>>(a);
        GPTQ_LAUNCH_CHECK();
    }
    return bits == 3 ? launch_runs<X, 3>(a, group, s) : bits == 4 ? launch_runs<X, 4>(a, group, s) : launch_runs<X, 8>(a, group, s);
}

// Shares of the columns: enough workgroups to fill the device, none below 512 columns.
static int64_t most_splits(int64_t d_col) {
    const int64_t most = (d_col + SHARE - 1) / SHARE;
    return most < 64 ? most : 64;
}
static int lora_splits(int64_t n, int64_t d_col, int rank) {
    const int64_t tiles = (n + 15) / 16 * ((rank + 15) / 16), most = most_splits(d_col);
    const int64_t want = (512 + tiles - 1) / tiles;
    return (int)(want < most ? want : most);
}

// n lora_splits(n) rows fall where a split less is taken, and a workspace made for the
// largest batch has to do for every smaller one: so the size is of a bound that only grows
// with n.  With R = ceil(rank / 16) there are at least n R / 16 tiles, so splits <= 511 / (n R
// / 16) + 1 and n splits <= 8176 / R + n.
size_t lora_ws_bytes(int64_t n, int64_t d_col, int rank) {
    const int64_t all = n * most_splits(d_col), some = 8176 / ((rank + 15) / 16) + n;
    return (size_t)(all < some ? all : some) * (size_t)rank * sizeof(float);
}

gptq_status linear_lora_launch(const uint8_t* codes, const uint16_t* scales, const uint16_t* zeros, int64_t d_row,
                               int64_t d_col, int bits, int group, const void* x, gptq_dtype xt, int64_t n, int64_t ldx,
                               const void* A, const void* B, int n_adapters, int rank, const int32_t* ids,
                               const float* scaling, void* y, gptq_dtype yt, void* ws, hipStream_t s) {
    LoraArgs a;
    a.L = stored_layer(codes, scales, zeros, d_col, bits, group);
    a.d_row = d_row; a.x = (const uint16_t*)x; a.ldx = ldx; a.n = n;
    a.A = (const uint16_t*)A; a.B = (const uint16_t*)B; a.n_adapters = n_adapters;
    a.rank = n_adapters > 0 ? rank : 0;
    a.ids = ids; a.scaling = scaling; a.v = (float*)ws;
    a.splits = a.rank ? lora_splits(n, d_col, rank) : 0;
    a.share = a.rank ? ((d_col + SHARE - 1) / SHARE + a.splits - 1) / a.splits * SHARE : 0;
    // few tokens: each adapter of a tile in a workgroup of its own; many: one after another
    a.slots = n <= 64 ? (n < 16 ? (int)n : 16) : 1;
    a.y = y; a.yt = yt;
    return xt == GPTQ_BF16 ? launch_bits<X_BF16>(a, bits, group, s) : launch_bits<X_F16>(a, bits, group, s);
}

}  // namespace gptq
