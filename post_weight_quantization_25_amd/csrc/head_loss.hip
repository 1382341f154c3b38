// Cross entropy and distillation at a stored head (gptqt_cross_entropy, gptqt_distill), in
// pieces of the vocabulary:
//   z = What x[t] / T;  loss = w T^2 sum_j p_j (log p_j - (z_j - lse z));
//   dx[t] = w T (sum_v softmax(z)_v What_v - sum_j p_j What_j),
// j over the token's entries (cross entropy: one, p = 1, T = 1).
//
// The entries' own words are kept apart from the others: with p_j near softmax(z)_j the two
// sums above nearly cancel, so a word v that is an entry takes the weight softmax(z)_v - p_j
// in fp32 (head_final_kernel) and only the others enter the large product.
//
// The vocabulary is split into spans; a round takes R spans, each with sums of its own:
//   logits  z of the round's words, fp32 (grouped.hip)
//   stats   per token and span: the entries' z are picked out, the maximum m and the sum of
//           exp(z - m) over the other words added to what the span's slot has, and exp(z - m)
//           written in fp16 (times 2^14 and the weight row's power of two): in one part, 2^-11 of
//           it, for bfloat16 dx, whose own rounding is 2^-8 (two would be three products in place of
//           one, the larger half of the call), in two otherwise
//   sums    O = O exp(m_old - m) + exp(z - m) What, fp32 (back_gemm.h)
// so the logits and the softmax are formed once, and nothing of the vocabulary's length is
// kept beyond a round.  Then head_final_kernel joins the slots.

#include "back_gemm.h"

namespace gptq {

struct HeadBuffers {
    float* z;                                                   // nc x R span
    uint16_t* A[2];                                             // exp(z - m) in fp16: [slab of 32 words][token][32]
    float* O;                                                   // R x nc x d
    float* m; float* s; float* f;                               // R x nc
    float* picked;                                              // nc x k
    void* forward;                                              // of grouped_prepare
    int8_t* e; Quad* T;                                         // vocab; a group's quads_of(vocab)
    int32_t* emax;                                              // of blocks of rows
};
constexpr int EB = 1024;                                        // rows per block of emax

// words: nc R span, rows: nc R, or bounds of them.
static size_t layout(HeadBuffers* b, uint8_t* w, int64_t nc, int64_t words, int64_t rows, int64_t d, int64_t vocab, int group, int k, int parts) {
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t here = at; at += up256(bytes); return w ? w + here : nullptr; };
    HeadBuffers h = {};
    h.z = (float*)take((size_t)words * 4);
    h.m = (float*)take((size_t)rows * 4); h.s = (float*)take((size_t)rows * 4); h.f = (float*)take((size_t)rows * 4);
    h.picked = (float*)take((size_t)(nc * k) * 4);
    h.forward = take(grouped_ws_bytes(nc, 1, vocab, d, group));
    if (parts) {
        h.A[0] = (uint16_t*)take((size_t)words * 2);
        h.A[1] = (uint16_t*)take(parts == 2 ? (size_t)words * 2 : 0);
        h.O = (float*)take((size_t)(rows * d) * 4);
        h.e = (int8_t*)take((size_t)vocab);
        h.T = (Quad*)take(quads_bytes(1, vocab, group ? d / group : 1));
        h.emax = (int32_t*)take((size_t)((vocab + EB - 1) / EB) * 4);
    }
    if (b) *b = h;
    return at;
}

size_t head_ws_bytes(int64_t n, int64_t d, int64_t vocab, int group, int k, bool grad) {
    const HeadMost most = head_most(n, d, vocab, grad);
    return layout(nullptr, nullptr, n < CHUNK ? n : CHUNK, most.words, most.rows, d, vocab, group, k, grad ? 2 : 0);
}

__global__ __launch_bounds__(256) void head_emax_kernel(const int8_t* e, int64_t vocab, int32_t* emax) {
    __shared__ int red[4];
    int m = -1000;
    for (int i = threadIdx.x; i < EB; i += 256) {
        const int64_t r = (int64_t)blockIdx.x * EB + i;
        if (r < vocab) m = e[r] > m ? e[r] : m;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
        const int v = __shfl_xor(m, o);
        m = v > m ? v : m;
    }
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 4; ++w) m = red[w] > m ? red[w] : m;
        emax[blockIdx.x] = m;
    }
}

// Over the workgroup of 256, in a fixed order; every thread gets it.
template <typename V, typename F>
GPTQ_DEV V over_block(V v, F&& f, V* red) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v = f(v, __shfl_xor(v, o));
    __syncthreads();                                             // the last use of red is over
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return f(f(red[0], red[1]), f(red[2], red[3]));
}

GPTQ_DEV int emax_of(const int32_t* emax, int blocks, int* red) {
    int m = -1000;
    for (int i = threadIdx.x; i < blocks; i += 256) m = emax[i] > m ? emax[i] : m;
    return over_block(m, [](int a, int b) { return a > b ? a : b; }, red);
}

struct HeadArgs {
    int64_t n, tok0, vocab, d;                                  // n tokens from tok0 on
    int k; const int32_t* ids;                                  // all tokens'
    const void* top; gptq_dtype topt;
    float T;
    const float* weights;
    HeadBuffers b;
    int R, round, slots; int64_t span;                          // slots: spans of this round; of all, in head_final_kernel
    int blocks;                                                 // of emax
    int64_t cols;                                               // columns of a workgroup of head_final_kernel
    Stored L;
    float* loss; void* dx; gptq_dtype dxt;                      // all tokens'
};

GPTQ_DEV bool entry_there(const HeadArgs& a, int64_t t, int j, int& id) {
    id = a.ids[(a.tok0 + t) * a.k + j];
    return id >= 0 && id < a.vocab;
}
GPTQ_DEV float weight_of(const HeadArgs& a, int64_t t) { return a.weights ? a.weights[a.tok0 + t] : 1.f; }

// e^d of d <= 0, to 2^-22 of it (0 below 2^-126, for d of -infinity too; NaN of a NaN): 2^t with t
// the rounded d log2(e), times 1 + ln(2) times what the rounding and the constant left out, which
// are no numbers where t overflows.
GPTQ_DEV float exp_of(float d) {
    const float t = d * 1.44269504f;
    const float rest = fmaf(d, 1.92596303e-8f, fmaf(d, 1.44269504f, -t));
    const float p = __builtin_amdgcn_exp2f(t);
    return d < -128.f ? 0.f : fmaf(p, rest * 0.693147181f, p);
}

// A workgroup per token and span, which it holds in registers: the logits are read once.  4096
// tokens x 8192 words, one part: 47 us, 201 MB at 4.3 TB/s (57 with expf and a load for each word's
// exponent); the vector unit and three joins over the workgroup keep it from more.
template <int PA>                                               // fp16 parts of exp(z - m); 0: no gradient
__global__ __launch_bounds__(256) void head_stats_kernel(HeadArgs a) {
    __shared__ uint32_t flag[SPAN / 32];
    __shared__ float red[4];
    __shared__ int redi[4];
    const int tid = threadIdx.x, slot = blockIdx.y;
    const int64_t t = blockIdx.x;
    const int64_t v0 = ((int64_t)a.round * a.R + slot) * a.span;
    const int words = (int)(a.vocab - v0 < a.span ? a.vocab - v0 : a.span);
    const int64_t ldz = a.R * a.span;                           // (of the round's words, as in head_launch)
    const float* z = a.b.z + t * ldz + slot * a.span;
    const float invT = 1.f / a.T;
    flag[tid] = 0;
    __syncthreads();
    int live = 0;
    for (int j = tid; j < a.k; j += 256) {
        int id;
        if (!entry_there(a, t, j, id)) continue;
        live = 1;
        const int64_t w = id - v0;
        if (w < 0 || w >= words) continue;
        atomicOr(&flag[w >> 5], 1u << (w & 31));
        a.b.picked[t * a.k + j] = z[w] * invT;
    }
    live = over_block(live, [](int x, int y) { return x | y; }, redi);
    if (weight_of(a, t) == 0.f) live = 0;
    // thread tid's words: 4 tid .. 4 tid + 3 of every 1024
    constexpr int U = SPAN / 1024;
    float v[U][4];
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (1024 * u >= a.span) break;                           // uniform
        const int w = 1024 * u + 4 * tid;
        f32x4_t q = {0.f, 0.f, 0.f, 0.f};
        if (w < words) q = *reinterpret_cast<const f32x4_t*>(z + w);   // the span is whole fours
        const uint32_t skip = flag[w >> 5] >> (w & 31);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = live && w + i < words && !((skip >> i) & 1);
            v[u][i] = in ? q[i] * invT : -INFINITY;
            m = v[u][i] > m ? v[u][i] : m;                       // (a NaN is met again in the sum)
        }
    }
    m = over_block(m, [](float x, float y) { return x > y ? x : y; }, red);
    const int64_t at = (int64_t)slot * a.n + t;
    const float m_old = a.round ? a.b.m[at] : -INFINITY, s_old = a.round ? a.b.s[at] : 0.f;
    m = m_old > m ? m_old : m;
    const float fall = m_old == -INFINITY ? 0.f : expf(m_old - m);
    const float top = m == -INFINITY ? 0.f : m;                  // (no word: every v is -infinity)
    const int em = PA ? emax_of(a.b.emax, a.blocks, redi) : 0;
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (1024 * u >= a.span) break;                           // uniform
        const int w = 1024 * u + 4 * tid;
        uint16_t hi[4], lo[4];
        uint32_t e4 = 0;                                         // (behind the vocabulary: p is 0)
        if (PA != 0 && w < words) e4 = *reinterpret_cast<const uint32_t*>(a.b.e + v0 + w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float p = exp_of(v[u][i] - top);
            s += p;
            if constexpr (PA != 0) f16_parts(__builtin_amdgcn_ldexpf(p, 14 + (int8_t)(e4 >> (8 * i)) - em), hi[i], lo[i]);
        }
        if constexpr (PA != 0) {
            if (w < a.span) {
                const int64_t to = ((slot * a.span + w) / BK * a.n + t) * BK + w % BK;
                uint2 o;
                o.x = hi[0] | ((uint32_t)hi[1] << 16); o.y = hi[2] | ((uint32_t)hi[3] << 16);
                *reinterpret_cast<uint2*>(a.b.A[0] + to) = o;
                if constexpr (PA == 2) {
                    o.x = lo[0] | ((uint32_t)lo[1] << 16); o.y = lo[2] | ((uint32_t)lo[3] << 16);
                    *reinterpret_cast<uint2*>(a.b.A[1] + to) = o;
                }
            }
        }
    }
    s = over_block(s, [](float x, float y) { return x + y; }, red);
    if (tid == 0) {
        a.b.m[at] = m;
        a.b.s[at] = s_old == 0.f ? s : fmaf(s_old, fall, s);
        a.b.f[at] = fall;
    }
}

// A span's O = O f + exp(z - m) What.  back_gemm.h says what bounds it; with two parts in both
// operands three products are formed (lo x lo is below the rounding): 301 tokens x 50021 x 2048 int4
// g64 227 us, 810 Tflop/s.
template <int CB, int P, int MT, int WC, bool DIRECT>
__global__ __launch_bounds__(128 * WC, P == 1 || MT == 1 || WC == 4 ? 2 : 1) void head_sums_kernel(BackArgs a, int gm, int gn, int64_t vocab, int64_t span, int v_first) {
    typedef BackGemm<CB, P, P, MT, 2, WC, DIRECT> G;
    __shared__ __align__(16) uint8_t lds[G::LDS_BYTES];
    int tm, tn;
    tile_of(gm, gn, tm, tn);
    const int slot = blockIdx.y;
    const int64_t tok0 = (int64_t)tm * G::BM, c0 = (int64_t)tn * G::BN;
    const int64_t k0 = v_first + slot * span, k1 = k0 + span < vocab ? k0 + span : vocab;
    f32x4_t acc[G::NI][MT];
    G::run(acc, a, a.L, a.T, tok0, a.n, c0, k0, k1, lds);
    float* O = a.sums + (int64_t)slot * a.n * a.L.d_col;
    const float* f = a.f + (int64_t)slot * a.n;
    G::each(acc, tok0, a.n, c0, a.L.d_col, [&](int64_t c, int64_t t, f32x4_t v, int have) {
        float* o = O + t * a.L.d_col + c;
        const float g = f[t];
        if (!a.first && g != 0.f) {
            if (have == 4) {
                f32x4_t was;
                __builtin_memcpy(&was, o, 16);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = fmaf(was[i], g, v[i]);
            } else {
                for (int i = 0; i < have; ++i) v[i] = fmaf(o[i], g, v[i]);
            }
        }
        store_four<GPTQ_F32>(o, 0, v, have);
    });
}

GPTQ_DEV float top_of(const HeadArgs& a, int64_t t, int j) {
    const int64_t i = (a.tok0 + t) * a.k + j;
    return a.topt == GPTQ_F32 ? load_as_f32<GPTQ_F32>(a.top, i) : a.topt == GPTQ_BF16 ? load_as_f32<GPTQ_BF16>(a.top, i)
                                                                                        : load_as_f32<GPTQ_F16>(a.top, i);
}

// The loss and the gradient of one token; where there are few tokens, of a.cols of its columns, the
// scalars by every workgroup anew.  Scalars in 64 bits: they cost nothing here, and
// p_j - softmax_j and the loss of a token that the model is sure of are small differences.
// Bound by its round trips: one after another the entries, the slots, the sums and the entries'
// rows.  4096 tokens x 4096, one entry, one slot: 51 us (100 MB); 2048 tokens, 64 entries: 128 us; 33 tokens x
// 1024, 8 entries, 32 slots: 12 us.
template <int CB>
__global__ __launch_bounds__(256) void head_final_kernel(HeadArgs a) {
    __shared__ double redd[4];
    __shared__ float red[4];
    __shared__ int redi[4];
    __shared__ int id_of[TUNE_MAX_TOP];
    __shared__ float coef[TUNE_MAX_TOP];
    __shared__ float slot_of[MOST_SPANS];
    __shared__ float joint[256][8];
    const int tid = threadIdx.x;
    const int64_t t = blockIdx.x, tt = a.tok0 + t;
    const int64_t col0 = blockIdx.y * a.cols, col1 = col0 + a.cols < a.d ? col0 + a.cols : a.d;
    const bool first_part = tid == 0 && blockIdx.y == 0;
    const float w = weight_of(a, t);
    const auto larger = [](float x, float y) { return x > y ? x : y; };
    const auto sum = [](double x, double y) { return x + y; };
    int live = 0;
    float tm = -INFINITY, zm = -INFINITY;                        // largest teacher's and model's among the entries
    for (int j = tid; j < a.k; j += 256) {
        int id;
        const bool in = entry_there(a, t, j, id);
        id_of[j] = in ? id : -1;
        if (!in) continue;
        live |= 1;
        if (a.top) {
            const float v = top_of(a, t, j);
            if (v != v) live |= 2;                               // a NaN masks nothing
            tm = larger(v / a.T, tm);
        }
        zm = larger(a.b.picked[t * a.k + j], zm);
    }
    live = over_block(live, [](int x, int y) { return x | y; }, redi);
    tm = over_block(tm, larger, red);
    if (!live || w == 0.f || (a.top && tm == -INFINITY && !(live & 2))) {   // no entry, or none with a weight
        if (first_part) a.loss[tt] = 0.f;
        if (a.dx)
            for (int64_t c = col0 + tid; c < col1; c += 256) store_out(a.dx, a.dxt, tt * a.d + c, 0.f);
        return;
    }
    for (int i = tid; i < a.slots; i += 256) zm = larger(a.b.m[(int64_t)i * a.n + t], zm);
    zm = over_block(zm, larger, red);
    double pt = 0., zt = 0.;                                     // sum of exp over the teacher's entries; the model's words
    for (int j = tid; j < a.k; j += 256) {
        if (id_of[j] < 0) continue;
        pt += a.top ? exp((double)(top_of(a, t, j) / a.T) - tm) : 1.;
        bool first = true;
        for (int i = 0; i < j && first; ++i) first = id_of[i] != id_of[j];
        coef[j] = first ? 1.f : 0.f;
        if (first) zt += exp((double)a.b.picked[t * a.k + j] - zm);
    }
    for (int i = tid; i < a.slots; i += 256) {
        const float m = a.b.m[(int64_t)i * a.n + t], s = a.b.s[(int64_t)i * a.n + t];
        if (s != 0.f) zt += s * exp((double)m - zm);
    }
    pt = over_block(pt, sum, redd);
    zt = over_block(zt, sum, redd);
    const double lpt = log(pt), lzt = log(zt);                   // lse z = zm + lzt
    double l = 0.;
    for (int j = tid; j < a.k; j += 256) {
        if (id_of[j] < 0) continue;
        const double lp = a.top ? (double)(top_of(a, t, j) / a.T) - tm - lpt : 0., lq = (double)a.b.picked[t * a.k + j] - zm - lzt;
        const double p = exp(lp);
        if (p != 0.) l += p * (lp - lq);
        coef[j] = (float)((coef[j] != 0.f ? exp(lq) : 0.) - p);
    }
    l = over_block(l, sum, redd);
    const float gain = w * a.T;
    if (first_part) a.loss[tt] = (float)((double)w * a.T * a.T * l);
    if (!a.dx) return;
    const int em = emax_of(a.b.emax, a.blocks, redi);
    for (int i = tid; i < a.R; i += 256) {                       // the slots' weights
        const float m = a.b.m[(int64_t)i * a.n + t], s = a.b.s[(int64_t)i * a.n + t];
        slot_of[i] = s == 0.f ? 0.f : ldexpf((float)exp((double)m - zm - lzt), em - 14);
    }
    __syncthreads();
    // 8 columns per thread; with fewer than 2048 of them several threads share a column's slots and
    // entries.
    int share = 1;
    while (share < 8 && a.cols * share <= 1024) share *= 2;
    const int per = 256 / share, col = tid % per, part = tid / per;
    for (int64_t c0 = col0; c0 < col1; c0 += 8 * per) {
        const int64_t c = c0 + 8 * col;
        const int have = (int)(col1 - c < 8 ? col1 - c : 8);
        float g[8] = {};
        if (have > 0) {
#pragma unroll 2
            for (int i = part; i < a.R; i += share) {
                const float q = slot_of[i];
                const float* o = a.b.O + ((int64_t)i * a.n + t) * a.d + c;
                float v[8];
                if (have == 8) __builtin_memcpy(v, o, 32);
                else
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = e < have ? o[e] : 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) g[e] = q == 0.f ? g[e] : fmaf(q, v[e], g[e]);
            }
            // entries four at a time, so that their loads are in flight together
            for (int j0 = part; j0 < a.k; j0 += 4 * share) {
                Raw<CB, 8> u[4];
                uint16_t S[4], zero[4];
                float k[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int j = j0 + x * share;
                    const bool in = j < a.k && id_of[j] >= 0;
                    const int64_t r = in ? id_of[j] : 0;
                    k[x] = in ? coef[j] : 0.f;
                    const uint8_t* src = a.L.codes + r * a.L.code_ld + c / 8 * CB;
                    if (have == 8) u[x] = load_raw<CB, 8>(src);
                    else u[x] = load_raw_tail<CB, 8>(src, have);
                    const int64_t i = r * a.L.n_groups + (a.L.n_groups == 1 ? 0 : c >> a.L.gshift);
                    S[x] = a.L.scales[i];
                    zero[x] = a.L.zeros[i];
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float s = f16_bits_to_f32(S[x]), z = f16_bits_to_f32(zero[x]);
                    if (k[x] == 0.f) continue;                   // an infinity in a word without a weight does not count
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        g[e] = fmaf(k[x], s * ((float)((code_bytes4<CB, 8>(u[x], e >> 2) >> (8 * (e & 3))) & 0xFFu) - z), g[e]);
                }
            }
        }
        if (share > 1) {                                         // uniform; one turn
            if (part > 0)
#pragma unroll
                for (int e = 0; e < 8; ++e) joint[(part - 1) * per + col][e] = g[e];
            __syncthreads();
            if (part == 0)
                for (int p = 1; p < share; ++p)
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[e] += joint[(p - 1) * per + col][e];
        }
        if (part == 0 && have > 0)
            for (int e = 0; e < have; ++e) store_out(a.dx, a.dxt, tt * a.d + c + e, gain * g[e]);
    }
}

template <int CB, int P, int MT, int WC>
static void launch_tiles(const BackArgs& b, int slots, int64_t vocab, int64_t span, int first_word, hipStream_t s) {
    typedef BackGemm<CB, P, P, MT, 2, WC, true> G;
    const int gm = (int)((b.n + G::BM - 1) / G::BM), gn = (int)((b.L.d_col + G::BN - 1) / G::BN);
    const dim3 grid((unsigned)(gm * gn), (unsigned)slots);
    if (direct_codes(b.L)) head_sums_kernel<CB, P, MT, WC, true><<<grid, G::THREADS, 0, s>>>(b, gm, gn, vocab, span, first_word);
    else head_sums_kernel<CB, P, MT, WC, false><<<grid, G::THREADS, 0, s>>>(b, gm, gn, vocab, span, first_word);
}

template <int CB, int P>
static void launch_parts(const BackArgs& b, int slots, int64_t vocab, int64_t span, int first_word, hipStream_t s) {
    const int bm = head_tile(b.n, P, CB).bm;
    if constexpr (P == 1) if (bm == 256) return launch_tiles<CB, P, 8, 4>(b, slots, vocab, span, first_word, s);
    if constexpr (P == 2 && CB != 8) if (bm == 128) return launch_tiles<CB, P, 4, 4>(b, slots, vocab, span, first_word, s);
    if (bm == 128) launch_tiles<CB, P, 4, 2>(b, slots, vocab, span, first_word, s);
    else launch_tiles<CB, P, 1, 2>(b, slots, vocab, span, first_word, s);
}

template <int CB>
static void launch_sums(const BackArgs& b, int parts, int slots, int64_t vocab, int64_t span, int first_word, hipStream_t s) {
    if (parts == 1) launch_parts<CB, 1>(b, slots, vocab, span, first_word, s);
    else launch_parts<CB, 2>(b, slots, vocab, span, first_word, s);
}

gptq_status head_launch(const HeadCall& c, hipStream_t s) {
    const int64_t d = c.L.d_col;
    const bool grad = c.dx != nullptr;
    const int parts = !grad ? 0 : c.dxt == GPTQ_BF16 ? 1 : 2;
    HeadArgs a = {};
    a.vocab = c.vocab; a.d = d; a.k = c.k; a.ids = c.ids; a.top = c.top; a.topt = c.topt; a.T = c.temperature;
    a.weights = c.weights; a.L = c.L; a.loss = c.loss; a.dx = c.dx; a.dxt = c.dxt;
    a.blocks = (int)((c.vocab + EB - 1) / EB);
    for (int64_t tok0 = 0; tok0 < c.n; tok0 += CHUNK) {
        const int64_t nc = c.n - tok0 < CHUNK ? c.n - tok0 : CHUNK;
        const HeadPlan p = head_plan(nc, d, c.vocab, parts, c.bits);
        layout(&a.b, (uint8_t*)c.ws, nc, nc * p.R * p.span, nc * p.R, d, c.vocab, c.group, c.k, parts);
        a.n = nc; a.tok0 = tok0; a.R = p.R; a.span = p.span;
        if (grad) {
            rows_launch(c.L, 1, c.vocab, a.b.e, a.b.T, s);
            head_emax_kernel<<<(unsigned)a.blocks, 256, 0, s>>>(a.b.e, c.vocab, a.b.emax);
            GPTQ_LAUNCH_CHECK();
        }
        GroupedArgs g = {};                                      // the whole head
        g.L = c.L; g.d_row = c.vocab; g.x = (const uint16_t*)c.x + tok0 * c.ldx; g.ldx = c.ldx; g.n = nc; g.E = 1;
        const bool large = grouped_large(g, p.R * p.span < c.vocab ? p.R * p.span : c.vocab);
        const gptq_status ready = large ? grouped_prepare(g, c.xt, c.bits, c.group, a.b.forward, s) : GPTQ_OK;
        if (ready != GPTQ_OK) return ready;
        int round = 0;
        for (int first = 0; first < p.spans; first += p.R, ++round) {
            const int slots = p.spans - first < p.R ? p.spans - first : p.R;
            const int64_t v0 = first * p.span, v1 = v0 + slots * p.span < c.vocab ? v0 + slots * p.span : c.vocab;
            GroupedArgs h = g;
            h.L.codes += v0 * c.L.code_ld;
            h.L.scales += v0 * c.L.n_groups;
            h.L.zeros += v0 * c.L.n_groups;
            h.d_row = v1 - v0; h.y = a.b.z; h.yt = GPTQ_F32; h.ldy = p.R * p.span;
            const gptq_status st = grouped_launch(h, c.xt, c.bits, c.group, large, a.b.forward, c.vocab, v0, s);
            if (st != GPTQ_OK) return st;
            a.round = round; a.slots = slots;
            const dim3 grid((unsigned)nc, (unsigned)slots);
            if (parts == 0) head_stats_kernel<0><<<grid, 256, 0, s>>>(a);
            else if (parts == 1) head_stats_kernel<1><<<grid, 256, 0, s>>>(a);
            else head_stats_kernel<2><<<grid, 256, 0, s>>>(a);
            GPTQ_LAUNCH_CHECK();
            if (grad) {
                BackArgs b = {};
                b.L = c.L; b.d_row = c.vocab; b.T = a.b.T; b.quads = quads_of(c.vocab);
                b.A[0] = a.b.A[0]; b.A[1] = a.b.A[1]; b.a0 = v0;
                b.n = nc; b.sums = a.b.O; b.f = a.b.f; b.first = round == 0;
                if (c.bits == 3) launch_sums<3>(b, parts, slots, c.vocab, p.span, (int)v0, s);
                else if (c.bits == 4) launch_sums<4>(b, parts, slots, c.vocab, p.span, (int)v0, s);
                else launch_sums<8>(b, parts, slots, c.vocab, p.span, (int)v0, s);
                GPTQ_LAUNCH_CHECK();
            }
        }
        a.slots = p.R;
        // 33 tokens x 1024 columns: 12 us in parts, 18 whole; 301 x 2048: 16 either way
        const int64_t most = grad ? ceil_div(d, 256) : 1, parts_of = 512 / nc < most ? 512 / nc : most;
        a.cols = parts_of > 1 ? ceil_div(ceil_div(d, parts_of), 64) * 64 : d;
        const dim3 grid((unsigned)nc, (unsigned)ceil_div(d, a.cols));
        if (c.bits == 3) head_final_kernel<3><<<grid, 256, 0, s>>>(a);
        else if (c.bits == 4) head_final_kernel<4><<<grid, 256, 0, s>>>(a);
        else head_final_kernel<8><<<grid, 256, 0, s>>>(a);
        GPTQ_LAUNCH_CHECK();
    }
    return GPTQ_OK;
}

}  // namespace gptq
