// A mixture-of-experts layer for a few tokens, the experts held as stored layers
// (gptqs_moe).  Four launches:
//   moe_logits_kernel  l = router x: 16 experts x 16 tokens per workgroup, columns over its waves
//   moe_topk_kernel    a wave per token: the largest logits one by one, softmax, ids and weights
//   moe_up_kernel      per chosen expert and 16 inner columns: gate and up products for the
//                      tokens that chose it, silu(gate) up w, written as two bfloat16 parts
//   moe_down_kernel    per 16 output columns: every chosen expert's product with the inner
//                      values of the tokens that chose it, summed over experts in one place
// Bound by the codes of the chosen experts, which the last two read once each.  Sums run
// in fixed orders without atomics.

#include "serving.h"
#include "stored_tile.h"

namespace gptq {

constexpr int MOE_T = 16;     // tokens per tile

struct MoeArgs {
    const uint16_t* x; int64_t ldx; int n; int64_t d, f;
    const uint16_t* router; int E, k; int renormalize;
    Stored up, down;          // E 2f x d, E d x f
    float* logits;            // n x E
    uint16_t* hi; uint16_t* lo;   // n k x f: w silu(gate) up as bfloat16 hi + lo
    int32_t* ids; float* weights;
    void* y; gptq_dtype yt;
};

constexpr int LOGW = 8;

template <int X>
__global__ __launch_bounds__(64 * LOGW) void moe_logits_kernel(MoeArgs a) {
    __shared__ float red[LOGW][4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n16 = lane & 15, q = lane >> 4;
    const int e0 = blockIdx.x * 16, t0 = blockIdx.y * MOE_T;
    const int e = e0 + n16 < a.E ? e0 + n16 : a.E - 1, t = t0 + n16 < a.n ? t0 + n16 : a.n - 1;
    const uint8_t* xrow = reinterpret_cast<const uint8_t*>(a.x + (int64_t)t * a.ldx);
    const uint8_t* rrow = reinterpret_cast<const uint8_t*>(a.router + (int64_t)e * a.d);
    f32x4_t cs = {0.f, 0.f, 0.f, 0.f};
    for (int64_t c0 = 128 * wave; c0 < a.d; c0 += 128 * LOGW) {
        const int64_t col = c0 + 32 * q;
        XRun<X, 32> xr, rr;
        if (c0 + 128 <= a.d) { xr = load_x<X, 32>(xrow + 2 * col); rr = load_x<X, 32>(rrow + 2 * col); }
        else {
            const int left = (int)(a.d - col < 32 ? a.d - col : 32);
            xr = load_x_tail<X, 32>(xrow + 2 * col, left);
            rr = load_x_tail<X, 32>(rrow + 2 * col, left);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
            cs = mfma16<X>(u32x4_t{xr.w[4 * s], xr.w[4 * s + 1], xr.w[4 * s + 2], xr.w[4 * s + 3]},
                           u32x4_t{rr.w[4 * s], rr.w[4 * s + 1], rr.w[4 * s + 2], rr.w[4 * s + 3]}, cs);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][i][lane] = cs[i];
    __syncthreads();
    if (threadIdx.x < 256) {
        const int m = threadIdx.x >> 4, n = threadIdx.x & 15;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < LOGW; ++w) v += red[w][m & 3][n + 16 * (m >> 2)];
        if (t0 + m < a.n && e0 + n < a.E) a.logits[(int64_t)(t0 + m) * a.E + e0 + n] = v;
    }
}

constexpr int MAXE = 512, MAXK = 32, EPL = MAXE / 64;   // experts per lane
constexpr int MAXN = 256;                               // tokens of a call

// One wave per token.  A NaN logit counts as -infinity; an expert already taken has index
// MAXE, behind every other of the same value.
__global__ __launch_bounds__(256) void moe_topk_kernel(MoeArgs a) {
    const int lane = threadIdx.x & 63, t = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= a.n) return;
    float v[EPL];
    int at[EPL];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane + 64 * i;
        const float l = e < a.E ? a.logits[(int64_t)t * a.E + e] : -INFINITY;
        v[i] = l == l ? l : -INFINITY;
        at[i] = e < a.E ? e : MAXE;
        top = fmaxf(top, v[i]);
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    float sum = 0.f;
    if (!a.renormalize) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) sum += lane + 64 * i < a.E ? expf(v[i] - top) : 0.f;
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
    }
    float mine = 0.f;           // lane j: the j-th choice's exp
    int id = 0;
    for (int j = 0; j < a.k; ++j) {
        float bv = -INFINITY;
        int bi = MAXE;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (v[i] > bv || (v[i] == bv && at[i] < bi)) { bv = v[i]; bi = at[i]; }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) {
            const float ov = __shfl_xor(bv, o);
            const int oi = __shfl_xor(bi, o);
            if (ov > bv || (ov == bv && oi < bi)) { bv = ov; bi = oi; }
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (at[i] == bi) { at[i] = MAXE; v[i] = -INFINITY; }
        const float p = expf(bv - top);
        if (a.renormalize) sum += p;
        if (lane == j) { mine = p; id = bi; }
    }
    if (lane < a.k) {
        a.ids[(int64_t)t * a.k + lane] = id;
        a.weights[(int64_t)t * a.k + lane] = mine / sum;
    }
}

// The experts that the calls' pairs name, as bits in LDS (every thread of the workgroup).
GPTQ_DEV void active_bits(const MoeArgs& a, int p0, int p1, uint32_t* bits, int threads) {
    if (threadIdx.x < MAXE / 32) bits[threadIdx.x] = 0;
    __syncthreads();
    for (int p = p0 + threadIdx.x; p < p1; p += threads) {
        const int e = a.ids[p];
        atomicOr(&bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
}

// The s-th expert of the bits, or -1.
GPTQ_DEV int nth_expert(const uint32_t* bits, int s) {
    for (int w = 0; w < MAXE / 32; ++w) {
        uint32_t b = bits[w];
        const int c = __popc(b);
        if (s < c) {
            for (; s > 0; --s) b &= b - 1;
            return 32 * w + __builtin_ctz(b);
        }
        s -= c;
    }
    return -1;
}

constexpr int UPW = 8;

// Grid: 16 inner columns x the s-th chosen expert.
template <int X, int CB, int RUN>
__global__ __launch_bounds__(64 * UPW) void moe_up_kernel(MoeArgs a) {
    __shared__ uint32_t bits[MAXE / 32];
    __shared__ int list[MAXN], count;
    __shared__ float red[UPW][2][4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n16 = lane & 15;
    const int pairs = a.n * a.k;
    active_bits(a, 0, pairs, bits, 64 * UPW);
    const int e = nth_expert(bits, blockIdx.y);
    if (e < 0) return;                                      // the whole workgroup
    if (wave == 0) {                                        // the pairs that chose e, in order
        int c = 0;
        for (int p0 = 0; p0 < pairs; p0 += 64) {
            const int p = p0 + lane;
            const bool mine = p < pairs && a.ids[p] == e;
            const uint64_t b = __ballot(mine);
            if (mine) list[c + __popcll(b & ((1ull << lane) - 1))] = p;
            c += __popcll(b);
        }
        if (lane == 0) count = c;
    }
    __syncthreads();
    const int cnt = count;
    const int64_t f0 = (int64_t)blockIdx.x * 16;
    const int64_t fr = f0 + n16 < a.f ? f0 + n16 : a.f - 1;
    const int64_t row[2] = {(int64_t)e * 2 * a.f + fr, (int64_t)e * 2 * a.f + a.f + fr};
    const int nck = (int)((a.d + SCK - 1) / SCK);
    for (int m0 = 0; m0 < cnt; m0 += MOE_T) {
        const int p = list[m0 + n16 < cnt ? m0 + n16 : cnt - 1];
        const uint8_t* const xrow[1] = {reinterpret_cast<const uint8_t*>(a.x + (int64_t)(p / a.k) * a.ldx)};
        f32x4_t acc[1][2] = {{f32x4_t{0.f, 0.f, 0.f, 0.f}, f32x4_t{0.f, 0.f, 0.f, 0.f}}};
        stored_accumulate<X, CB, RUN, 1, 2, RUN == 32 ? 2 : 1>(acc, a.up, row, xrow, wave, UPW, nck);
        __syncthreads();                                    // the last tile's sums are read
#pragma unroll
        for (int rb = 0; rb < 2; ++rb)
#pragma unroll
            for (int i = 0; i < 4; ++i) red[wave][rb][i][lane] = acc[0][rb][i];
        __syncthreads();
        if (threadIdx.x < 256) {
            const int m = threadIdx.x >> 4, n = threadIdx.x & 15;
            if (m0 + m < cnt && f0 + n < a.f) {
                float g = 0.f, u = 0.f;
#pragma unroll
                for (int w = 0; w < UPW; ++w) {
                    g += red[w][0][m & 3][n + 16 * (m >> 2)];
                    u += red[w][1][m & 3][n + 16 * (m >> 2)];
                }
                const int pr = list[m0 + m];
                const float h = g / (1.f + expf(-g)) * u * a.weights[pr];
                const uint16_t hb = f32_to_bf16_bits(h);
                a.hi[(int64_t)pr * a.f + f0 + n] = hb;
                a.lo[(int64_t)pr * a.f + f0 + n] = f32_to_bf16_bits(h - bf16_bits_to_f32(hb));
            }
        }
    }
}

// Grid: 16 output columns x NTT tiles of 16 tokens.  The waves share the (expert, chunk)
// pairs; token t of a tile keeps its place in the operand, empty where it did not choose
// the expert, and its sums are left alone there.
template <int CB, int RUN, int NTT, int W>
__global__ __launch_bounds__(64 * W) void moe_down_kernel(MoeArgs a) {
    constexpr int X = X_BF16, P = 32 / RUN;
    __shared__ uint32_t bits[MAXE / 32];
    __shared__ uint16_t experts[MAXE];
    __shared__ uint8_t choice[MAXE][16 * NTT];              // [active expert][token]: its j, or 255
    __shared__ float red[W][NTT][4][64];
    __shared__ int n_active;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n16 = lane & 15, q = lane >> 4;
    const int t0 = blockIdx.y * 16 * NTT, t1 = t0 + 16 * NTT < a.n ? t0 + 16 * NTT : a.n;
    const int64_t r0 = (int64_t)blockIdx.x * 16;
    active_bits(a, t0 * a.k, t1 * a.k, bits, 64 * W);
    auto rank_of = [&](int e) {                             // active experts below e
        int c = 0;
        for (int w = 0; w < (e >> 5); ++w) c += __popc(bits[w]);
        return c + __popc(bits[e >> 5] & ((1u << (e & 31)) - 1));
    };
    for (int e = threadIdx.x; e < MAXE; e += 64 * W)
        if ((bits[e >> 5] >> (e & 31)) & 1) experts[rank_of(e)] = (uint16_t)e;
    if (threadIdx.x == 0) {
        int c = 0;
        for (int w = 0; w < MAXE / 32; ++w) c += __popc(bits[w]);
        n_active = c;
    }
    __syncthreads();
    const int na = n_active;
    for (int i = threadIdx.x; i < na * 16 * NTT; i += 64 * W) (&choice[0][0])[i] = 255;
    __syncthreads();
    for (int p = t0 * a.k + threadIdx.x; p < t1 * a.k; p += 64 * W)
        choice[rank_of(a.ids[p])][p / a.k - t0] = (uint8_t)(p % a.k);
    __syncthreads();

    const Stored& L = a.down;
    const int64_t rr = r0 + n16 < a.d ? r0 + n16 : a.d - 1;
    const int nck = (int)((a.f + SCK - 1) / SCK);
    f32x4_t acc[NTT];
#pragma unroll
    for (int tt = 0; tt < NTT; ++tt) acc[tt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // chunk c of expert e goes to wave (e nck + c) % W: the same one whichever other experts
    // are active, so a token's sums do not depend on the other tokens' choices
    int s = 0, c = -1;
    auto next = [&]() {                                     // wave-uniform
        if (c >= 0) { c += W; if (c < nck) return; ++s; }
        for (; s < na; ++s) {
            c = (int)(((int64_t)wave - (int64_t)experts[s] * nck) % W);
            c = c < 0 ? c + W : c;
            if (c < nck) return;
        }
    };
    for (next(); s < na; next()) {
        const int64_t row = (int64_t)experts[s] * a.d + rr;
        const bool full = (int64_t)(c + 1) * SCK <= a.f;
        uint32_t has[NTT];
        int64_t hrow[NTT];
        bool mine[NTT];
#pragma unroll
        for (int tt = 0; tt < NTT; ++tt) {
            const int j = choice[s][16 * tt + n16];
            mine[tt] = j != 255;
            has[tt] = (uint32_t)__ballot(mine[tt]) & 0xFFFFu;
            hrow[tt] = ((int64_t)(t0 + 16 * tt + n16) * a.k + j) * a.f;
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int64_t col = (int64_t)c * SCK + p * 4 * RUN + q * RUN;
            const int left = (int)(a.f - col < RUN ? a.f - col : RUN);
            int g = RUN == 32 ? c / L.cpg : c * P + p;
            g = g < L.n_groups ? g : L.n_groups - 1;
            const uint8_t* src = L.codes + row * L.code_ld + col / 8 * CB;
            const Raw<CB, RUN> cw = full ? load_raw<CB, RUN>(src) : load_raw_tail<CB, RUN>(src, left);
            const float S = f16_bits_to_f32(L.scales[row * L.n_groups + g]);
            const float z = f16_bits_to_f32(L.zeros[row * L.n_groups + g]);
            XRun<X, RUN> xh[NTT], xl[NTT];
#pragma unroll
            for (int tt = 0; tt < NTT; ++tt) {
                const int m = mine[tt] ? left : 0;          // nothing of a token that did not choose it
                const uint8_t* hp = reinterpret_cast<const uint8_t*>(a.hi + hrow[tt] + col);
                const uint8_t* lp = reinterpret_cast<const uint8_t*>(a.lo + hrow[tt] + col);
                if (m == RUN) { xh[tt] = load_x<X, RUN>(hp); xl[tt] = load_x<X, RUN>(lp); }
                else { xh[tt] = load_x_tail<X, RUN>(hp, m); xl[tt] = load_x_tail<X, RUN>(lp, m); }
            }
            const float zc = zero_part<X, CB>(z), rz = z - zc;
            float xs[NTT][4];
#pragma unroll
            for (int tt = 0; tt < NTT; ++tt)
#pragma unroll
                for (int i = 0; i < 4; ++i) xs[tt][i] = 0.f;
            if (__ballot(!(rz == 0.f)) != 0) {
                const u32x4_t w1 = {ones_word<X>(), ones_word<X>(), ones_word<X>(), ones_word<X>()};
#pragma unroll
                for (int tt = 0; tt < NTT; ++tt) {
                    f32x4_t sm = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int u = 0; u < RUN / 8; ++u) {
                        const uint32_t *h = xh[tt].w + 4 * u, *l = xl[tt].w + 4 * u;
                        sm = mfma16<X>(u32x4_t{h[0], h[1], h[2], h[3]}, w1, sm);
                        sm = mfma16<X>(u32x4_t{l[0], l[1], l[2], l[3]}, w1, sm);
                    }
                    settle(sm);
#pragma unroll
                    for (int i = 0; i < 4; ++i) xs[tt][i] = sm[i];
                }
            }
            f32x4_t cs[NTT];
#pragma unroll
            for (int tt = 0; tt < NTT; ++tt) cs[tt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int u = 0; u < RUN / 8; ++u) {
                uint32_t b0[2], b1[2];
                minus_zero_16<X>(code_bytes4<CB, RUN>(cw, 2 * u), zc, b0);
                minus_zero_16<X>(code_bytes4<CB, RUN>(cw, 2 * u + 1), zc, b1);
                const u32x4_t b = {b0[0], b0[1], b1[0], b1[1]};
#pragma unroll
                for (int tt = 0; tt < NTT; ++tt) {
                    const uint32_t *h = xh[tt].w + 4 * u, *l = xl[tt].w + 4 * u;
                    cs[tt] = mfma16<X>(u32x4_t{h[0], h[1], h[2], h[3]}, b, cs[tt]);
                    cs[tt] = mfma16<X>(u32x4_t{l[0], l[1], l[2], l[3]}, b, cs[tt]);
                }
            }
#pragma unroll
            for (int tt = 0; tt < NTT; ++tt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float v = fmaf(S, fmaf(-rz, xs[tt][i], cs[tt][i]), acc[tt][i]);
                    acc[tt][i] = (has[tt] >> (4 * q + i)) & 1 ? v : acc[tt][i];
                }
        }
    }
#pragma unroll
    for (int tt = 0; tt < NTT; ++tt)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[wave][tt][i][lane] = acc[tt][i];
    __syncthreads();
    for (int o = threadIdx.x; o < NTT * 256; o += 64 * W) {
        const int tt = o >> 8, m = (o >> 4) & 15, n = o & 15;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) v += red[w][tt][m & 3][n + 16 * (m >> 2)];
        const int t = t0 + 16 * tt + m;
        if (t < a.n && r0 + n < a.d) store_out(a.y, a.yt, (int64_t)t * a.d + r0 + n, v);
    }
}

template <int X, int CB, int RUN>
static gptq_status launch(const MoeArgs& a, hipStream_t s) {
    const unsigned ef = (unsigned)((a.f + 15) / 16), dd = (unsigned)((a.d + 15) / 16);
    const int slots = a.E < a.n * a.k ? a.E : a.n * a.k;
    moe_logits_kernel<X><<<dim3((unsigned)((a.E + 15) / 16), (unsigned)((a.n + 15) / 16)), 64 * LOGW, 0, s>>>(a);
    GPTQ_LAUNCH_CHECK();
    moe_topk_kernel<<<(unsigned)((a.n + 3) / 4), 256, 0, s>>>(a);
    GPTQ_LAUNCH_CHECK();
    moe_up_kernel<X, CB, RUN><<<dim3(ef, (unsigned)slots), 64 * UPW, 0, s>>>(a);
    GPTQ_LAUNCH_CHECK();
    if (a.n <= 16) moe_down_kernel<CB, RUN, 1, 16><<<dim3(dd, 1), 64 * 16, 0, s>>>(a);
    else moe_down_kernel<CB, RUN, 4, 8><<<dim3(dd, (unsigned)((a.n + 63) / 64)), 64 * 8, 0, s>>>(a);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

template <int X, int CB>
static gptq_status launch_runs(const MoeArgs& a, int group, hipStream_t s) {
    return group == 32 ? launch<X, CB, 8>(a, s) : group == 64 ? launch<X, CB, 16>(a, s) : launch<X, CB, 32>(a, s);
}

template <int X>
static gptq_status launch_bits(const MoeArgs& a, int bits, int group, hipStream_t s) {
    return bits == 3 ? launch_runs<X, 3>(a, group, s) : bits == 4 ? launch_runs<X, 4>(a, group, s) : launch_runs<X, 8>(a, group, s);
}

static size_t up16(size_t v) { return (v + 15) & ~(size_t)15; }

size_t moe_ws_bytes(int64_t n, int64_t f, int E, int k) {
    return up16((size_t)n * E * sizeof(float)) + 2 * up16((size_t)n * k * (size_t)f * sizeof(uint16_t));
}

gptq_status moe_launch(const MoeCall& c, hipStream_t s) {
    MoeArgs a;
    a.x = (const uint16_t*)c.x; a.ldx = c.ldx; a.n = (int)c.n; a.d = c.d; a.f = c.f;
    a.router = (const uint16_t*)c.router; a.E = c.E; a.k = c.k; a.renormalize = c.renormalize;
    a.up = stored_layer(c.up_codes, c.up_scales, c.up_zeros, c.d, c.bits, c.group);
    a.down = stored_layer(c.down_codes, c.down_scales, c.down_zeros, c.f, c.bits, c.group);
    uint8_t* w = (uint8_t*)c.ws;
    a.logits = (float*)w;
    w += up16((size_t)c.n * c.E * sizeof(float));
    a.hi = (uint16_t*)w;
    a.lo = (uint16_t*)(w + up16((size_t)c.n * c.k * (size_t)c.f * sizeof(uint16_t)));
    a.ids = c.ids; a.weights = c.weights; a.y = c.y; a.yt = c.yt;
    return c.xt == GPTQ_BF16 ? launch_bits<X_BF16>(a, c.bits, c.group, s) : launch_bits<X_F16>(a, c.bits, c.group, s);
}

}  // namespace gptq
