// A mixture-of-experts layer for a few tokens, the experts held as stored layers
// (gptqs_moe):
//   moe_logits_kernel  l = router x: 16 experts x 16 tokens per workgroup, columns over its waves
//   moe_plan_kernel    a wave per token takes the largest logits one by one; softmax; the pairs
//                      (token, choice) sorted by expert
//   moe_up_kernel      per expert in use and 16 inner columns: gate and up products for the
//                      tokens that chose it, silu(gate) up w, written as bfloat16 parts (two
//                      for 16-bit outputs, three for fp32)
//   moe_down_kernel    per expert in use and 16 output columns: the pairs' outputs, fp32
//   moe_sum_kernel     y = a token's pairs added in the order of its choices
// Sums that are not finite are taken once more as sum S (u - z) x (finite_sum in
// stored_tile.h), in up behind its tiles and for down in moe_sum_kernel.
// Bound by the codes of the chosen experts, which up and down read once each.  One token,
// 8 of 64 experts of 2048 x 1408 int4: 4.2 + 5.7 + 14 + 10.6 + 3.9 us for 35 MB of codes,
// latency of five dependent launches; 32 tokens, 2 of 16 experts of 4096 x 5504: 8.8 + 4.5
// + 4.8 + 121 + 89 + 4.7 us (choice and plan in two launches), up at 3.0 TB/s and down at
// 2.0: vector unit half busy, and nothing in flight while a wave multiplies (one chunk in
// registers); in down the inner values' parts are most of the loads (32 rows per workgroup,
// gathered loads of them through LDS, and two chunks ahead all measured slower).  Every 16
// tokens of an expert read its codes again: 64 tokens 261 us, 256 679.  A first form in
// which a workgroup of down walked all experts took 494 us.  Sums run in fixed orders
// without atomics, and a token's do not depend on the other tokens' choices.

#include "serving.h"
#include "stored_tile.h"

namespace gptq {

constexpr int MOE_T = 16;     // tokens per tile

struct MoeArgs {
    const uint16_t* x; int64_t ldx; int n; int64_t d, f;
    const uint16_t* router; int E, k; int renormalize;
    Stored up, down;          // E 2f x d, E d x f
    float* logits;            // n x E
    uint16_t* inner;          // n k x f, for each part of w silu(gate) up in bfloat16
    float* part;              // n k x d: w D h per pair
    int32_t* plan;            // see moe_plan_kernel
    int32_t* ids; float* weights;
    void* y; gptq_dtype yt;
};

// Elements from one part of the inner values to the next: whole 16 bytes.
GPTQ_DEV int64_t part_elems(const MoeArgs& a) { return ((int64_t)a.n * a.k * a.f + 7) & ~(int64_t)7; }

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
    settle(cs);                                             // products end behind the loop's branch
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

static_assert(MOE_MAX_EXPERTS == 512, "a plan's expert has 9 bits");
constexpr int MAXE = 512, EPL = MAXE / 64;   // experts per lane

// Maximum over the wave, in every lane's copy of lane 63 (DPP, no LDS).
GPTQ_DEV uint32_t wave_umax(uint32_t v) {
#define GPTQ_STEP(CTRL, ROWS)                                                                                  \
    {                                                                                                          \
        const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, ROWS, 0xf, false);      \
        v = o > v ? o : v;                                                                                     \
    }
    GPTQ_STEP(0x111, 0xf) GPTQ_STEP(0x112, 0xf) GPTQ_STEP(0x114, 0xf) GPTQ_STEP(0x118, 0xf)   // row_shr 1, 2, 4, 8
    GPTQ_STEP(0x142, 0xa) GPTQ_STEP(0x143, 0xc)                                               // row_bcast 15, 31
#undef GPTQ_STEP
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// The top_k largest logits of token t and their softmax, by one wave.  A logit's key orders
// as the logits do (a NaN as -infinity, -0 as 0); 0 is no logit's key and marks what is
// taken or absent.  Of equal keys the lowest expert is found as the largest MAXE - 1 - e.
GPTQ_DEV void topk_of(const MoeArgs& a, int t) {
    const int lane = threadIdx.x & 63;
    uint32_t key[EPL];
    float l[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane + 64 * i;
        float v = e < a.E ? a.logits[(int64_t)t * a.E + e] : -INFINITY;
        v = v == v ? v + 0.f : -INFINITY;
        const uint32_t u = __float_as_uint(v);
        l[i] = v;
        key[i] = e < a.E ? u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u) : 0u;
    }
    float top = 0.f, sum = 0.f, mine = 0.f;           // mine: lane j holds the j-th choice's exp
    int id = 0;
    for (int j = 0; j < a.k; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) best = key[i] > best ? key[i] : best;
        best = wave_umax(best);
        uint32_t at = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) at = key[i] == best && (uint32_t)(MAXE - lane - 64 * i) > at ? MAXE - lane - 64 * i : at;
        const int e = MAXE - (int)wave_umax(at);
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = e == lane + 64 * i ? 0u : key[i];
        const float v = __uint_as_float(best ^ ((best >> 31) ? 0x80000000u : 0xFFFFFFFFu));
        if (j == 0) top = v;
        const float p = expf(v - top);
        sum += p;
        if (lane == j) { mine = p; id = e; }
    }
    if (!a.renormalize) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) sum += lane + 64 * i < a.E ? expf(l[i] - top) : 0.f;
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
    }
    if (lane < a.k) {
        a.ids[(int64_t)t * a.k + lane] = id;
        a.weights[(int64_t)t * a.k + lane] = mine / sum;
    }
}

__global__ __launch_bounds__(256) void moe_topk_kernel(MoeArgs a) {
    const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t < a.n) topk_of(a, t);
}

// The plan: the chosen experts in rising order, and the pairs (token, choice) sorted by
// expert, in token order within one.  plan: [0] experts in use, [1 + 2 s] the s-th of them,
// [2 + 2 s] where its pairs begin (the last one's end with the pairs), from PAIRS on the pairs.
constexpr int PAIRS = 1 + 2 * MAXE;
constexpr int PLAN_W = 16;

// A stable counting sort: each wave counts its share of the pairs, a prefix over the waves and
// one over the experts say where each wave's pairs of an expert go, and a lane's place among
// its 64 is the number of lower lanes with its expert (ballots of the expert's 9 bits).  256
// tokens, 32 of 512 experts: 11 us, where a walk over all pairs for each expert took 708.
//
// TOPK: the same workgroup chooses first (few tokens: one launch less).
template <bool TOPK>
__global__ __launch_bounds__(64 * PLAN_W) void moe_plan_kernel(MoeArgs a) {
    __shared__ int next[PLAN_W][MAXE], count[MAXE], start[MAXE];   // next: a wave's counts, then where its next pair goes
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, pairs = a.n * a.k;
    if (TOPK) {
        for (int t = wave; t < a.n; t += PLAN_W) topk_of(a, t);
        __threadfence_block();
    }
    const int share = (pairs + 64 * PLAN_W - 1) / (64 * PLAN_W) * 64;                       // pairs per wave
    const int first = wave * share, last = first + share < pairs ? first + share : pairs;
    for (int e = threadIdx.x; e < PLAN_W * MAXE; e += 64 * PLAN_W) (&next[0][0])[e] = 0;
    __syncthreads();
    for (int p = first + lane; p < last; p += 64) atomicAdd(&next[wave][a.ids[p]], 1);      // whole numbers: any order
    __syncthreads();
    for (int e = threadIdx.x; e < MAXE; e += 64 * PLAN_W) {
        int c = 0;
#pragma unroll
        for (int w = 0; w < PLAN_W; ++w) {
            const int mine = next[w][e];
            next[w][e] = c;
            c += mine;
        }
        count[e] = c;
    }
    __syncthreads();
    if (wave == 0) {                                        // prefix sums over the experts, EPL per lane
        int c[EPL], mine = 0, used = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) { c[i] = count[EPL * lane + i]; mine += c[i]; used += c[i] > 0; }
        int at = mine, us = used;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int u = __shfl_up(at, o), v = __shfl_up(us, o);
            if (lane >= o) { at += u; us += v; }
        }
        const int total = __shfl(us, 63);
        at -= mine;
        us -= used;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = EPL * lane + i;
            start[e] = at;
            if (c[i]) { a.plan[1 + 2 * us] = e; a.plan[2 + 2 * us] = at; ++us; }
            at += c[i];
        }
        if (lane == 0) a.plan[0] = total;
    }
    __syncthreads();
    for (int p0 = first; p0 < last; p0 += 64) {             // wave-uniform
        const int p = p0 + lane, e = p < last ? a.ids[p] : 0;
        uint64_t same = __ballot(p < last);                 // the lanes with this lane's expert
#pragma unroll
        for (int b = 0; b < 9; ++b) {
            const uint64_t set = __ballot((e >> b) & 1);
            same &= (e >> b) & 1 ? set : ~set;
        }
        const int before = next[wave][e];
        lds_handover();                                     // all read before the last of them adds
        if (p < last) {
            a.plan[PAIRS + start[e] + before + __popcll(same & ((1ull << lane) - 1))] = p;
            if (same >> lane == 1) next[wave][e] = before + __popcll(same);
        }
        lds_handover();
    }
}

constexpr int MW = 8;         // waves per workgroup of the gate and up products

// Pair pr's inner value at column c from its gate and up sums; whether it is finite.
GPTQ_DEV bool inner_value(const MoeArgs& a, int pr, int64_t c, float g, float u) {
    const float h = g / (1.f + expf(-g)) * u * a.weights[pr];
    uint16_t part[3];
    bf16_parts(h, part);
    uint16_t* to = a.inner + (int64_t)pr * a.f + c;
    const int64_t plane = part_elems(a);
    to[0] = part[0];
    to[plane] = part[1];
    if (a.yt == GPTQ_F32) to[2 * plane] = part[2];
    return fabsf(h) < INFINITY;
}

// Grid: 16 inner columns x the s-th expert in use.
template <int X, int CB, int RUN>
__global__ __launch_bounds__(64 * MW, 4) void moe_up_kernel(MoeArgs a) {
    __shared__ float red[MW][2][4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n16 = lane & 15;
    const int s = blockIdx.y;
    if (s >= a.plan[0]) return;                             // the whole workgroup
    const int e = a.plan[1 + 2 * s], p0 = a.plan[2 + 2 * s];
    const int cnt = (s + 1 < a.plan[0] ? a.plan[4 + 2 * s] : a.n * a.k) - p0;
    const int64_t f0 = (int64_t)blockIdx.x * 16;
    const int64_t fr = f0 + n16 < a.f ? f0 + n16 : a.f - 1;
    const int64_t row[2] = {(int64_t)e * 2 * a.f + fr, (int64_t)e * 2 * a.f + a.f + fr};
    uint64_t lost = 0;
    for (int m0 = 0; m0 < cnt; m0 += MOE_T) {
        const bool live = m0 + n16 < cnt;
        const int p = live ? a.plan[PAIRS + p0 + m0 + n16] : 0;
        const XScattered<1> xr = {{live ? reinterpret_cast<const uint8_t*>(a.x + (int64_t)(p / a.k) * a.ldx) : nullptr}};
        f32x4_t acc[1][2] = {{f32x4_t{0.f, 0.f, 0.f, 0.f}, f32x4_t{0.f, 0.f, 0.f, 0.f}}};
        stored_accumulate<X, CB, RUN, 1, 2, 1>(acc, a.up, row, xr, wave, MW);
        __syncthreads();                                    // the last tile's sums are read
#pragma unroll
        for (int rb = 0; rb < 2; ++rb)
#pragma unroll
            for (int i = 0; i < 4; ++i) red[wave][rb][i][lane] = acc[0][rb][i];
        __syncthreads();
        if (threadIdx.x < 256) {
            const int m = threadIdx.x >> 4, n = threadIdx.x & 15;
            bool bad = false;
            if (m0 + m < cnt && f0 + n < a.f) {
                float g = 0.f, u = 0.f;
#pragma unroll
                for (int w = 0; w < MW; ++w) {
                    g += red[w][0][m & 3][n + 16 * (m >> 2)];
                    u += red[w][1][m & 3][n + 16 * (m >> 2)];
                }
                bad = !inner_value(a, a.plan[PAIRS + p0 + m0 + m], f0 + n, g, u);
            }
            lost |= __ballot(bad);
        }
    }
    // Values that are not finite, once more from sums by wave_sum (see finite_sum: an infinite
    // g or u, or one that is no number, leaves no finite value).  Behind the loop, whose
    // registers it would take.
    if (lost == 0) return;                                  // wave-uniform; no barrier below
    for (int m0 = 0; m0 < cnt; m0 += MOE_T) {
        const int m = threadIdx.x >> 4, n = threadIdx.x & 15;
        const bool mine = m0 + m < cnt && f0 + n < a.f;
        const int pr = mine ? a.plan[PAIRS + p0 + m0 + m] : 0;
        const float h = mine ? bf16_bits_to_f32(a.inner[(int64_t)pr * a.f + f0 + n]) : 0.f;
        const auto x8 = [&](int i, int64_t c, int m8, float (&x)[8]) {
            load_x8<X>(a.x + (int64_t)(a.plan[PAIRS + p0 + m0 + (i >> 4)] / a.k) * a.ldx + c, m8, x);
        };
        const float g = finite_sum<CB>(h, mine, a.up, [&](int i) { return (int64_t)e * 2 * a.f + f0 + (i & 15); }, x8);
        const float u = finite_sum<CB>(h, mine, a.up, [&](int i) { return ((int64_t)e * 2 + 1) * a.f + f0 + (i & 15); }, x8);
        if (!(fabsf(h) < INFINITY)) inner_value(a, pr, f0 + n, g, u);
    }
}

// Grid: 16 output columns x the s-th expert in use.  The bfloat16 parts of a pair's inner
// values are tiles of the same tokens; their sums are added at the end.
//
// Three parts take 157 registers, which eight waves per workgroup would leave one workgroup
// per compute unit, four waves three of them: fp32 outputs, eight / four: 32 tokens, 2 of 16
// experts of 4096 x 5504, 291 / 257 us a call; one, 8 of 64 of 2048 x 1408, 42.0 / 37.4 (with
// two parts for 16-bit outputs 226 and 36.2).
template <int PARTS> constexpr int down_waves() { return PARTS == 2 ? 8 : 4; }

template <int CB, int RUN, int PARTS>
__global__ __launch_bounds__(64 * down_waves<PARTS>(), PARTS == 2 ? 4 : RUN == 32 ? 3 : 2)
void moe_down_kernel(MoeArgs a) {
    constexpr int W = down_waves<PARTS>();
    __shared__ float red[W][4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n16 = lane & 15;
    const int s = blockIdx.y;
    if (s >= a.plan[0]) return;
    const int e = a.plan[1 + 2 * s], p0 = a.plan[2 + 2 * s];
    const int cnt = (s + 1 < a.plan[0] ? a.plan[4 + 2 * s] : a.n * a.k) - p0;
    const int64_t r0 = (int64_t)blockIdx.x * 16;
    const int64_t row[1] = {(int64_t)e * a.d + (r0 + n16 < a.d ? r0 + n16 : a.d - 1)};
    for (int m0 = 0; m0 < cnt; m0 += MOE_T) {
        const bool live = m0 + n16 < cnt;
        const int64_t at = live ? (int64_t)a.plan[PAIRS + p0 + m0 + n16] * a.f : 0;
        XScattered<PARTS> xr;
        f32x4_t acc[PARTS][1];
#pragma unroll
        for (int j = 0; j < PARTS; ++j) {
            xr.row[j] = live ? reinterpret_cast<const uint8_t*>(a.inner + j * part_elems(a) + at) : nullptr;
            acc[j][0] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
        stored_accumulate<X_BF16, CB, RUN, PARTS, 1, 1>(acc, a.down, row, xr, wave, W);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v = acc[PARTS - 1][0][i];                 // the smallest first
#pragma unroll
            for (int j = PARTS - 2; j >= 0; --j) v += acc[j][0][i];
            red[wave][i][lane] = v;
        }
        __syncthreads();
        if (threadIdx.x < 256) {
            const int m = threadIdx.x >> 4, n = threadIdx.x & 15;
            if (m0 + m < cnt && r0 + n < a.d) {
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) v += red[w][m & 3][n + 16 * (m >> 2)];
                a.part[(int64_t)a.plan[PAIRS + p0 + m0 + m] * a.d + r0 + n] = v;
            }
        }
    }
}

// y from the pairs' outputs; those that are not finite once more from down's rows (finite_sum:
// here and not in down, whose registers are all taken).
template <int CB>
__global__ __launch_bounds__(256) void moe_sum_kernel(MoeArgs a) {
    const int64_t r0 = (int64_t)blockIdx.x * 256, r = r0 + threadIdx.x;
    const int t = blockIdx.y;
    const bool live = r < a.d;
    const float* part = a.part + (int64_t)t * a.k * a.d + (live ? r : 0);
    float v = 0.f;
    for (int j = 0; j < a.k; ++j) v += part[j * a.d];
    if (__ballot(live && !(fabsf(v) < INFINITY)) != 0) {    // wave-uniform, rare
        v = 0.f;
        for (int j = 0; j < a.k; ++j) {
            const int64_t pr = (int64_t)t * a.k + j;
            v += finite_sum<CB>(
                part[j * a.d], live, a.down, [&](int i) { return (int64_t)a.ids[pr] * a.d + r0 + i; },
                [&](int, int64_t c, int m8, float (&x)[8]) {
                    const uint16_t* h = a.inner + pr * a.f + c;
                    load_x8<X_BF16>(h, m8, x);
                    for (int q = 1; q < (a.yt == GPTQ_F32 ? 3 : 2); ++q) {
                        float y[8];
                        load_x8<X_BF16>(h + q * part_elems(a), m8, y);
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] += y[e];
                    }
                });
        }
    }
    if (live) store_out(a.y, a.yt, (int64_t)t * a.d + r, v);
}

template <int X, int CB, int RUN>
static gptq_status launch(const MoeArgs& a, hipStream_t s) {
    const unsigned ef = (unsigned)((a.f + 15) / 16);
    const int slots = a.E < a.n * a.k ? a.E : a.n * a.k;
    moe_logits_kernel<X><<<dim3((unsigned)((a.E + 15) / 16), (unsigned)((a.n + 15) / 16)), 64 * LOGW, 0, s>>>(a);
    GPTQ_LAUNCH_CHECK();
    // While each of its waves has one token at most, one workgroup chooses and plans; beyond,
    // choosing is spread over the device first.  Whole calls, 512 x 256 int4 g128, one workgroup /
    // two launches, us: 1 token, 8, 64 and 256 experts: 16.4 / 17.7, 17.1 / 18.3, 17.1 / 18.2; 16
    // tokens: 18.8 / 19.1, 23.0 / 23.2, 23.0 / 23.2; 32 tokens: 22.2 / 19.5, 30.9 / 26.7, 32.9 /
    // 30.8.
    if (a.n <= PLAN_W) moe_plan_kernel<true><<<1, 64 * PLAN_W, 0, s>>>(a);
    else {
        moe_topk_kernel<<<(unsigned)((a.n + 3) / 4), 256, 0, s>>>(a);
        GPTQ_LAUNCH_CHECK();
        moe_plan_kernel<false><<<1, 64 * PLAN_W, 0, s>>>(a);
    }
    GPTQ_LAUNCH_CHECK();
    moe_up_kernel<X, CB, RUN><<<dim3(ef, (unsigned)slots), 64 * MW, 0, s>>>(a);
    GPTQ_LAUNCH_CHECK();
    const dim3 down((unsigned)((a.d + 15) / 16), (unsigned)slots);
    // Parts of the inner values: two, 2^-17 of each, are far below a 16-bit output's rounding
    // (2^-8, 2^-11); fp32 outputs take three, which are the values themselves.
    if (a.yt == GPTQ_F32) moe_down_kernel<CB, RUN, 3><<<down, 64 * down_waves<3>(), 0, s>>>(a);
    else moe_down_kernel<CB, RUN, 2><<<down, 64 * down_waves<2>(), 0, s>>>(a);
    GPTQ_LAUNCH_CHECK();
    moe_sum_kernel<CB><<<dim3((unsigned)((a.d + 255) / 256), (unsigned)a.n), 256, 0, s>>>(a);
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

// Offsets of the workspace's parts, in this order, each 16-byte aligned; the last is its size.
struct MoeWs { size_t inner, part, plan, end; };
static MoeWs moe_ws(int64_t n, int64_t d, int64_t f, int E, int k) {
    MoeWs w;
    const size_t inner = up16((size_t)n * k * (size_t)f * sizeof(uint16_t));   // one part (part_elems)
    w.inner = up16((size_t)n * E * sizeof(float));
    w.part = w.inner + 3 * inner;
    w.plan = w.part + up16((size_t)n * k * (size_t)d * sizeof(float));
    w.end = w.plan + up16((size_t)(PAIRS + n * k) * sizeof(int32_t));
    return w;
}

size_t moe_ws_bytes(int64_t n, int64_t d, int64_t f, int E, int k) { return moe_ws(n, d, f, E, k).end; }

gptq_status moe_launch(const MoeCall& c, hipStream_t s) {
    MoeArgs a;
    a.x = (const uint16_t*)c.x; a.ldx = c.ldx; a.n = (int)c.n; a.d = c.d; a.f = c.f;
    a.router = (const uint16_t*)c.router; a.E = c.E; a.k = c.k; a.renormalize = c.renormalize;
    a.up = stored_layer(c.up_codes, c.up_scales, c.up_zeros, c.d, c.bits, c.group);
    a.down = stored_layer(c.down_codes, c.down_scales, c.down_zeros, c.f, c.bits, c.group);
    uint8_t* w = (uint8_t*)c.ws;
    const MoeWs o = moe_ws(c.n, c.d, c.f, c.E, c.k);
    a.logits = (float*)w;
    a.inner = (uint16_t*)(w + o.inner);
    a.part = (float*)(w + o.part);
    a.plan = (int32_t*)(w + o.plan);
    a.ids = c.ids; a.weights = c.weights; a.y = c.y; a.yt = c.yt;
    return c.xt == GPTQ_BF16 ? launch_bits<X_BF16>(a, c.bits, c.group, s) : launch_bits<X_F16>(a, c.bits, c.group, s);
}

}  // namespace gptq
