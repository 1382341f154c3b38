// RMS norm with the residual's addition, written as 8-bit rows (gptqs_rmsnorm_int8).
//
// With h = T(x + r), p = h w, rstd = 1 / sqrt(mean h^2 + eps) and am = max |p|, the
// normalised value is p rstd, the row's scale am rstd / 127, and the code
// rne(p rstd / scale) = rne(127 p / am): rstd cancels, so no sum enters a code.  For
// 16-bit h and w the product p is exact in fp32 and the code is decided exactly: the fp32
// estimate t = p (127 / am) is off by at most 3 roundings of 127, under 2^-14, so only
// where t lies within 2^-13 of a half-integer m + 1/2 is the decision taken from
// 254 |p| against (2 m + 1) am, both exact in 64 bits.  That makes the codes the same for
// every order of the sums and every launch shape.
//
// One pass: a row's x and residual are read once into registers (16 bytes per load), h
// and the codes are written from there.  Bound by HBM: 2 (x) + 2 (residual) + 2 (h) + 1
// (q) bytes per element of a 16-bit row; the squares' sum is kept in 64 bits (one
// conversion and one fp64 multiply-add per element, hidden behind the loads).  8192 x 4096
// bf16 with a residual: 52 us, 4.5 TB/s of 5.4 a copy reaches; one row of 4096: 3.8 us, a
// launch and one round trip.  With the 64-bit path's operands kept in registers beside the
// others (138 registers against 68) the same rows took 89 us.  333 rows of 11008 take 10.9 us,
// 5 times their bytes: 1024 threads of 70 registers are one workgroup per compute unit, so
// the rows come in two rounds.  fp32 weights or rows go through the two passes in 64 bits:
// 8192 x 4096 with a residual, replayed, 57 us (bf16 rows, fp32 weights) and 103 (fp32)
// against 43.
//
// Threads per row by width: a wave to 512, then 256 threads with one or two vectors of 8,
// 512 and 1024 with two, so that a row is read in one or two loads per thread.

#include "common.h"
#include "serving.h"

namespace gptq {

typedef unsigned long long u64;

template <gptq_dtype T>
GPTQ_DEV float round_to(float v) {
    if constexpr (T == GPTQ_F32) return v;
    else if constexpr (T == GPTQ_BF16) return (float)(__bf16)v;
    else return (float)(_Float16)v;
}

// Eight consecutive elements from idx on, of which the first m exist (0 for the others).
template <gptq_dtype T>
GPTQ_DEV void load8(const void* base, int64_t idx, int m, float (&v)[8]) {
    if (m >= 8) {
        if constexpr (T == GPTQ_F32) {
            float b[8];
            __builtin_memcpy(b, reinterpret_cast<const float*>(base) + idx, 32);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = b[e];
        } else {
            uint32_t b[4];
            __builtin_memcpy(b, reinterpret_cast<const uint16_t*>(base) + idx, 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint16_t lo = (uint16_t)(b[e] & 0xffffu), hi = (uint16_t)(b[e] >> 16);
                if constexpr (T == GPTQ_BF16) { v[2 * e] = bf16_bits_to_f32(lo); v[2 * e + 1] = bf16_bits_to_f32(hi); }
                else { v[2 * e] = f16_bits_to_f32(lo); v[2 * e + 1] = f16_bits_to_f32(hi); }
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < m ? load_as_f32<T>(base, idx + e) : 0.f;
    }
}

template <gptq_dtype T>
GPTQ_DEV void store8(void* base, int64_t idx, int m, const float (&v)[8]) {
    if constexpr (T == GPTQ_F32) {
        if (m >= 8) __builtin_memcpy(reinterpret_cast<float*>(base) + idx, v, 32);
        else
#pragma unroll
            for (int e = 0; e < 8; ++e) if (e < m) reinterpret_cast<float*>(base)[idx + e] = v[e];
    } else {
        uint16_t b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            b[e] = T == GPTQ_BF16 ? __builtin_bit_cast(uint16_t, (__bf16)v[e]) : __builtin_bit_cast(uint16_t, (_Float16)v[e]);
        if (m >= 8) __builtin_memcpy(reinterpret_cast<uint16_t*>(base) + idx, b, 16);
        else
#pragma unroll
            for (int e = 0; e < 8; ++e) if (e < m) reinterpret_cast<uint16_t*>(base)[idx + e] = b[e];
    }
}

GPTQ_DEV void store_codes(int8_t* q, int64_t idx, int m, const int (&k)[8]) {
    int8_t b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = (int8_t)k[e];
    if (m >= 8) __builtin_memcpy(q + idx, b, 8);
    else
#pragma unroll
        for (int e = 0; e < 8; ++e) if (e < m) q[idx + e] = b[e];
}

// Codes of eight products p in a row with maximum am (all exact, inv = 127 / am): see the
// head of the file.
GPTQ_DEV void codes_exact32(const float (&p)[8], float inv, float am, int (&k)[8]) {
    float near = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float t = p[e] * inv, r = rintf(t);
        near = fmaxf(near, fabsf(t - r));
        k[e] = (int)r;
    }
    if (near > 0.5f - 0x1p-13f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = fabsf(p[e] * inv), m = floorf(a);
            if (fabsf(a - m - 0.5f) < 0x1p-13f) {
                const double l = 254.0 * (double)fabsf(p[e]), r = (2.0 * (double)m + 1.0) * (double)am;
                const int up = (int)m + 1, c = l > r ? up : l < r ? (int)m : (((int)m & 1) ? up : (int)m);
                k[e] = p[e] < 0.f ? -c : c;
            }
        }
    }
}

GPTQ_DEV double wave_add(double v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
    return v;
}
GPTQ_DEV uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) { const uint32_t u = __shfl_xor(v, o); v = u > v ? u : v; }
    return v;
}
GPTQ_DEV u64 wave_max(u64 v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) { const u64 u = __shfl_xor(v, o); v = u > v ? u : v; }
    return v;
}

// |v|'s bits: their order is that of the magnitudes, with infinities and NaNs on top.
GPTQ_DEV uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
GPTQ_DEV u64 mag_bits(double v) { return (u64)__double_as_longlong(v) & 0x7fffffffffffffffull; }
constexpr u64 INF64 = 0x7ff0000000000000ull;

// A row's maximum product is usable in fp32 when neither it nor a product near it can have
// been rounded by underflow or overflow.
GPTQ_DEV bool plain_max(uint32_t b) { return b >= 0x0f800000u && b < 0x7b800000u; }   // 2^-96 .. 2^120

// A row by TPR threads in two passes over memory, products in 64 bits: rows too long for
// registers, fp32 rows or weights (their products are not exact in fp32), and 16-bit rows
// whose products are all tiny or zero, or of which one is huge or not finite.  FIRST: h is
// formed, and written where it is wanted; else it has been.  The second pass reads h where
// it was written (each thread its own elements), else x and the residual again.
template <gptq_dtype XT, gptq_dtype WT, int TPR, bool FIRST>
GPTQ_DEV void row_in_64(const NormArgs& a, int64_t row, int tid, double* s_sum, u64* s_max) {
    constexpr int WAVES = TPR / 64;
    double ss = 0.0;
    u64 mb = 0;
#pragma unroll 1
    for (int64_t c = 8 * (int64_t)tid; c < a.d; c += 8 * TPR) {
        const int m = c + 8 <= a.d ? 8 : (int)(a.d - c);
        float h[8], r[8], w[8];
        if (!FIRST && a.h) {
            load8<XT>(a.h, row * a.ldh + c, m, h);
        } else {
            load8<XT>(a.x, row * a.ldx + c, m, h);
            if (a.r) {
                load8<XT>(a.r, row * a.ldr + c, m, r);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = round_to<XT>(h[e] + r[e]);
            }
        }
        load8<WT>(a.w, c, m, w);
        if (FIRST && a.h) store8<XT>(a.h, row * a.ldh + c, m, h);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            ss = fma((double)h[e], (double)h[e], ss);
            const u64 b = mag_bits((double)h[e] * (double)w[e]);
            mb = b > mb ? b : mb;
        }
    }
    ss = wave_add(ss);
    mb = wave_max(mb);
    if constexpr (WAVES > 1) {
        __syncthreads();                                  // earlier uses of the arrays are read
        if ((tid & 63) == 0) { s_sum[tid >> 6] = ss; s_max[tid >> 6] = mb; }
        __syncthreads();
        ss = 0.0;
        for (int k = 0; k < WAVES; ++k) { ss += s_sum[k]; mb = s_max[k] > mb ? s_max[k] : mb; }
    }
    const double rstd = 1.0 / sqrt(ss / (double)a.d + (double)a.eps);
    const bool bad = mb >= INF64;
    const double am = __longlong_as_double((long long)mb);
    if (tid == 0) a.scale[row] = bad ? __uint_as_float(0x7fc00000u) : am == 0.0 ? 1.f : (float)(am * rstd / 127.0);
#pragma unroll 1
    for (int64_t c = 8 * (int64_t)tid; c < a.d; c += 8 * TPR) {
        const int m = c + 8 <= a.d ? 8 : (int)(a.d - c);
        float h[8], r[8], w[8], y[8];
        int k[8];
        if (a.h) {
            load8<XT>(a.h, row * a.ldh + c, m, h);
        } else {
            load8<XT>(a.x, row * a.ldx + c, m, h);
            if (a.r) {
                load8<XT>(a.r, row * a.ldr + c, m, r);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = round_to<XT>(h[e] + r[e]);
            }
        }
        load8<WT>(a.w, c, m, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double p = (double)h[e] * (double)w[e];
            k[e] = bad || am == 0.0 ? 0 : (int)rint(p * 127.0 / am);
            y[e] = (float)(p * rstd);
        }
        store_codes(a.q, row * a.ldq + c, m, k);
        if (a.y) store8<XT>(a.y, row * a.ldy + c, m, y);
    }
}

// 16-bit rows and weights.  TPR threads per row (a wave, or a workgroup), NV vectors of 8
// elements per thread; rows of up to 8 TPR NV elements.
template <gptq_dtype XT, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_kernel(NormArgs a) {
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;       // rows per workgroup
    constexpr int WAVES = TPR / 64;                       // waves per row
    __shared__ double s_sum[WAVES];
    __shared__ u64 s_max[WAVES];
    const int tid = threadIdx.x % TPR, wave = tid >> 6;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
    if (WAVES == 1 && row >= a.n) return;                 // whole waves: no barrier below

    float p[NV][8];                                       // first h, then the products
    double ss = 0.0;
    uint32_t mb = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t c = 8 * ((int64_t)tid + (int64_t)TPR * j);
        const int m = c + 8 <= a.d ? 8 : c < a.d ? (int)(a.d - c) : 0;
        load8<XT>(a.x, row * a.ldx + c, m, p[j]);
        if (a.r) {
            float r[8];
            load8<XT>(a.r, row * a.ldr + c, m, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) p[j][e] = round_to<XT>(p[j][e] + r[e]);
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t c = 8 * ((int64_t)tid + (int64_t)TPR * j);
        const int m = c + 8 <= a.d ? 8 : c < a.d ? (int)(a.d - c) : 0;
        float w[8];
        load8<XT>(a.w, c, m, w);
        if (a.h) store8<XT>(a.h, row * a.ldh + c, m, p[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            ss = fma((double)p[j][e], (double)p[j][e], ss);
            p[j][e] *= w[e];
            const uint32_t b = mag_bits(p[j][e]);
            mb = b > mb ? b : mb;
        }
    }
    ss = wave_add(ss);
    mb = wave_max(mb);
    if constexpr (WAVES > 1) {
        if ((threadIdx.x & 63) == 0) { s_sum[wave] = ss; s_max[wave] = mb; }
        __syncthreads();
        ss = 0.0;
#pragma unroll
        for (int k = 0; k < WAVES; ++k) {
            ss += s_sum[k];
            mb = (uint32_t)s_max[k] > mb ? (uint32_t)s_max[k] : mb;
        }
    }
    if (!plain_max(mb)) {                                 // row-uniform, rare
        row_in_64<XT, XT, TPR, false>(a, row, tid, s_sum, s_max);
        return;
    }
    const double rstd = 1.0 / sqrt(ss / (double)a.d + (double)a.eps);
    const float am = __uint_as_float(mb), inv = 127.f / am;
    // rstd = rm 2^re: with eps = 0 a row of subnormals, or near the type's largest value, has one
    // that is no normal fp32 number
    int re;
    const float rm = (float)frexp(rstd, &re);
    if (tid == 0) a.scale[row] = (float)((double)am * rstd / 127.0);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t c = 8 * ((int64_t)tid + (int64_t)TPR * j);
        const int m = c + 8 <= a.d ? 8 : c < a.d ? (int)(a.d - c) : 0;
        int k[8];
        codes_exact32(p[j], inv, am, k);
        store_codes(a.q, row * a.ldq + c, m, k);
        if (a.y) {
#pragma unroll
            for (int e = 0; e < 8; ++e) p[j][e] = ldexpf(p[j][e] * rm, re);
            store8<XT>(a.y, row * a.ldy + c, m, p[j]);
        }
    }
}

template <gptq_dtype XT, gptq_dtype WT, int TPR>
__global__ __launch_bounds__(TPR) void norm_64_kernel(NormArgs a) {
    __shared__ double s_sum[TPR / 64];
    __shared__ u64 s_max[TPR / 64];
    row_in_64<XT, WT, TPR, true>(a, blockIdx.x, threadIdx.x, s_sum, s_max);
}

template <gptq_dtype XT, gptq_dtype WT>
static gptq_status launch(const NormArgs& a, hipStream_t s) {
    const unsigned n = (unsigned)a.n;
    if constexpr (XT != GPTQ_F32 && WT == XT) {
        if (a.d <= 16384) {
            if (a.d <= 512) norm_kernel<XT, 64, 1><<<(unsigned)((a.n + 3) / 4), 256, 0, s>>>(a);
            else if (a.d <= 2048) norm_kernel<XT, 256, 1><<<n, 256, 0, s>>>(a);
            else if (a.d <= 4096) norm_kernel<XT, 256, 2><<<n, 256, 0, s>>>(a);
            else if (a.d <= 8192) norm_kernel<XT, 512, 2><<<n, 512, 0, s>>>(a);
            else norm_kernel<XT, 1024, 2><<<n, 1024, 0, s>>>(a);
            GPTQ_LAUNCH_CHECK();
            return GPTQ_OK;
        }
    }
    if (a.d <= 4096) norm_64_kernel<XT, WT, 256><<<n, 256, 0, s>>>(a);
    else norm_64_kernel<XT, WT, 1024><<<n, 1024, 0, s>>>(a);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

gptq_status norm_launch(const NormArgs& a, gptq_dtype xt, gptq_dtype wt, hipStream_t s) {
    switch (xt) {
        case GPTQ_F32: return launch<GPTQ_F32, GPTQ_F32>(a, s);
        case GPTQ_BF16:
            return wt == GPTQ_F32 ? launch<GPTQ_BF16, GPTQ_F32>(a, s) : launch<GPTQ_BF16, GPTQ_BF16>(a, s);
        case GPTQ_F16:
            return wt == GPTQ_F32 ? launch<GPTQ_F16, GPTQ_F32>(a, s) : launch<GPTQ_F16, GPTQ_F16>(a, s);
    }
    return GPTQ_ERR_UNSUPPORTED;
}

}  // namespace gptq
