// Host-side launchers of the tuning operators and what their kernels share (internal to the
// library).
#pragma once
#include "gptq_tuning.h"
#include "serving.h"
#include "stored_tile.h"
#include "tuning_rules.h"

namespace gptq {

constexpr int TUNE_MAX_EXPERTS = 4096;
constexpr int TUNE_MAX_TOP = 1024;
constexpr int64_t TUNE_MAX_WIDTH = ((int64_t)1 << 17) - 1;      // columns (see gemm_fits)
constexpr int64_t TUNE_MAX_PITCH = (int64_t)1 << 23;            // elements between rows of 16-bit activations

// ---- rows of experts
struct Segment { int e; int64_t tok0, end; };                   // rows tok0 .. min(tok0 + per, end) - 1 of expert e

// Tile number `tile` of the segments' tiles of `per` rows, experts in order; false behind the
// last.  offsets == nullptr: one segment of n rows.  Offsets are taken clamped to 0 .. n and to
// never fall, so that segments never overlap whatever the buffer holds.  The whole wave calls
// it with one tile.
GPTQ_DEV bool segment_of(const int32_t* offsets, int E, int64_t n, int per, int tile, Segment& s) {
    if (offsets == nullptr) {
        s = Segment{0, (int64_t)tile * per, n};
        return s.tok0 < n;
    }
    const int lane = threadIdx.x & 63, most = (int)n;
    auto clamped = [&](int v) { return v < 0 ? 0 : v < most ? v : most; };
    int run = clamped(offsets[0]), base = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        int end = e0 + lane < E ? clamped(offsets[e0 + lane + 1]) : 0;
        end = end > run ? end : run;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(end, o);
            end = lane >= o && v > end ? v : end;
        }
        const int before = __shfl_up(end, 1), start = lane ? before : run;
        const int tiles = (end - start + per - 1) / per;
        int sum = tiles;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(sum, o);
            sum += lane >= o ? v : 0;
        }
        const uint64_t past = __ballot(base + sum > tile);
        if (past != 0) {                                         // wave-uniform
            const int l = __builtin_ctzll(past);
            s.e = e0 + l;
            s.tok0 = __shfl(start, l) + (int64_t)(tile - base - __shfl(sum - tiles, l)) * per;
            s.end = __shfl(end, l);
            return true;
        }
        base += __shfl(sum, 63);
        run = __shfl(end, 63);
    }
    return false;
}

// Most tiles that n rows of E experts have: every expert with a row may end in a part of one.
inline int64_t most_tiles(const int32_t* offsets, int64_t E, int64_t n, int per) {
    const int64_t used = offsets ? (E < n ? E : n) : 1;
    return (n + used * (per - 1)) / per;
}

// The layer of expert e.
GPTQ_DEV Stored expert_of(Stored L, int64_t d_row, int e) {
    L.codes += (int64_t)e * d_row * L.code_ld;
    L.scales += (int64_t)e * d_row * L.n_groups;
    L.zeros += (int64_t)e * d_row * L.n_groups;
    return L;
}

// One weight, S (u - z).  (A 3-bit code may lie in two bytes.)
GPTQ_DEV float weight_at(const Stored& L, int bits, int64_t r, int64_t c) {
    const uint8_t* src = L.codes + r * L.code_ld + (c * bits >> 3);
    const int bit = (int)(c * bits & 7);
    uint32_t u = src[0] >> bit;
    if (bit + bits > 8) u |= (uint32_t)src[1] << (8 - bit);
    const int64_t at = r * L.n_groups + (L.n_groups == 1 ? 0 : c >> L.gshift);
    return f16_bits_to_f32(L.scales[at]) * ((float)(u & ((1u << bits) - 1)) - f16_bits_to_f32(L.zeros[at]));
}

// Which of eight 16-bit elements from p on, the first m of which exist, are infinities or NaNs.
template <int X>
GPTQ_DEV uint32_t not_finite8(const uint16_t* p, int m) {
    float v[8];
    load_x8<X>(p, m, v);
    uint32_t found = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) found |= fabsf(v[i]) < INFINITY ? 0u : 1u << i;
    return found;
}

// ---- y[t] = What_e x[t] (grouped.hip)
struct GroupedArgs {
    Stored L; int64_t d_row;                                    // rows of each expert
    const uint16_t* x; int64_t ldx; int64_t n;
    const int32_t* offsets; int E;
    void* y; gptq_dtype yt; int64_t ldy;
    const int32_t* unless_zero;                                 // the kernel of stored_gemm.h: not nullptr: works only if not 0
};
// grouped_large: whether products of `rows` rows (of each expert) are for the large tiles.  Then
// grouped_prepare lays the activations and the scales of all E d_row rows out, once for products
// of several spans of the rows, and grouped_launch takes rows row0 .. row0 + a.d_row - 1 of
// all_rows (with experts: all).  ws: grouped_ws_bytes, which is 0 where they never are.
size_t grouped_ws_bytes(int64_t n, int64_t E, int64_t d_row, int64_t d_col, int group);
bool grouped_large(const GroupedArgs& a, int64_t rows);
gptq_status grouped_prepare(const GroupedArgs& a, gptq_dtype xt, int bits, int group, void* ws, hipStream_t s);
gptq_status grouped_launch(const GroupedArgs& a, gptq_dtype xt, int bits, int group, bool large, void* ws, int64_t all_rows,
                           int64_t row0, hipStream_t s);

// ---- dx[t] = What_e^T dy[t] (grouped_back.hip)
struct BackCall {
    Stored L; int64_t d_row; int bits;
    const void* dy; gptq_dtype dyt; int64_t ldy; int64_t n;
    const int32_t* offsets; int E;
    void* dx; gptq_dtype dxt;                                   // pitch d_col
    void* ws;
};
size_t back_ws_bytes(int64_t n, int64_t E, int64_t d_row, int64_t d_col, int group);
gptq_status back_launch(const BackCall& c, hipStream_t s);

// ---- losses at a stored head (head_loss.hip)
struct HeadCall {
    Stored L; int64_t vocab; int bits, group;
    const void* x; gptq_dtype xt; int64_t ldx; int64_t n;
    const int32_t* ids; int k;                                  // n x k
    const void* top; gptq_dtype topt;                           // n x k teacher's logits, or nullptr: one target each
    float temperature;
    const float* weights;
    float* loss;
    void* dx; gptq_dtype dxt;                                   // or nullptr
    void* ws;
};
size_t head_ws_bytes(int64_t n, int64_t d, int64_t vocab, int group, int k, bool grad);
gptq_status head_launch(const HeadCall& c, hipStream_t s);

inline size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace gptq
