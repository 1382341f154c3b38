// Which kernels the tuning operators take, and how the losses cut the vocabulary: rules on sizes
// alone, host code.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace gptq {

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---- y = What x
// Rows per expert from which workspace for the 256 x 256 tiles is asked for.
constexpr int64_t FORWARD_ROWS = 160;
constexpr bool many_rows(int64_t n, int64_t E) { return ceil_div(n, E) > FORWARD_ROWS; }

// Whether they pay: a round of them (256 workgroups) takes 125 us at 4096 columns and 20 more to
// begin, a round of the 128 x 128 tiles (512 workgroups) 82 us and 30, and 60 however few.  An
// expert ends in half a tile on average.  Both measured, us, 256 / 128 tiles, int4 g128, rows x columns,
// tokens (experts): 4096 x 4096, 1024: 144 / 74, 4096: 160 / 175; 11008 x 4096, 1024: 146 / 144,
// 2048: 272 / 255, 2048 (4): 272 / 293, 4096 (16): 790 / 656, 8192 (16): 1059 / 1096; 8-bit 32000 x
// 4096, 256: 143 / 110, 512: 154 / 190; 4096 x 4096, 4096 tokens: g64 185 / 201, g32 198 / 261,
// int3 g128 159 / 175, 8-bit per row 153 / 174.
constexpr bool forward_pays(int64_t n, int64_t E, int64_t rows, int64_t d_col) {
    const int64_t used = E < n ? E : n, partly = used > 1 ? used : 0;
    const int64_t large = (n + partly * 127 + 255) / 256 * ceil_div(rows, 256);
    const int64_t small = (n + partly * 64 + 127) / 128 * ceil_div(rows, 128);
    const int64_t a = ceil_div(large, 256) * 125 + 20 * 4096 / (d_col > 0 ? d_col : 1), b = 30 + small * 82 / 512;
    return many_rows(n, E) && a < (b > 60 ? b : 60);
}

// Groups that the 256 x 256 tiles take per turn of four slabs (128 columns): 1, 2 or 4; 0: one scale
// per row, as a row of a single group has, however few its columns.  Their tables hold whole
// turns of groups, and one where there is one scale per row.
constexpr int forward_turn_groups(int64_t n_groups, int group) { return n_groups == 1 || group <= 0 ? 0 : 128 / group; }
constexpr int64_t forward_groups(int64_t n_groups, int group) {
    const int per = forward_turn_groups(n_groups, group);
    return per ? ceil_div(n_groups, per) * per : 1;
}

// Tiles of 16 x 16, or the LDS kernel's of 64 (up to 96 tokens per expert) or 128 tokens x 128
// rows, by what either takes at 4096 columns, in ns: a 16 x 16 tile 9 and 9 / 16 for each of its
// tokens; a tile of the LDS kernel 120 (128 tokens: 160) where there are many, and the call 37000
// (60000) however few.  Both measured, us, int4 g128, 16 x 16 / LDS: 4096 x 4096, 16 tokens: 12 / 37,
// 32: 14 / 38, 64: 24 / 39, 96: 33 / 39, 128: 43 / 60; 11008 x 4096, 32: 32 / 39, 48: 48 / 41, 128:
// 106 / 61; 4096 x 11008, 64: 50 / 97, 128: 94 / 146; 2048 x 1024, 128: 11 / 23; 131072 x 4096, 1: 81 /
// 104, 8: 114 / 107, 16: 158 / 107; 131072 x 2048 int3 per row, 8: 48 / 48, 16: 70 / 49; 32000 x 4096
// 8-bit, 16: 47 / 48, 24: 77 / 49; 64 experts of 2816 x 2048, 8 rows: 14 / 24, 256: 67 / 86, 512: 81 /
// 99, 1024: 130 / 103; 61 of 2047 x 1408 int3, 488: 33 / 45, 777: 43 / 46 (there the rule, which knows
// no columns, takes the LDS kernel); 16 of 11008 x 4096, 128: 155 / 155, 256: 239 / 182; 8 of 4096 x
// 4096, 128: 50 / 54, 256: 85 / 55.  Calls in a chain from Python, where none takes less than 10 to
// 12; replayed from a graph 4096 x 4096, 1 / 16 / 32 / 64 / 128 tokens: 4.8 / 7.5 / 12 / 21 / 39.
// gptq_quantized_linear, which has no experts, takes 5.1 / 8.7 / 12 / 16 / 23 for those and 32 / 62 / 121 for
// 256 / 512 / 1024 (here 64 / 66 / 68): for one expert of 4096 x 4096 int4 it is the better call from 64
// to 512 tokens.  At 11008 x 4096, 64 / 128 / 256: 40 / 62 / 92 (here 44 / 65 / 66); 32000 x 4096 8-bit, 16 /
// 128: 198 / 1395 (here 47 / 87).
constexpr int64_t likely_tiles(int64_t n, int64_t E, int per) { // of n rows spread over E experts
    if (E == 1) return ceil_div(n, per);
    const int64_t used = E < n ? E : n, t = n / per + used / 2;
    return t > used ? t : used;
}
constexpr bool small_tiles(int64_t n, int64_t E, int64_t d_row) {
    const bool many = n / E > 96;
    const int64_t tile = ceil_div(d_row, 16) * (9 * likely_tiles(n, E, 16) + 9 * n / 16);
    const int64_t lds = likely_tiles(n, E, many ? 128 : 64) * ceil_div(d_row, 128) * (many ? 160 : 120), least = many ? 60000 : 37000;
    return tile < (lds > least ? lds : least) && n / 16 + E < 65536;   // the tiles of a launch
}

// ---- dx = What^T dy, and the sums of the losses: tokens and columns of a tile, and how many tiles
// the device takes at once.  parts: 2 where sums want two fp16 parts of the weights.
// Both sides measured, us, 32 x 128 / 128 x 128 / 256 x 256, int4 g128, bfloat16 out, 4096 x 4096: 32
// rows 33 / 35 / 38, 64: 34 / 40 / 43, 128: 41.5 / 41.8 / 44, 200: 55 / 43 / 47, 512: 82 / 54 / 59, 1024:
// 119 / 75 / 76; 11008 x 4096, 2048: 530 / 255 / 216; 16 experts of 4096 x 5504, 2048: 348 / 277 / 280,
// 8192: 1082 / 643 / 698; 61 of 2047 x 1408, 777: 68 / 90 / 133; fp32 out, 4096 x 4096, 512: 109 / 64.
struct SumTile { int bm, bn, places; };
constexpr SumTile sum_tile(int64_t each, int parts, int bits) {
    return each > 1024 && parts == 1 ? SumTile{256, 256, 256}
         : each > 96 ? SumTile{128, 128, parts == 1 || bits != 8 ? 512 : 256} : SumTile{32, 128, 512};
}

// Shares of the weight rows among workgroups: one for every place there is for a tile, none below
// 256 rows, and MOST_SUMS bytes of sums at most.
constexpr int64_t MOST_SUMS = (int64_t)64 << 20;
constexpr int64_t shares_of(int64_t tiles, int64_t places, int64_t d_row, int64_t sums) {
    int64_t s = places / tiles;
    if (s > ceil_div(d_row, 256)) s = ceil_div(d_row, 256);
    while (s > 1 && s * sums > MOST_SUMS) --s;
    return s < 1 ? 1 : s;
}

// ---- losses
constexpr int SPAN = 8192;                                      // most words of a span
constexpr int64_t CHUNK = 4096;                                 // tokens taken at a time
constexpr int64_t ROUND = (int64_t)1 << 25;                     // most logits of a round
constexpr int MOST_SPANS = 1024;                                // of a round

struct HeadPlan {
    int64_t nc;                                                 // tokens at a time
    int spans; int64_t span;                                    // span: words, a multiple of 64
    int R;                                                      // spans per round
};

// The losses' tile: their two-part sums have two-part exp(z - m) as well, for which 3- and 4-bit
// codes leave room for 256 columns.
constexpr SumTile head_tile(int64_t nc, int parts, int bits) {
    return nc > 96 && parts == 2 ? (bits != 8 ? SumTile{128, 256, 256} : SumTile{128, 128, 256}) : sum_tile(nc, parts, bits);
}

// Spans: with few tiles, as many as fill the device once, twice, .. with each span's tiles in a
// round of its own, of 512 to 8192 words; else of 8192 words, one after the other.  A round has
// at most ROUND logits.  parts 0: no gradient.
inline HeadPlan head_plan(int64_t nc, int64_t d, int64_t vocab, int parts, int bits) {
    HeadPlan p;
    p.nc = nc;
    int64_t spans = ceil_div(vocab, SPAN), R = spans;
    if (parts) {
        const SumTile t = head_tile(nc, parts, bits);
        const int64_t tiles = ceil_div(nc, t.bm) * ceil_div(d, t.bn);
        if (2 * tiles <= t.places) {
            int64_t times = 1;
            while (times * t.places / tiles < spans) ++times;
            spans = times * t.places / tiles;
            const int64_t most = ceil_div(vocab, 512);
            if (spans > most) spans = most;
            if (spans > MOST_SPANS && vocab <= SPAN * (int64_t)MOST_SPANS) spans = MOST_SPANS;
            R = spans;
        } else {
            R = 1;
        }
    }
    p.span = ceil_div(ceil_div(vocab, spans), 64) * 64;
    p.spans = (int)ceil_div(vocab, p.span);
    const int64_t fit = ROUND / (nc * p.span);
    if (R > p.spans) R = p.spans;
    if (R > MOST_SPANS) R = MOST_SPANS;
    if (R > fit) R = fit;
    if (R < 1) R = 1;
    p.R = (int)ceil_div(p.spans, ceil_div(p.spans, R));         // the same number in each round
    return p;
}

// The most logits of a round and the most sums (tokens x spans of a round) of any batch up to n
// tokens, of any dx type and bits: a larger batch takes fewer spans per round, and a workspace
// made for the largest has to do for every smaller one.  Batches of one number of 32-token tiles
// have the same spans; the smallest of them the most per round.
struct HeadMost { int64_t words, rows; };
inline HeadMost head_most(int64_t n, int64_t d, int64_t vocab, bool grad) {
    const int64_t nc = n < CHUNK ? n : CHUNK;
    HeadMost most = {0, 0};
    for (int parts = grad ? 1 : 0; parts <= (grad ? 2 : 0); ++parts)
        for (int bits = 4; bits <= (parts == 2 ? 8 : 4); bits += 4)
            for (int64_t T = 1; T <= ceil_div(nc, 32); ++T) {
                const int64_t tokens = 32 * T < nc ? 32 * T : nc;
                const HeadPlan a = head_plan(32 * (T - 1) + 1, d, vocab, parts, bits);
                const int64_t cap = ROUND > tokens * a.span ? ROUND : tokens * a.span;
                const int64_t rows = tokens * a.R, words = rows * a.span < cap ? rows * a.span : cap;
                most.words = words > most.words ? words : most.words;
                most.rows = rows > most.rows ? rows : most.rows;
            }
    return most;
}

}  // namespace gptq
