"""The tuning operators' rules on sizes (csrc/tuning_rules.h), compiled for the host: where the
kernels change, that the losses' plan covers the vocabulary within its limits, and that a
workspace of a batch holds every smaller batch's rounds."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include "tuning_rules.h"
#include <cstdio>
#include <initializer_list>
using namespace gptq;
static int bad = 0;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); ++bad; } } while (0)
int main() {
    // both sides of the measured changes
    CHECK(!forward_pays(1024, 1, 4096, 4096) && forward_pays(4096, 1, 4096, 4096));
    CHECK(!forward_pays(2048, 1, 11008, 4096) && !forward_pays(4096, 16, 11008, 4096) && forward_pays(8192, 16, 11008, 4096));
    CHECK(!forward_pays(256, 1, 32000, 4096) && forward_pays(512, 1, 32000, 4096) && !forward_pays(160, 1, 1 << 20, 4096));
    CHECK(forward_pays(2048, 4, 11008, 4096) && !forward_pays(1024, 1, 11008, 4096));
    CHECK(forward_pays(4096, 1, 8192, 4096) && forward_pays(4096, 1, 8192, 2048) && !forward_pays(301, 1, 50021, 2048));
    // what the tests of the large tiles mean to take
    for (int c : {4096, 4032, 4000, 4128, 4224, 3904, 4112}) CHECK(forward_pays(4090, 1, 4083, c));
    for (int c : {288, 320, 384}) CHECK(forward_pays(17001, 1, 17000, c));
    CHECK(forward_pays(16000, 5, 4000, 2048));
    CHECK(head_plan(4096, 2048, 16384, 1, 8).R * head_plan(4096, 2048, 16384, 1, 8).span == 8192 && forward_pays(4096, 1, 8192, 2048));
    CHECK(small_tiles(1, 1, 131072) && !small_tiles(16, 1, 131072) && small_tiles(16, 1, 32000) && !small_tiles(24, 1, 32000));
    CHECK(small_tiles(128, 1, 4096) && small_tiles(32, 1, 11008) && !small_tiles(48, 1, 11008) && !small_tiles(128, 1, 11008));
    CHECK(small_tiles(8, 64, 2816) && small_tiles(512, 64, 2816) && !small_tiles(1024, 64, 2816) && small_tiles(488, 61, 2047));
    CHECK(small_tiles(128, 16, 11008) && !small_tiles(256, 16, 11008) && !small_tiles(256, 8, 4096));
    CHECK(!small_tiles((int64_t)1 << 22, 1, 1) && !small_tiles((int64_t)1 << 20, 4096, 16));
    // what the tests of the LDS kernel mean to take
    for (int n : {40, 64, 65, 96, 97, 130, 300}) CHECK(!small_tiles(n, 1, 17000));
    CHECK(!small_tiles(700, 3, 17000 / 3) && !small_tiles(301, 1, 20000));
    CHECK(sum_tile(1025, 1, 4).bm == 256 && sum_tile(1024, 1, 4).bm == 128 && sum_tile(1025, 2, 4).bm == 128);
    CHECK(sum_tile(97, 1, 8).bm == 128 && sum_tile(96, 1, 8).bm == 32);
    CHECK(shares_of(128, 256, 11008, 1 << 20) == 2 && shares_of(300, 256, 11008, 1) == 1 && shares_of(1, 512, 700, 1) == 3);
    CHECK(shares_of(1, 512, 1 << 20, (int64_t)40 << 20) == 1);
    // plans: whole spans of 64 words up to 8192, the last one not empty, rounds within their limits
    const int64_t words[] = {1, 63, 64, 65, 511, 1000, 8192, 8193, 32000, 50021, 131072, 262145, 1 << 22, 1 << 25};
    const int64_t widths[] = {8, 64, 1024, 2048, 4096, 16384, 131071};
    for (int64_t V : words)
        for (int64_t d : widths)
            for (int parts = 0; parts < 3; ++parts)
                for (int bits = 4; bits <= 8; bits += 4) {
                    HeadMost last = {0, 0};
                    for (int64_t n = 1; n <= CHUNK; n += n < 300 ? 1 : n < 1100 ? 37 : 211) {
                        const HeadPlan p = head_plan(n, d, V, parts, bits);
                        CHECK(p.span % 64 == 0 && p.span >= 64 && p.span <= SPAN && p.R >= 1 && p.R <= p.spans && p.R <= MOST_SPANS);
                        CHECK((p.spans - 1) * p.span < V && p.spans * p.span >= V);
                        CHECK(p.R == 1 || n * p.R * p.span <= ROUND);
                        const HeadMost m = head_most(n, d, V, parts != 0);
                        CHECK(m.words >= n * p.R * p.span && m.rows >= n * p.R);
                        CHECK(m.words >= last.words && m.rows >= last.rows);
                        last = m;
                        if (bad > 10) return 1;
                    }
                }
    return bad != 0;
}
"""


def test_rules(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    src = tmp_path / "rules.cpp"
    src.write_text(SOURCE)
    exe = tmp_path / "rules"
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", f"-I{ROOT}/post_weight_quantization_25_amd/csrc", str(src),
                    "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
