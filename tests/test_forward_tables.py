"""The large forward tiles' tables of scales (csrc/tuning_rules.h), compiled for the host: a turn of
four slabs reads as many groups as the kernel's instantiation takes, and every one of them is
laid out, for rows of any number of columns from a single group on."""
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
    for (int group : {0, 32, 64, 128})
        for (int64_t d_col = group ? group : 8; d_col < 2000; d_col += group ? group : 8) {
            const int64_t n_groups = group ? d_col / group : 1, turns = (d_col + 127) / 128;
            const int per = forward_turn_groups(n_groups, group);
            const int64_t laid_out = forward_groups(n_groups, group);
            CHECK(per == 0 || per == 128 / group);
            CHECK(laid_out >= n_groups);
            CHECK(laid_out == (per ? turns * per : 1));        // what the turns read
            CHECK(per != 0 || n_groups == 1);                  // one set of tables serves every column
        }
    CHECK(forward_turn_groups(1, 32) == 0 && forward_turn_groups(1, 64) == 0 && forward_turn_groups(1, 128) == 0);
    CHECK(forward_turn_groups(2, 32) == 4 && forward_turn_groups(3, 64) == 2 && forward_turn_groups(2, 128) == 1);
    // what tests/test_gpu_forward_narrow.py means to take the large tiles
    CHECK(forward_pays(32768, 1, 20480, 64) && forward_pays(65536, 1, 20480, 32) && forward_pays(32768, 1, 20480, 96));
    CHECK(forward_pays(40000, 3, 20001, 64) && forward_pays(65536, 3, 24001, 32));
    return bad != 0;
}
"""


def test_tables_hold_what_the_turns_read(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    src = tmp_path / "tables.cpp"
    src.write_text(SOURCE)
    exe = tmp_path / "tables"
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", f"-I{ROOT}/post_weight_quantization_25_amd/csrc", str(src),
                    "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
