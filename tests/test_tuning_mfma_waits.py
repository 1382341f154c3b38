"""The tuning kernels' matrix products in the built library: the wait states between each product
and the first use of its result (tests/test_mfma_waits.py says how they are counted)."""
import os
import re
import subprocess

import pytest

from test_mfma_waits import LIB, OBJDUMP, code_objects, functions, short_waits

KERNELS = re.compile(r"grouped_tile_kernel|grouped_gemm_kernel|forward_gemm_kernel|back_gemm_kernel|head_sums_kernel")


def test_every_product_of_the_tuning_kernels(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("llvm-objdump is not installed")
    if not os.path.exists(LIB):
        import __graft_entry__
        __graft_entry__.build()
    kernels = products = 0
    for k, obj in enumerate(code_objects()):
        path = tmp_path / f"{k}.elf"
        path.write_bytes(obj)
        names = subprocess.run(["nm", str(path)], capture_output=True, text=True).stdout
        if not KERNELS.search(names):
            continue
        text = subprocess.run([OBJDUMP, "-d", "--symbolize-operands", "--no-show-raw-insn", "--no-leading-addr", str(path)],
                              capture_output=True, text=True, check=True).stdout
        for name, lines in functions(text):
            if KERNELS.search(name):
                kernels += 1
                products += sum(ln.startswith("v_mfma") for ln in lines)
                assert (bad := short_waits(lines)) == [], (name, bad[:3])
    assert kernels > 100 and products > 10000
