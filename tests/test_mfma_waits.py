"""The serving kernels' matrix products in the built library: on every path from a product to
the first instruction that touches its result registers (other than the next product
adding to them) the wait states that the hardware needs have passed.  The compiler places
the waits; it counts them along one path only where several meet behind a branch, which
the sources answer with waits of their own, so each build is looked at here.

A product of n passes needs n + 4 wait states before its result is read or overwritten by a
vector, memory or LDS instruction or enters a product as A or B; an instruction is one
wait state, s_nop k is k + 1."""
import os
import re
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "post_weight_quantization_25_amd", "libgptq.so")
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
KERNELS = re.compile(r"int8_tile|int8_gemm|lora_shrink|lora_tile|lora_gemm|moe_")
PASSES = {"16x16x64_i8": 4, "16x16x32_bf16": 4, "16x16x32_f16": 4, "16x16x32_i8": 4}
STORES = ("global_store", "ds_write", "buffer_store", "scratch_store", "flat_store")


def code_objects():
    """The gfx950 code objects bundled into the library."""
    b, i, out = open(LIB, "rb").read(), 0, []
    while (i := b.find(b"__CLANG_OFFLOAD_BUNDLE__", i)) >= 0:
        n, p = struct.unpack_from("<Q", b, i + 24)[0], i + 32
        for _ in range(n):
            off, size, length = struct.unpack_from("<QQQ", b, p)
            if b"gfx950" in b[p + 24:p + 24 + length] and size:
                out.append(b[i + off:i + off + size])
            p += 24 + length
        i += 24
    return out


def functions(listing):
    """(name, lines) of each function of a listing; labels are lines that end with a colon."""
    name, lines = None, []
    for ln in listing.splitlines():
        if m := re.match(r"^(?:[0-9a-f]+ )?<(\S+)>:$", ln):
            if re.match(r"^L\d+$", m.group(1)):
                lines.append(m.group(1) + ":")
                continue
            if name:
                yield name, lines
            name, lines = m.group(1), []
        elif name and ln.startswith("\t"):
            lines.append(ln.split("//")[0].strip())
    if name:
        yield name, lines


def registers(text):
    out = set()
    for m in re.finditer(r"\bv\[(\d+):(\d+)\]|\bv(\d+)\b", text):
        out |= {int(m.group(3))} if m.group(3) else set(range(int(m.group(1)), int(m.group(2)) + 1))
    return out


def needed(op):
    for shape, passes in PASSES.items():
        if shape in op:
            return passes + 4
    raise AssertionError(f"a product this test does not know: {op}")


def short_waits(lines):
    """(product, instruction, wait states) of each result touched too soon."""
    at = {ln[:-1]: i for i, ln in enumerate(lines) if ln.endswith(":")}
    bad = []
    for start, ins in enumerate(lines):
        if not ins.startswith("v_mfma"):
            continue
        op, args = ins.split(None, 1)
        need, dst = needed(op), registers(args.split(",")[0])
        todo, seen = [(start + 1, 0)], {}
        while todo:
            i, w = todo.pop()
            while i < len(lines) and w < need:
                ln = lines[i]
                if ln.endswith(":"):
                    if seen.get(ln, need) <= w:
                        break
                    seen[ln] = w
                    i += 1
                    continue
                o, _, rest = ln.partition(" ")
                a = rest.split(",")
                if o.startswith("v_mfma"):
                    if registers(",".join(a[1:3])) & dst:
                        bad.append((ins, ln, w))
                        break
                    if registers(a[0]) & dst:                  # adds to the result: that product's own wait counts
                        break
                elif o == "s_nop":
                    w += int(rest)
                elif o in ("s_endpgm", "s_branch") or o.startswith("s_cbranch"):
                    if o != "s_endpgm":
                        todo.append((at[rest.strip()], w + 1))
                    if not o.startswith("s_cbranch"):
                        break
                elif not o.startswith("s_") and registers(rest) & dst:
                    bad.append((ins, ln, w))
                    break
                i, w = i + 1, w + 1
    return bad


def test_the_search_finds_a_short_wait():
    """A result read behind a branch after 5 states on one path and 8 on the other; with one
    more s_nop on the short path nothing is short."""
    head = ["v_mfma_f32_16x16x32_bf16 v[0:3], v[4:7], v[8:11], 0", "s_cbranch_execz L0", "s_nop 2", "v_mov_b32_e32 v9, v8", "L0:"]
    tail = ["v_add_u32_e32 v8, v7, v9", "s_nop 1", "s_nop 0", "v_add_f32_e32 v12, v3, v3", "s_endpgm"]
    assert [b[2] for b in short_waits(head + tail)] == [5]
    assert short_waits(head + ["s_nop 2"] + tail) == []
    assert short_waits(head[:1] + ["v_mfma_f32_16x16x32_bf16 v[12:15], v[0:3], v[8:11], 0"]) != []
    assert short_waits(head[:1] + ["v_mfma_f32_16x16x32_bf16 v[0:3], v[4:7], v[8:11], v[0:3]", "s_nop 7", "v_mov_b32_e32 v5, v0"]) == []
    assert short_waits(head[:1] + ["s_nop 6", "global_store_dword v20, v2, s[0:1]"]) != []


def test_every_product_of_the_serving_kernels(tmp_path):
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
    assert kernels > 200 and products > 10000
