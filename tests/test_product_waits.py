"""The tiled products' matrix instructions are inline assembly, which the compiler gives no wait states: in
the assembly that it makes of them, no sum leaves an accumulation register, and none is overwritten,
until the instruction that writes it is done.  (A matrix instruction of 8 passes needs 11 wait states
before its result is read; the waits behind the products are 20.)"""
import os
import re
import subprocess

import pytest

from spectral_correction_optimizer_amd import build

WAIT = 18


def early_reads(asm):
    """{kernel: accesses of an accumulation register within WAIT issue slots of the product that writes it}."""
    found = {}
    for name in re.findall(r"^(_ZN5scopt19tile_product_kernel\S+):", asm, re.M):
        start = asm.index("\n" + name + ":")
        written, slot, bad = {}, 0, []
        for line in asm[start:asm.index(".Lfunc_end", start)].split("\n")[1:]:
            line = line.split(";")[0].strip()
            if not line or line.startswith(".") or line.endswith(":"):
                continue
            op, _, args = line.partition(" ")
            slot += int(args) + 1 if op == "s_nop" else 1
            regs = [r for m in re.finditer(r"\ba(?:(\d+)\b|\[(\d+):(\d+)\])", args)
                    for r in (range(int(m[2]), int(m[3]) + 1) if m[2] else [int(m[1])])]
            if op.startswith("v_mfma"):
                written.update(dict.fromkeys(regs, slot))
            else:
                bad += [line for r in regs if slot - written.get(r, -WAIT) < WAIT]
        found[name] = bad
    return found


def test_the_check_sees_an_early_read():
    asm = "\n_ZN5scopt19tile_product_kernelX:\n v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]\n%s\n" \
          " v_accvgpr_read_b32 v9, a2\n.Lfunc_end0:\n"
    assert early_reads(asm % " s_nop 3") == {"_ZN5scopt19tile_product_kernelX": ["v_accvgpr_read_b32 v9, a2"]}
    assert early_reads(asm % " s_nop 15\n s_nop 3") == {"_ZN5scopt19tile_product_kernelX": []}


def test_products_wait_for_their_sums(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    out = tmp_path / "tile_product.s"
    cmd = [build.HIPCC, "-x", "hip", "-S", "--cuda-device-only", os.path.join(build.CSRC, "tile_product.hip"), "-o",
           str(out)] + build.COMMON
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    found = early_reads(out.read_text())
    assert len(found) >= 24  # three tile shapes, eight ways each
    assert not {k: v[:3] for k, v in found.items() if v}
