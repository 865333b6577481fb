"""Every instance of the tiled products is in the assembly that the check of their waits reads, and keeps its sums and
fragments in registers: none accesses scratch memory between its products.  One instance does elsewhere: the row
statistics of float16 planes in 256 x 256 tiles, a few values a tile, before its products and behind them."""
import os
import re
import subprocess

import pytest

from spectral_correction_optimizer_amd import build
from tests.test_product_waits import early_reads

# shapes x what becomes of the sums.  Each of three shapes: the logits' statistics, gradients (of bfloat16 and of
# float16 planes), both gradients' products stored or left in parts, and of live tokens the statistics (of both
# kinds of planes) and both gradients; the two shapes of few tokens: the statistics of both kinds.
INSTANCES = 3 * (1 + 2 + 4 + 2 + 2) + 2 * 2
SPILLS = r"TpShapeILi256ELi256E\w+ELb1ELb1ELi5ELb1EEE"


def spills(asm, name):
    """(accesses of scratch memory, those between the first and the last matrix instruction)"""
    start = asm.index("\n" + name + ":")
    ops = [x.split(";")[0].split() for x in asm[start:asm.index(".Lfunc_end", start)].split("\n")[1:]]
    ops = [x[0] for x in ops if x and not x[0].startswith(".")]
    at = [i for i, op in enumerate(ops) if op.startswith("scratch_")]
    products = [i for i, op in enumerate(ops) if op.startswith("v_mfma")]
    return len(at), sum(products[0] < i < products[-1] for i in at)


def test_the_check_sees_a_spill():
    asm = "\nk:\n scratch_store_dword off, v1, off\n v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]\n%s" \
          " v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]\n.Lfunc_end0:\n"
    assert spills(asm % "", "k") == (1, 0)
    assert spills(asm % " scratch_load_dword v1, off, off\n", "k") == (2, 1)


def test_every_instance(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    out = tmp_path / "tile_product.s"
    cmd = [build.HIPCC, "-x", "hip", "-S", "--cuda-device-only", os.path.join(build.CSRC, "tile_product.hip"), "-o",
           str(out)] + build.COMMON
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    asm = out.read_text()
    names = re.findall(r"^\s*\.amdhsa_kernel (_ZN5scopt19tile_product_kernel\S+)", asm, re.M)
    assert len(names) == len(set(names)) == INSTANCES
    found = early_reads(asm)
    assert set(found) == set(names) and not {k: v[:3] for k, v in found.items() if v}
    for name in names:
        every, inside = spills(asm, name)
        assert inside == 0, name
        assert every == 0 or re.search(SPILLS, name), name
