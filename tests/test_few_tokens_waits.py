"""The weights' gradient of few tokens fetches a step's rows one step ahead, and the wait at a step's end lets the
step's 8 stores be on their way.  Such a wait covers the fetches only where each of them goes out before the
first store, and where there are no fewer than 8 of these: read from the assembly that the compiler makes of it."""
import os
import re
import subprocess

import pytest

from spectral_correction_optimizer_amd import build

KERNEL = r"^(_ZN5scopt17few_tokens_kernelILi(\d+)E\S*):"


def steps(asm):
    """{64-token tiles: [(fetches before the first store, after it, whole-row stores) of each step]}: a step
    reaches from a barrier to the wait for all but 8."""
    found = {}
    for m in re.finditer(KERNEL, asm, re.M):
        body = asm[m.end():asm.index(".Lfunc_end", m.end())].split("\n")
        out, cur = [], None
        for line in body:
            line = line.split(";")[0].strip()
            op = line.partition(" ")[0]
            if op == "s_barrier":
                cur = [0, 0, 0]
            elif cur is None:
                continue
            elif op.startswith("buffer_load") and line.endswith(" lds"):
                cur[1 if cur[2] else 0] += 1
            elif op.startswith("global_store_dwordx4"):
                cur[2] += 1
            elif op == "s_waitcnt" and "vmcnt(8)" in line:
                out.append(tuple(cur))
                cur = None
        found[int(m[2])] = out
    return found


def test_the_check_sees_a_late_fetch():
    asm = "\n_ZN5scopt17few_tokens_kernelILi1EEEvX:\n s_barrier\n buffer_load_dwordx4 v1, s[0:3], 0 offen lds\n%s" \
          " s_waitcnt vmcnt(8) lgkmcnt(0)\n.Lfunc_end0:\n"
    store, fetch = " global_store_dwordx4 v[0:1], v[2:5], off\n", " buffer_load_dwordx4 v3, s[0:3], 0 offen lds\n"
    assert steps(asm % (fetch + 8 * store)) == {1: [(2, 0, 8)]}
    assert steps(asm % (store + fetch + 7 * store)) == {1: [(1, 1, 8)]}


def test_fetches_go_out_before_the_stores(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    out = tmp_path / "few_tokens.s"
    cmd = [build.HIPCC, "-x", "hip", "-S", "--cuda-device-only", os.path.join(build.CSRC, "few_tokens.hip"), "-o",
           str(out)] + build.COMMON
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    # two steps, one for each half of LDS; a 64 x 64 tile of 16-bit values is two fetches of 256 threads
    assert steps(out.read_text()) == {kt: [(2 * kt, 0, 8)] * 2 for kt in (1, 2)}
    # and the fetches are kept there by the source, whatever order the compiler likes
    text = open(os.path.join(build.CSRC, "few_tokens.hip")).read()
    after = text[text.index("issue(blk + 1, next);"):].split("\n")
    code = [x.strip() for x in after[1:] if x.strip() and not x.strip().startswith("//")]
    assert code[0].startswith("__builtin_amdgcn_sched_barrier(")
