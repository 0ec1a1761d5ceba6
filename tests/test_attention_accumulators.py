"""The wide attention kernel's accumulators in the generated code: between an
MFMA that is written as assembly, whose duration the compiler does not know, and
the wait states behind it, nothing but further such MFMAs touches an accumulation
register -- no move, no arithmetic, no store from it and no load into it."""
import os
import re
import subprocess

import pytest

from paged_mqa_logits_indexer_amd import build as b

WIDE = [f"attention_kernelILi{dt}ELi{kind}ELi128E" for dt in range(2) for kind in range(3)]
ACCUMULATOR = re.compile(r"(?<![\w.])a(\[\d|\d)")


def touched(lines):
    """Lines with an accumulation register behind such an MFMA, up to the wait
    states; and how many of these MFMAs there are."""
    running, mfmas, found = False, 0, []
    for ln in lines:
        ln = ln.split(";")[0].strip()
        if ln.startswith("v_mfma") and ACCUMULATOR.search(ln.split(",")[0]):
            running, mfmas = True, mfmas + 1
        elif ln.startswith("s_nop 15"):
            running = False
        elif running and ACCUMULATOR.search(ln):
            found.append(ln)
    return found, mfmas


def test_touched_finds_every_kind():
    mfma = "v_mfma_f32_32x32x16_bf16 a[0:15], v[0:3], v[4:7], a[0:15]"
    for ln in ("v_accvgpr_read_b32 v1, a0", "v_accvgpr_write_b32 a3, v1", "ds_write_b128 v1, a[0:3] offset:16",
               "global_store_dwordx4 v[0:1], a[4:7], off", "v_mul_f32_e32 v0, v1, a7", "ds_read_b128 a[0:3], v1"):
        assert touched([mfma, ln])[0] == [ln]
        assert touched([mfma, "s_nop 15", ln])[0] == []
        assert touched([mfma, "v_mfma_f32_32x32x16_bf16 v[0:15], v[0:3], v[4:7], v[0:15]", ln])[0] == [ln]
    assert touched([mfma, "v_add_f32_e32 v0, v1, v2", "s_add_i32 s0, s1, s2", mfma]) == ([], 2)


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    out = os.path.join(tmp_path_factory.mktemp("isa"), "attention.s")
    src = os.path.join(b.CSRC, "attention_kernels.hip")
    subprocess.run([b._hipcc(), *b.COMPILE_FLAGS, "--cuda-device-only", "-S", src, "-o", out], check=True,
                   capture_output=True)
    with open(out) as f:
        return f.read()


@pytest.mark.parametrize("kernel", WIDE)
def test_accumulators_are_left_alone_until_the_wait_states(assembly, kernel):
    at = assembly.index(":", assembly.index(kernel))
    found, mfmas = touched(assembly[at:assembly.index(".end_amdhsa_kernel", at)].split("\n"))
    assert mfmas and not found, found[:5]
