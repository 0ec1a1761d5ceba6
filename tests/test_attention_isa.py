"""The attention kernel's MFMAs that are written as assembly, checked in the
generated code: the compiler does not know how long their results take, so no
instruction may read an accumulation register between such an MFMA and the
wait states that the source puts before its own reads."""
import os
import subprocess

import pytest

from paged_mqa_logits_indexer_amd import build as b

WIDE = [f"attention_kernelILi{dt}ELi{kind}ELi128E" for dt in range(2) for kind in range(3)]


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    out = os.path.join(tmp_path_factory.mktemp("isa"), "attention.s")
    src = os.path.join(b.CSRC, "attention_kernels.hip")
    subprocess.run([b._hipcc(), *b.COMPILE_FLAGS, "--cuda-device-only", "-S", src, "-o", out], check=True,
                   capture_output=True)
    with open(out) as f:
        return f.read()


@pytest.mark.parametrize("kernel", WIDE)
def test_accumulators_are_read_after_the_wait_states(assembly, kernel):
    at = assembly.index(":", assembly.index(kernel))
    lines = [ln.strip() for ln in assembly[at:assembly.index(".end_amdhsa_kernel", at)].split("\n")]
    running, mfmas, reads = False, 0, 0
    for ln in lines:
        if ln.startswith("v_mfma") and " a[" in ln.split(",")[0]:
            running, mfmas = True, mfmas + 1
        elif ln.startswith("s_nop 15"):
            running = False
        elif ln.startswith(("v_accvgpr_read", "v_accvgpr_mov")):
            reads += 1
            assert not running, f"{kernel}: {ln} right behind an MFMA"
    assert mfmas == 64 and reads >= 256  # two value products; rescale and output


@pytest.mark.parametrize("kernel", WIDE)
def test_step_has_no_scratch_access(assembly, kernel):
    """A reload between the score MFMAs would wait for every load in flight."""
    at = assembly.index(":", assembly.index(kernel))
    lines = [ln.strip() for ln in assembly[at:assembly.index(".end_amdhsa_kernel", at)].split("\n")]
    scores = [i for i, ln in enumerate(lines) if ln.startswith("v_mfma") and " v[" in ln.split(",")[0]]
    assert len(scores) == 36
    assert not [ln for ln in lines[scores[0]:scores[-1]] if ln.startswith("scratch_")]
