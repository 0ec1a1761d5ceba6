"""The wide attention kernel over 4-bit rows in the generated code: its MFMAs that are
written as assembly have the wait states and the untouched accumulators of the 16-bit
kernel's, and nothing between the score MFMAs waits for scratch memory; the kernel
whose waves have keys of their own keeps everything in registers."""
import os
import re
import subprocess

import pytest

import tests.test_attention_accumulators as accumulators
import tests.test_attention_isa as isa
from paged_mqa_logits_indexer_amd import build as b

WIDE = [f"attention_kernelILi{dt}ELi{kind}ELi128ELb1E" for dt in range(2) for kind in range(3)]
OWN = [f"own_keys_kernelILi{dt}ELi{kind}E" for dt in range(2) for kind in range(3)]


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    out = os.path.join(tmp_path_factory.mktemp("isa"), "attention.s")
    src = os.path.join(b.CSRC, "attention_mxfp4_kernels.hip")
    subprocess.run([b._hipcc(), *b.COMPILE_FLAGS, "--cuda-device-only", "-S", src, "-o", out], check=True,
                   capture_output=True)
    with open(out) as f:
        return f.read()


@pytest.mark.parametrize("kernel", WIDE)
def test_wide(assembly, kernel):
    isa.test_accumulators_are_read_after_the_wait_states(assembly, kernel)
    isa.test_step_has_no_scratch_access(assembly, kernel)
    accumulators.test_accumulators_are_left_alone_until_the_wait_states(assembly, kernel)


@pytest.mark.parametrize("kernel", OWN)
def test_own_keys_has_no_scratch(assembly, kernel):
    at = assembly.index(kernel, assembly.index(".amdhsa_kernel"))
    size = re.search(r"\.amdhsa_private_segment_fixed_size (\d+)", assembly[assembly.index(".amdhsa_kernel", assembly.index(kernel)):])
    assert at > 0 and size.group(1) == "0"
