"""The 16-bit kernels over selections in the generated code: what only selections over
4-bit rows have, the count of the tiles of a list that hold a key, costs them nothing."""
import re

import pytest

from tests.test_attention_isa import assembly  # noqa: F401

SPARSE = [f"attention_kernelILi{dt}ELi2ELi{pairs}E" for dt in range(2) for pairs in (16, 32, 64, 128)]
# of the argument block: row_lens, the workspace, and what stands behind prefix_pages
UNREAD = [(0x20, 0x28), (0x58, 0x60), (0x8C, 0x90)]


@pytest.mark.parametrize("kernel", SPARSE)
def test_counts_are_not_looked_for(assembly, kernel):  # noqa: F811
    at = assembly.index(":", assembly.index(kernel))
    code = assembly[at:assembly.index(".end_amdhsa_kernel", at)]
    loads = re.findall(r"s_load_dword(?:x(\d+))? s\S+, s\[0:1\], 0x([0-9a-f]+)", code)
    assert loads
    for words, offset in loads:
        first = int(offset, 16)
        last = first + 4 * int(words or 1)
        assert not any(first < end and begin < last for begin, end in UNREAD), (words, offset)
