"""Limits of the attention's scale and softcap, on the host: what float32 cannot
hold times log2(e) is refused before anything is launched."""
import pytest

import paged_mqa_logits_indexer_amd as pmqa
from tests.test_attention_abi import IDX_EALIGN, IDX_EINVAL, A, attend

LIMIT = 2.0 ** 127
ABOVE = LIMIT * (1 + 2.0 ** -23)  # the next float32


@pytest.fixture(scope="module")
def lib():
    return pmqa.load_library()


@pytest.mark.parametrize("name", ["paged_attention", "shared_prefix_attention", "sparse_attention"])
def test_scale_and_softcap_limits(lib, name):
    for bad in (dict(scale=ABOVE), dict(scale=-ABOVE), dict(scale=3.4e38), dict(softcap=ABOVE), dict(softcap=3.4e38),
                dict(scale=-float("inf"))):
        assert attend(lib, name, **bad) == IDX_EINVAL
    # at the limits the calls pass this check and fail a later one
    for good in (dict(scale=LIMIT), dict(scale=-LIMIT), dict(scale=0.0), dict(softcap=LIMIT)):
        assert attend(lib, name, q=A + 8, **good) == IDX_EALIGN
