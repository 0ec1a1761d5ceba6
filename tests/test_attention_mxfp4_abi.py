"""Refusals of the attention over 4-bit rows, on the host: those of the 16-bit calls,
argument by argument, and the binding's checks of the packed cache."""
import pytest
import torch

import paged_mqa_logits_indexer_amd as pmqa
import tests.test_attention_abi as base
import tests.test_attention_limits as limits
from tests.test_attention_abi import IDX_EINVAL, A

NAMES = ("paged_attention", "shared_prefix_attention", "sparse_attention")


class FourBit:
    """The library with the _mxfp4 calls under the names of the 16-bit ones."""

    def __init__(self, lib):
        self.lib = lib

    def __getattr__(self, name):
        return getattr(self.lib, name + "_mxfp4" if name in NAMES else name)


@pytest.fixture(scope="module")
def four():
    return FourBit(pmqa.load_library())


def cases():
    marks = {m.args[0]: m.args[1] for m in base.test_attention_rejects.pytestmark}
    return [(name, kw, status) for name in marks["name"] for kw, status in marks["kw,status"]]


@pytest.mark.parametrize("name,kw,status", cases())
def test_rejects(four, name, kw, status):
    assert base.attend(four, name, **kw) == status


def test_rejects_by_kind(four):
    base.test_attention_rejects_by_kind(four)


@pytest.mark.parametrize("name", NAMES)
def test_limits(four, name):
    limits.test_scale_and_softcap_limits(four, name)


def test_failing_calls_disarm_the_timing_events(four):
    for call in (lambda: base.attend(four, "paged_attention", q=None),
                 lambda: base.attend(four, "shared_prefix_attention", prefix=0),
                 lambda: base.attend(four, "sparse_attention", k=0)):
        assert four.indexer_time_next_call(A, A) == 0
        assert call() == IDX_EINVAL


def test_binding_checks_before_the_library():
    cpu = torch.zeros(2, 16, 576, dtype=torch.bfloat16)
    pages = torch.zeros(3, 64, 400, dtype=torch.uint8)
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        pmqa.paged_attention_mxfp4(cpu, pages, i32.view(2, 1), i32, 1, 0.1, cpu[:, :, :512])
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        pmqa.sparse_attention_mxfp4(cpu.float(), pages, i32.view(2, 1), i32.view(2, 1), 1, 0.1, cpu)
    with pytest.raises(ValueError, match="GPU"):
        pmqa.latent_append_mxfp4(cpu[0], i32, i32, torch.zeros(4, 64), pages)
