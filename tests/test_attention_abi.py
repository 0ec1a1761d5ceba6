"""Refusals of the cache appends and of the latent-cache attention, on the host:
every bad argument returns its documented status before anything is launched
(no GPU is touched), and the workspace queries and shape checks of the binding
hold without one."""
import ctypes

import pytest
import torch

import paged_mqa_logits_indexer_amd as pmqa

IDX_OK, IDX_EINVAL, IDX_EUNSUPPORTED, IDX_EALIGN, IDX_ELAUNCH, IDX_EWORKSPACE = range(6)
BF16, FP16, FP32 = 0, 1, 2

# Fake but aligned device addresses: every call below fails its checks before
# any of them could be dereferenced or anything launched.
A = 0x10000


@pytest.fixture(scope="module")
def lib():
    return pmqa.load_library()


def append(lib, name, **kw):
    a = dict(rows=A, stride=576, dtype=BF16, pos=A, slots=A, rope=A, max_pos=100, inter=0, tokens=4, pages=8, cache=A,
             sc=A, stream=None)
    a.update(kw)
    tail = (a["sc"], a["stream"]) if name == "index_k_append" else (a["stream"],)
    return getattr(lib, name)(a["rows"], a["stride"], a["dtype"], a["pos"], a["slots"], a["rope"], a["max_pos"],
                              a["inter"], a["tokens"], a["pages"], a["cache"], *tail)


@pytest.mark.parametrize("name", ["index_k_append", "index_k_append_mxfp4", "latent_append"])
@pytest.mark.parametrize("kw,status", [
    (dict(rows=None), IDX_EINVAL), (dict(pos=None), IDX_EINVAL), (dict(slots=None), IDX_EINVAL),
    (dict(rope=None), IDX_EINVAL), (dict(cache=None), IDX_EINVAL), (dict(tokens=0), IDX_EINVAL),
    (dict(tokens=-1), IDX_EINVAL), (dict(pages=0), IDX_EINVAL), (dict(max_pos=0), IDX_EINVAL),
    (dict(stride=120), IDX_EINVAL), (dict(stride=-576), IDX_EINVAL),
    (dict(dtype=3), IDX_EUNSUPPORTED), (dict(dtype=-1), IDX_EUNSUPPORTED),
    (dict(tokens=(1 << 24) + 1), IDX_EUNSUPPORTED), (dict(pages=1 << 25), IDX_EUNSUPPORTED),
    (dict(stride=1 << 62), IDX_EUNSUPPORTED),
    (dict(rows=A + 8), IDX_EALIGN), (dict(stride=580), IDX_EALIGN), (dict(pos=A + 2), IDX_EALIGN),
    (dict(slots=A + 1), IDX_EALIGN), (dict(rope=A + 4), IDX_EALIGN), (dict(cache=A + 4), IDX_EALIGN),
])
def test_append_rejects(lib, name, kw, status):
    assert append(lib, name, **kw) == status


def test_append_rejects_by_kind(lib):
    assert append(lib, "index_k_append", sc=None) == IDX_EINVAL
    assert append(lib, "index_k_append", sc=A + 2) == IDX_EALIGN
    assert append(lib, "index_k_append", stride=127) == IDX_EINVAL
    assert append(lib, "latent_append", stride=568) == IDX_EINVAL
    assert append(lib, "latent_append", dtype=FP32) == IDX_EUNSUPPORTED
    # a multiple of 4 floats is enough for float32 rows: refused for the cache instead
    assert append(lib, "index_k_append", dtype=FP32, stride=132, cache=A + 4) == IDX_EALIGN
    assert append(lib, "index_k_append", dtype=FP32, stride=130) == IDX_EALIGN


def attend(lib, name, **kw):
    a = dict(q=A, cache=A, dtype=BF16, bt=A, lens=A, starts=None, idx=A, k=64, cu=None, rows=8, heads=16, requests=4,
             next_n=2, prefix=1, pages=100, max_pages=10, scale=0.1, softcap=0.0, slopes=None, pos=None, out=A,
             lse=None, ws=A, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    shape = (a["rows"], a["heads"], a["requests"], a["next_n"])
    tail = (a["pages"], a["max_pages"], a["scale"], a["softcap"], a["slopes"], a["pos"], a["out"], a["lse"], a["ws"],
            a["ws_bytes"], a["stream"])
    head = (a["q"], a["cache"], a["dtype"], a["bt"])
    if name == "paged_attention":
        return lib.paged_attention(*head, a["lens"], a["starts"], a["cu"], *shape, *tail)
    if name == "shared_prefix_attention":
        return lib.shared_prefix_attention(*head, a["lens"], a["starts"], *shape, a["prefix"], *tail)
    return lib.sparse_attention(*head, a["idx"], a["k"], a["cu"], *shape, *tail)


@pytest.mark.parametrize("name", ["paged_attention", "shared_prefix_attention", "sparse_attention"])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), IDX_EINVAL), (dict(cache=None), IDX_EINVAL), (dict(bt=None), IDX_EINVAL),
    (dict(lens=None, idx=None), IDX_EINVAL), (dict(out=None), IDX_EINVAL), (dict(ws=None), IDX_EINVAL),
    (dict(rows=0), IDX_EINVAL), (dict(heads=0), IDX_EINVAL), (dict(requests=0), IDX_EINVAL),
    (dict(pages=0), IDX_EINVAL), (dict(max_pages=0), IDX_EINVAL), (dict(next_n=-1), IDX_EINVAL),
    (dict(next_n=0), IDX_EINVAL), (dict(next_n=3), IDX_EINVAL), (dict(rows=7), IDX_EINVAL),
    (dict(next_n=1 << 30, requests=4, rows=8), IDX_EINVAL),
    (dict(scale=float("nan")), IDX_EINVAL), (dict(scale=float("inf")), IDX_EINVAL),
    (dict(softcap=-1.0), IDX_EINVAL), (dict(softcap=float("inf")), IDX_EINVAL),
    (dict(softcap=float("nan")), IDX_EINVAL), (dict(scale=1e10, softcap=1e-30), IDX_EINVAL),
    (dict(dtype=FP32), IDX_EUNSUPPORTED), (dict(dtype=7), IDX_EUNSUPPORTED), (dict(heads=129), IDX_EUNSUPPORTED),
    (dict(rows=65536, requests=4096, next_n=16), IDX_EUNSUPPORTED),
    (dict(rows=8194, requests=4097), IDX_EUNSUPPORTED), (dict(pages=1 << 25), IDX_EUNSUPPORTED),
    (dict(max_pages=(1 << 20) + 1), IDX_EUNSUPPORTED),
    (dict(rows=8192, requests=4096, max_pages=1 << 20), IDX_EUNSUPPORTED),
    (dict(q=A + 8), IDX_EALIGN), (dict(cache=A + 8), IDX_EALIGN), (dict(bt=A + 2), IDX_EALIGN),
    (dict(lens=A + 2, idx=A + 2), IDX_EALIGN), (dict(out=A + 8), IDX_EALIGN), (dict(lse=A + 2), IDX_EALIGN),
    (dict(ws=A + 128), IDX_EALIGN), (dict(slopes=A + 2, pos=A), IDX_EALIGN), (dict(pos=A + 2), IDX_EALIGN),
    (dict(ws_bytes=0), IDX_EWORKSPACE),
])
def test_attention_rejects(lib, name, kw, status):
    assert attend(lib, name, **kw) == status


def test_attention_rejects_by_kind(lib):
    for name in ("paged_attention", "sparse_attention"):
        assert attend(lib, name, cu=A) == IDX_EINVAL               # next_n and cu_q
        assert attend(lib, name, cu=A + 2, next_n=0) == IDX_EALIGN
        assert attend(lib, name, ws_bytes=lib.attention_workspace_bytes(8, 16, 4) - 1) == IDX_EWORKSPACE
    for name in ("paged_attention", "shared_prefix_attention"):
        assert attend(lib, name, starts=A + 2) == IDX_EALIGN
    assert attend(lib, "shared_prefix_attention", prefix=0) == IDX_EINVAL
    assert attend(lib, "shared_prefix_attention", prefix=11) == IDX_EINVAL
    assert attend(lib, "shared_prefix_attention",
                  ws_bytes=lib.shared_prefix_workspace_bytes(8, 16, 4) - 1) == IDX_EWORKSPACE
    assert attend(lib, "sparse_attention", k=0) == IDX_EINVAL
    assert attend(lib, "sparse_attention", k=8193) == IDX_EINVAL
    assert attend(lib, "sparse_attention", slopes=A) == IDX_EINVAL  # no positions to count from


def test_failing_calls_disarm_the_timing_events(lib):
    for call in (lambda: append(lib, "index_k_append", sc=None), lambda: append(lib, "latent_append", rows=None),
                 lambda: attend(lib, "paged_attention", q=None),
                 lambda: attend(lib, "shared_prefix_attention", prefix=0),
                 lambda: attend(lib, "sparse_attention", k=0)):
        assert lib.indexer_time_next_call(A, A) == IDX_OK
        assert call() == IDX_EINVAL


def test_workspace_queries(lib):
    for query in (pmqa.attention_workspace_bytes, pmqa.shared_prefix_workspace_bytes):
        assert query(0, 16, 1) == query(1, 0, 1) == query(1, 16, 0) == 0
        assert query(8, 128, 8) > 0
    # a fixed number of pieces, whatever the rows
    assert pmqa.attention_workspace_bytes(65535, 128, 100) == pmqa.attention_workspace_bytes(800, 128, 100)


def test_binding_checks_before_the_library():
    cpu = torch.zeros(2, 16, 576, dtype=torch.bfloat16)
    pages = torch.zeros(3, 64, 576, dtype=torch.bfloat16)
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        pmqa.paged_attention(cpu, pages, i32.view(2, 1), i32, 1, 0.1, cpu[:, :, :512])
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        pmqa.sparse_attention(cpu.float(), pages, i32.view(2, 1), i32.view(2, 1), 1, 0.1, cpu)
    with pytest.raises(ValueError, match="GPU"):
        pmqa.latent_append(cpu[0], i32, i32, torch.zeros(4, 64), pages)
    with pytest.raises(TypeError):
        pmqa.index_k_append(cpu[0].double(), i32, i32, torch.zeros(4, 64), torch.zeros(1, 64, 128), pages)


def test_argument_types_are_c_sized(lib):
    for name in ("paged_attention", "shared_prefix_attention", "sparse_attention"):
        types = getattr(lib, name).argtypes
        assert types.count(ctypes.c_float) == 2 and types[-2] is ctypes.c_size_t
