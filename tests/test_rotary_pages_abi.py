"""Refusals of the 4-bit latent append, of the rotations of queries and of the care
of pages, on the host: every bad argument returns its documented status before
anything is launched (no GPU is touched); the shape checks of the binding; and the
oracle of the pages against cases worked out by hand."""
import ctypes

import numpy as np
import pytest
import torch

import oracle as O
import paged_mqa_logits_indexer_amd as pmqa

IDX_OK, IDX_EINVAL, IDX_EUNSUPPORTED, IDX_EALIGN, IDX_ELAUNCH, IDX_EWORKSPACE = range(6)
BF16, FP16, FP32 = 0, 1, 2
# Fake but aligned device addresses, as every call below fails its checks.
A, B, C = 0x10000, 0x20000, 0x30000


@pytest.fixture(scope="module")
def lib():
    return pmqa.load_library()


def append(lib, **kw):
    a = dict(rows=A, stride=576, dtype=BF16, pos=A, slots=A, rope=A, max_pos=100, inter=0, tokens=4, pages=8, cache=A)
    a.update(kw)
    return lib.latent_append_mxfp4(*[a[k] for k in ("rows", "stride", "dtype", "pos", "slots", "rope", "max_pos",
                                                    "inter", "tokens", "pages", "cache")], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=None), IDX_EINVAL), (dict(pos=None), IDX_EINVAL), (dict(slots=None), IDX_EINVAL),
    (dict(rope=None), IDX_EINVAL), (dict(cache=None), IDX_EINVAL), (dict(tokens=0), IDX_EINVAL),
    (dict(pages=0), IDX_EINVAL), (dict(max_pos=0), IDX_EINVAL), (dict(stride=568), IDX_EINVAL),
    (dict(dtype=FP32), IDX_EUNSUPPORTED), (dict(dtype=-1), IDX_EUNSUPPORTED),
    (dict(tokens=(1 << 24) + 1), IDX_EUNSUPPORTED), (dict(pages=1 << 25), IDX_EUNSUPPORTED),
    (dict(stride=1 << 62), IDX_EUNSUPPORTED), (dict(rows=A + 8), IDX_EALIGN), (dict(stride=580), IDX_EALIGN),
    (dict(cache=A + 8), IDX_EALIGN), (dict(rope=A + 4), IDX_EALIGN), (dict(slots=A + 2), IDX_EALIGN),
])
def test_append_rejects(lib, kw, status):
    assert append(lib, **kw) == status


def compose(lib, **kw):
    a = dict(pos=A, axes=2, map=0, tokens=4, rope=A, max_pos=100, out=B)
    a.update(kw)
    return lib.axis_rotations(*[a[k] for k in ("pos", "axes", "map", "tokens", "rope", "max_pos", "out")], None)


ROTARY = [
    (dict(pos=None), IDX_EINVAL), (dict(rope=None), IDX_EINVAL), (dict(out=None), IDX_EINVAL),
    (dict(tokens=0), IDX_EINVAL), (dict(max_pos=0), IDX_EINVAL), (dict(axes=0), IDX_EINVAL),
    (dict(axes=5), IDX_EINVAL), (dict(axes=1, map=1 << 62), IDX_EINVAL), (dict(axes=3, map=3), IDX_EINVAL),
    (dict(axes=2, map=2 << 10), IDX_EINVAL), (dict(tokens=(1 << 24) + 1), IDX_EUNSUPPORTED),
    (dict(pos=A + 2), IDX_EALIGN), (dict(rope=A + 8), IDX_EALIGN), (dict(out=B + 8), IDX_EALIGN),
]


@pytest.mark.parametrize("kw,status", ROTARY)
def test_axis_rotations_rejects(lib, kw, status):
    assert compose(lib, **kw) == status


def turn(lib, **kw):
    a = dict(x=A, xt=512, xh=64, dtype=BF16, pos=A, axes=2, map=0, rope=A, max_pos=100, inter=0, tokens=4, heads=8,
             out=B, ot=512, oh=64)
    a.update(kw)
    return lib.rotate_queries(*[a[k] for k in ("x", "xt", "xh", "dtype", "pos", "axes", "map", "rope", "max_pos",
                                               "inter", "tokens", "heads", "out", "ot", "oh")], None)


@pytest.mark.parametrize("kw,status", ROTARY + [
    (dict(x=None), IDX_EINVAL), (dict(heads=0), IDX_EINVAL), (dict(heads=129), IDX_EUNSUPPORTED),
    (dict(dtype=FP32), IDX_EUNSUPPORTED), (dict(xt=-512), IDX_EINVAL), (dict(oh=-64), IDX_EINVAL),
    (dict(xt=1 << 61), IDX_EUNSUPPORTED), (dict(ot=1 << 61), IDX_EUNSUPPORTED),
    (dict(x=A + 8), IDX_EALIGN), (dict(xh=68), IDX_EALIGN), (dict(ot=516), IDX_EALIGN),
    # rows of the output that overlap: heads, tokens, one within the other
    (dict(oh=56), IDX_EINVAL), (dict(oh=0), IDX_EINVAL), (dict(ot=0), IDX_EINVAL), (dict(ot=448), IDX_EINVAL),
    (dict(ot=64, oh=128), IDX_EINVAL), (dict(ot=64, oh=192), IDX_EINVAL),
    # in place, but elsewhere
    (dict(out=A, oh=128, ot=1024), IDX_EINVAL), (dict(out=A, ot=1024), IDX_EINVAL),
])
def test_rotate_queries_rejects(lib, kw, status):
    assert turn(lib, **kw) == status


def codes(lib, **kw):
    a = dict(x=A, xt=4096, xh=128, dtype=BF16, pos=A, axes=2, map=0, rope=A, max_pos=100, inter=0, tokens=4, out=B)
    a.update(kw)
    return lib.rotate_index_queries(*[a[k] for k in ("x", "xt", "xh", "dtype", "pos", "axes", "map", "rope",
                                                     "max_pos", "inter", "tokens", "out")], None)


@pytest.mark.parametrize("kw,status", ROTARY + [
    (dict(x=None), IDX_EINVAL), (dict(dtype=3), IDX_EUNSUPPORTED), (dict(xt=-8), IDX_EINVAL),
    (dict(xt=4100), IDX_EALIGN), (dict(dtype=FP32, xt=4098), IDX_EALIGN), (dict(x=A + 8), IDX_EALIGN),
    (dict(xh=1 << 61), IDX_EUNSUPPORTED),
])
def test_rotate_index_queries_rejects(lib, kw, status):
    assert codes(lib, **kw) == status


def pool(lib, name, **kw):
    a = dict(table=A, lens=A, mask=A, requests=4, max_pages=8, refs=A, pages=32, new_table=B, new_lens=B, new_refs=B,
             src=C, dst=C, tokens=C, counts=C, ws=A, ws_bytes=1 << 20)
    a.update(kw)
    g = lambda *names: [a[k] for k in names]
    if name == "release_pages":
        return lib.release_pages(*g("table", "lens", "mask", "requests", "max_pages", "refs", "pages", "new_lens",
                                    "new_refs"), None)
    if name == "fork_pages":
        return lib.fork_pages(*g("table", "lens", "mask", "requests", "max_pages", "refs", "pages", "new_lens",
                                 "new_refs", "src", "dst", "tokens", "counts", "ws", "ws_bytes"), None)
    return lib.compact_pages(*g("table", "lens", "requests", "max_pages", "refs", "pages", "new_table", "new_refs",
                                "src", "dst", "counts", "ws", "ws_bytes"), None)


@pytest.mark.parametrize("name", ["release_pages", "fork_pages", "compact_pages"])
@pytest.mark.parametrize("kw,status", [
    (dict(table=None), IDX_EINVAL), (dict(lens=None), IDX_EINVAL), (dict(refs=None), IDX_EINVAL),
    (dict(new_refs=None), IDX_EINVAL), (dict(requests=0), IDX_EINVAL), (dict(max_pages=0), IDX_EINVAL),
    (dict(pages=0), IDX_EINVAL), (dict(requests=4097), IDX_EUNSUPPORTED), (dict(pages=1 << 25), IDX_EUNSUPPORTED),
    (dict(max_pages=(1 << 20) + 1), IDX_EUNSUPPORTED), (dict(requests=4096, max_pages=1 << 20), IDX_EUNSUPPORTED),
    (dict(table=A + 2), IDX_EALIGN), (dict(refs=A + 1), IDX_EALIGN), (dict(new_refs=B + 2), IDX_EALIGN),
])
def test_pool_rejects(lib, name, kw, status):
    assert pool(lib, name, **kw) == status


def test_pool_rejects_by_kind(lib):
    for name in ("release_pages", "fork_pages"):
        assert pool(lib, name, mask=None) == IDX_EINVAL
        assert pool(lib, name, new_lens=None) == IDX_EINVAL
        assert pool(lib, name, mask=A + 2) == IDX_EALIGN
    for name in ("fork_pages", "compact_pages"):
        for key in ("src", "dst", "counts", "ws"):
            assert pool(lib, name, **{key: None}) == IDX_EINVAL
        assert pool(lib, name, ws=A + 128) == IDX_EALIGN
        need = lib.pages_workspace_bytes(4, 32)
        assert pool(lib, name, ws_bytes=need - 1) == IDX_EWORKSPACE
    assert pool(lib, "fork_pages", tokens=None) == IDX_EINVAL
    assert pool(lib, "compact_pages", new_table=None) == IDX_EINVAL
    assert lib.pages_workspace_bytes(0, 4) == 0 and lib.pages_workspace_bytes(4, -1) == 0
    assert lib.pages_workspace_bytes(4096, 1) >= 4 * 4096 and lib.pages_workspace_bytes(1, 10 ** 6) >= 4 * 10 ** 6


def copy(lib, caches=(A, B), sizes=(400, 128), n_caches=None, pages=8, src=C, dst=C, tokens=None, count=None, n=4):
    c = (ctypes.c_void_p * len(caches))(*caches) if caches is not None else None
    s = (ctypes.c_int32 * len(sizes))(*sizes) if sizes is not None else None
    return lib.copy_pages(c, s, len(caches or ()) if n_caches is None else n_caches, pages, src, dst, tokens, count,
                          n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(caches=None, n_caches=2), IDX_EINVAL), (dict(sizes=None), IDX_EINVAL), (dict(src=None), IDX_EINVAL),
    (dict(dst=None), IDX_EINVAL), (dict(n_caches=0), IDX_EINVAL), (dict(pages=0), IDX_EINVAL), (dict(n=0), IDX_EINVAL),
    (dict(caches=(A, None)), IDX_EINVAL), (dict(sizes=(400, 0)), IDX_EINVAL),
    (dict(caches=(A,) * 1025, sizes=(4,) * 1025), IDX_EUNSUPPORTED), (dict(pages=1 << 25), IDX_EUNSUPPORTED),
    (dict(n=1 << 25), IDX_EUNSUPPORTED), (dict(sizes=(400, 16388)), IDX_EUNSUPPORTED),
    (dict(src=C + 2), IDX_EALIGN), (dict(tokens=C + 2), IDX_EALIGN), (dict(count=C + 1), IDX_EALIGN),
    (dict(caches=(A, B + 8)), IDX_EALIGN), (dict(sizes=(400, 66)), IDX_EALIGN),
])
def test_copy_rejects(lib, kw, status):
    assert copy(lib, **kw) == status


def test_axis_map():
    assert pmqa.axis_map([0] * 32) == 0
    assert pmqa.axis_map([3] + [0] * 30 + [2]) == 3 | 2 << 62
    for bad in ([0] * 31, [0] * 33, [4] + [0] * 31, [-1] + [0] * 31):
        with pytest.raises(ValueError):
            pmqa.axis_map(bad)


def test_binding_refuses_before_the_library():
    f = torch.float32
    with pytest.raises(ValueError):  # not on a GPU
        pmqa.rotate_queries(torch.zeros(2, 3, 64, dtype=torch.bfloat16), None, None, None)
    with pytest.raises(TypeError):
        pmqa.rotate_queries(torch.zeros(2, 3, 64, dtype=f), None, None, None)
    with pytest.raises(ValueError):
        pmqa.PageCaches([])
    with pytest.raises(ValueError):
        pmqa.PageCaches([torch.zeros(4, 64, 16)])


def test_oracle_fork_by_hand():
    # request 0 holds 130 tokens in pages 5, 2, 7; 1 and 3 are forked from it, 2 from 1, 4 is busy, 5 has a bad parent
    table = [[5, 2, 7], [9, 9, 9], [9, 9, 9], [9, 9, 9], [4, 9, 9], [9, 9, 9]]
    lens, parents = [130, 0, 0, 0, 64, 0], [-1, 0, 1, 0, 0, 6]
    refs = [0, 0, 1, 0, 1, 1, 0, 1]
    t, after, r, src, dst, tokens, counts = O.pages.fork(table, lens, parents, refs)
    assert t == [[5, 2, 7], [5, 2, 0], [9, 9, 9], [5, 2, 1], [4, 9, 9], [9, 9, 9]]
    assert after == [130, 130, 0, 130, 64, 0] and r == [1, 1, 3, 0, 1, 3, 0, 1]
    assert (src, dst, tokens) == ([-1, 7, -1, 7, -1, -1], [-1, 0, -1, 1, -1, -1], [0, 2, 0, 2, 0, 0])
    assert counts == [2, 0]
    # one free page: the first gets it, the second goes without
    t, after, r, src, dst, tokens, counts = O.pages.fork(table, lens, parents, [1, 1, 1, 0, 1, 1, 1, 1])
    assert after == [130, 130, 0, 0, 64, 0] and dst == [-1, 3, -1, -1, -1, -1] and counts == [1, 1]
    assert t[3] == [9, 9, 9] and r == [1, 1, 2, 1, 1, 2, 1, 1]


def test_oracle_release_and_compact_by_hand():
    table, lens = [[5, 2, 7], [5, 6, 1], [4, 8, 8]], [130, 65, 1]
    refs = [0, 0, 1, 0, 1, 2, 1, 1]
    after, r = O.pages.release(table, lens, [1, 0, 0], refs)
    assert after == [0, 65, 1] and r == [0, 0, 0, 0, 1, 1, 1, 0]
    t, r2, src, dst, counts = O.pages.compact(table, after, r)
    assert counts == [3, 3] and src[:3] == [4, 5, 6] and dst[:3] == [0, 1, 2] and src[3:] == [-1] * 5
    assert t == [[5, 2, 7], [1, 2, 1], [0, 8, 8]] and r2 == [1, 1, 1, 0, 0, 0, 0, 0]


def test_oracle_values_of_a_row():
    row = np.zeros((1, 400), np.uint8)
    row[0, 0] = 0x72      # dimensions 0, 1: codes 2 (1.0) and 7 (6.0)
    row[0, 17] = 0x9F     # dimensions 34, 35: -6 and -0.5
    row[0, 256], row[0, 257], row[0, 271] = 128, 125, 255
    row[0, 272:274] = np.frombuffer(np.uint16(0x3C00).tobytes(), np.uint8)
    v = O.latent.latent_mxfp4_values(row, "fp16")[0]
    assert (v[0], v[1], v[34], v[35], v[512]) == (2.0, 12.0, -1.5, -0.125, 1.0)
    assert np.isnan(v[480:512]).all() and (v[64:480] == 0).all()
    assert O.latent.latent_mxfp4_values(row, "bf16")[0, 512] == 2.0 ** -7
