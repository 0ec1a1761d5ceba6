"""Attention over the latent cache against the root-mean-square allowance of
oracle/latent.py, which a weight of too few bits or a rescale left out passes
(shown on the host), and on the work lists that only large batches have: ragged
selections and shared prefixes of more pair tiles than one wave, and one
workgroup, scan at a time."""
import numpy as np
import pytest
import torch

import oracle as O
from tests.gpu_harness import DEV, announce
from tests.test_gpu_attention import LENGTHS, SCALE, WIDE, Batch, growing, selections

pytestmark = pytest.mark.gpu
L = O.latent
WIDTHS = pytest.mark.parametrize("width", [0, WIDE])
TYPES = pytest.mark.parametrize("dtype", ["bf16", "fp16"])


def check_rms(b, out, lse, softcap=0.0, slopes=None, positions=None, picked=None, rows=None):
    """Every given row of the batch, head by head."""
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    cache = b.cache.view(-1, 576)
    for r in range(len(b.ends)) if rows is None else rows:
        at = b.visible(r) if picked is None else picked[r]
        keys = cache[torch.from_numpy(b.slots(r, at))].double().numpy()
        pos = int(positions[r]) if positions is not None else int(b.ends[r]) - 1
        want, wl, allowed, lse_allowed = L.attend_row_rms(b.q[r].double().numpy(), keys, at, SCALE, softcap, slopes,
                                                          pos, b.dtype)
        if len(at) == 0:
            assert (out[r] == 0).all() and (lse[r] == -np.inf).all(), f"row {r} without keys"
            continue
        off = np.sqrt(((out[r] - want) ** 2).mean(1))
        assert (off <= allowed).all(), f"row {r} ({len(at)} keys): {(off / allowed).max():.2f} of the allowance"
        assert (np.abs(lse[r] - wl) <= lse_allowed).all(), f"row {r}: lse off by {np.abs(lse[r] - wl).max()}"


@WIDTHS
@TYPES
@pytest.mark.parametrize("q_scale", [0.5, 2.0])
@pytest.mark.parametrize("heads,next_n", [(1, 1), (16, 1), (32, 1), (24, 3), (64, 1), (128, 2)])
def test_decode(gpu, heads, next_n, q_scale, dtype, width):
    announce(f"paged_attention rms heads={heads} next_n={next_n} {dtype} q {q_scale}")
    ends = [n + j if n else 0 for n in LENGTHS + [2500] for j in range(next_n)]
    b = Batch(300 + heads, heads, [next_n] * (len(LENGTHS) + 1), ends, dtype=dtype, q_scale=q_scale, width=width)
    out, lse = b.run(gpu)
    check_rms(b, out, lse)


@WIDTHS
@TYPES
@pytest.mark.parametrize("heads", [16, 32, 64, 128])
def test_growing_scores(gpu, heads, dtype, width):
    announce(f"paged_attention rms growing heads={heads} {dtype}")
    b = Batch(337, heads, [1] * 5, [3000, 900, 400, 64, 640], dtype=dtype, q_scale=4.0, width=width)
    growing(b, 1)
    check_rms(b, *b.run(gpu))


@WIDTHS
@TYPES
@pytest.mark.parametrize("softcap,bias", [(20.0, False), (0.0, True), (30.0, True)])
def test_caps_windows_and_bias(gpu, softcap, bias, dtype, width):
    announce(f"paged_attention rms softcap={softcap} bias={bias} {dtype}")
    heads, rows, prefix = 16, [9, 30, 2], [0, 300, 700]
    pos = np.concatenate([np.arange(p, p + n) for n, p in zip(rows, prefix)])
    b = Batch(341, heads, rows, pos + 1, np.maximum(0, pos - 150), dtype=dtype, width=width)
    slopes = (2.0 ** (-8.0 * np.arange(1, heads + 1) / heads)).astype(np.float32) if bias else None
    out, lse = b.run(gpu, softcap=softcap, slopes=b.dev(slopes))
    check_rms(b, out, lse, softcap, slopes)


@TYPES
@pytest.mark.parametrize("heads,k", [(16, 64), (20, 300), (32, 1000), (64, 512), (128, 2048)])
def test_selections(gpu, heads, k, dtype):
    announce(f"sparse_attention rms heads={heads} k={k} {dtype}")
    b = Batch(391 + k, heads, [1] * 5, [400, 70, 2500, 1000, 64], dtype=dtype)
    lists, picked = selections(b, k, k)
    out, lse = b.out()
    gpu.sparse_attention(b.q.to(DEV), b.cache.to(DEV), b.dev(b.table), b.dev(lists), 1, SCALE, out, lse)
    torch.cuda.synchronize()
    check_rms(b, out, lse, picked=picked)


def around(*edges):
    """Rows on both sides of each edge."""
    return sorted({e + d for e in edges for d in (-1, 0)})


@TYPES
@pytest.mark.parametrize("heads,k", [(16, 70), (32, 128), (40, 1024), (64, 1024), (128, 700), (100, 700)])
def test_ragged_selections(gpu, heads, k, dtype):
    """A ragged batch over selections with more than 64 and more than 256 pair
    tiles, at lists that take 16-, 32-, 64- and 128-pair tiles: requests without
    rows at the front, in the middle and at the end, and rows of no request
    before the first and behind the last."""
    announce(f"sparse_attention ragged heads={heads} k={k} {dtype}")
    counts, lead, tail = [0, 37, 1, 0, 0, 300, 150, 5, 0], 6, 9
    n = sum(counts)
    rng = np.random.default_rng(k)
    b = Batch(401, heads, counts, rng.integers(1, 900, n), dtype=dtype)
    lists, picked = selections(b, k, 5)
    pad = lambda x, fill: np.concatenate([np.full((lead, *x.shape[1:]), fill, x.dtype), x,
                                          np.full((tail, *x.shape[1:]), fill, x.dtype)])
    q = torch.cat([torch.ones(lead, heads, 576), b.q.float(), torch.ones(tail, heads, 576)]).to(b.q.dtype)
    out, lse = b.out(lead + tail)
    gpu.sparse_attention(q.to(DEV), b.cache.to(DEV), b.dev(b.table), b.dev(pad(lists, 0)), 0, SCALE, out, lse,
                         cu_q=b.dev((b.first + lead).astype(np.int32)))
    torch.cuda.synchronize()
    mine = slice(lead, lead + n)
    for x in (out, lse):
        assert (x[:lead] == 5).all() and (x[lead + n:] == 5).all()
        assert torch.isfinite(x[mine][[r for r in range(n) if len(picked[r])]]).all()
    # (one pair tile per row of the padded batch)
    edges = around(1, 37, 38, 338, n - 1, 64 - lead, 65 - lead, 256 - lead, 257 - lead)
    check_rms(b, out[mine], lse[mine], picked=picked, rows=edges)
    b.check(out[mine], lse[mine], picked=picked, rows=edges)


@TYPES
@pytest.mark.parametrize("heads,requests,next_n,width", [(16, 64, 4, 0), (16, 300, 1, 0), (8, 260, 2, 0),
                                                         (32, 90, 1, WIDE), (64, 130, 1, WIDE), (128, 300, 1, WIDE)])
def test_shared_prefix_of_many(gpu, heads, requests, next_n, width, dtype):
    """Batches on a shared prefix with more than 64 and more than 256 pair tiles."""
    announce(f"shared_prefix_attention heads={heads} requests={requests} next_n={next_n} {dtype}")
    prefix, rng = 2, np.random.default_rng(requests)
    tails = rng.choice([0, 1, 30, 64, 100, 200], requests)
    tails[1], tails[-1] = 0, 333
    ends = np.concatenate([prefix * 64 + t - np.arange(next_n)[::-1] for t in tails])
    ends[5 * next_n:6 * next_n] = 0
    b = Batch(411, heads, [next_n] * requests, ends, shared=prefix, dtype=dtype, width=width)
    out, lse = b.out()
    gpu.shared_prefix_attention(b.q.to(DEV), b.cache.to(DEV), b.dev(b.table), b.dev(ends.astype(np.int32)), next_n,
                                prefix, SCALE, out, lse)
    torch.cuda.synchronize()
    live = torch.from_numpy(ends > 0)
    assert torch.isfinite(out).all() and torch.isfinite(lse.cpu()[live]).all()
    n = len(ends)
    rows = [r for r in around(1, 6 * next_n, 64, 65, n // 2, 256, 257, n) if r < n]
    check_rms(b, out, lse, rows=rows)
    b.check(out, lse, rows=rows)


@TYPES
@pytest.mark.parametrize("heads", [64, 128])
def test_ragged_extend_of_many(gpu, heads, dtype):
    """A ragged extend batch over whole pages with more than 64 and more than 256
    pair tiles of 128 pairs, rows of no request on both sides."""
    announce(f"paged_attention ragged extend heads={heads} {dtype}")
    counts, lead, tail = [0, 200, 0, 90, 1, 60, 0], 4, 7
    n = sum(counts)
    pos = np.concatenate([np.arange(p, p + c) for c, p in zip(counts, [0, 100, 0, 640, 50, 3, 9])])
    b = Batch(421, heads, counts, pos + 1, dtype=dtype, width=WIDE)
    q = torch.cat([torch.ones(lead, heads, 576), b.q.float(), torch.ones(tail, heads, 576)]).to(b.q.dtype)
    lens = np.concatenate([np.full(lead, 40), b.ends, np.full(tail, 40)]).astype(np.int32)
    out, lse = b.out(lead + tail)
    gpu.paged_attention(q.to(DEV), b.cache.to(DEV), b.dev(b.table), b.dev(lens), 0, SCALE, out, lse,
                        cu_q=b.dev((b.first + lead).astype(np.int32)))
    torch.cuda.synchronize()
    mine = slice(lead, lead + n)
    for x in (out, lse):
        assert (x[:lead] == 5).all() and (x[lead + n:] == 5).all() and torch.isfinite(x[mine]).all()
    rows = around(1, 64, 200, 201, 256, 290, 291, n - 1)
    check_rms(b, out[mine], lse[mine], rows=rows)
    b.check(out[mine], lse[mine], rows=rows)
