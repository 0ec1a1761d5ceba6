"""Attention over the latent cache on the GPU -- over a request's pages, over
pages that a batch shares, and over selected keys -- against a plain float64
implementation.  Every cache slot that no row of a test sees holds NaN, so an
unmasked read shows; bounds are derived in oracle/latent.py."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from tests.gpu_harness import DEV, announce

pytestmark = pytest.mark.gpu
L = O.latent

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
SCALE = 192 ** -0.5


class Batch:
    """Rows over requests' pages.  rows: rows of each request; ends: keys of
    each row; starts: first key of each row (or None); width: columns of the
    block table (the calls size their pair tiles by it: with WIDE columns 33 to
    64 pairs together take 64-pair tiles and more of them 128-pair tiles, with
    the few that the lengths need 16- and 32-pair tiles)."""

    def __init__(self, seed, heads, rows, ends, starts=None, dtype="bf16", shared=0, spare=3, q_scale=1.0, width=0):
        rng = np.random.default_rng(seed)
        self.rng, self.heads, self.dtype = rng, heads, dtype
        self.counts = list(rows)
        self.ends = np.asarray(ends, np.int64)
        self.starts = None if starts is None else np.asarray(starts, np.int64)
        self.first = np.concatenate([[0], np.cumsum(self.counts)])
        assert len(self.ends) == self.first[-1]
        need = [max([1] + [-(-int(e) // 64) for e in self.ends[a:b]]) for a, b in zip(self.first[:-1], self.first[1:])]
        need = [max(n, shared) for n in need]
        self.max_pages = max(max(need), width)
        self.pages = sum(n - shared for n in need) + shared + spare
        perm = rng.permutation(self.pages)
        self.table = rng.integers(-5, self.pages + 5, (len(need), self.max_pages)).astype(np.int32)
        used = shared
        for b, n in enumerate(need):
            self.table[b, :shared] = perm[:shared]
            self.table[b, shared:n] = perm[used:used + n - shared]
            used += n - shared
        self.request = np.repeat(np.arange(len(need)), self.counts)
        t = DTYPES[dtype]
        g = torch.Generator().manual_seed(seed)
        cache = torch.randn(self.pages * 64, 576, generator=g).to(t)
        seen = np.zeros(self.pages * 64, bool)
        for r in range(len(self.ends)):
            seen[self.slots(r, self.visible(r))] = True
        cache[torch.from_numpy(~seen)] = float("nan")
        self.cache = cache.view(self.pages, 64, 576)
        self.q = (torch.randn(len(self.ends), heads, 576, generator=g) * q_scale).to(t)

    def visible(self, r):
        lo = 0 if self.starts is None else max(0, int(self.starts[r]))
        return np.arange(lo, max(lo, int(self.ends[r])))

    def slots(self, r, at):
        return self.table[self.request[r], at // 64].astype(np.int64) * 64 + at % 64

    def dev(self, x):
        return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(DEV)

    def out(self, extra_rows=0):
        n = len(self.ends) + extra_rows
        return (torch.full((n, self.heads, 512), 5.0, dtype=DTYPES[self.dtype], device=DEV),
                torch.full((n, self.heads), 5.0, device=DEV))

    def uniform(self):
        return self.counts[0] if len(set(self.counts)) == 1 else 0

    def run(self, gpu, **kw):
        next_n = self.uniform()
        cu = None if next_n else self.dev(self.first.astype(np.int32))
        out, lse = self.out()
        gpu.paged_attention(self.q.to(DEV), self.cache.to(DEV), self.dev(self.table),
                            self.dev(self.ends.astype(np.int32)), next_n, SCALE, out, lse, cu_q=cu,
                            row_starts=self.dev(None if self.starts is None else self.starts.astype(np.int32)), **kw)
        torch.cuda.synchronize()
        return out, lse

    def check(self, out, lse, softcap=0.0, slopes=None, positions=None, picked=None, rows=None):
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        cache = self.cache.view(-1, 576)
        for r in range(len(self.ends)) if rows is None else rows:
            at = self.visible(r) if picked is None else picked[r]
            keys = cache[torch.from_numpy(self.slots(r, at))].double().numpy()
            pos = int(positions[r]) if positions is not None else int(self.ends[r]) - 1
            want, wl, ob, lb = L.attend_row(self.q[r].double().numpy(), keys, at, SCALE, softcap, slopes, pos,
                                            self.dtype)
            if len(at) == 0:
                assert (out[r] == 0).all() and (lse[r] == -np.inf).all(), f"row {r} without keys"
                continue
            bad = ~(np.abs(out[r] - want) <= ob)
            assert not bad.any(), (f"row {r} ({len(at)} keys): {bad.sum()} of {bad.size} outputs off, worst "
                                   f"{np.nanmax(np.abs(out[r] - want) / np.maximum(ob, 1e-30)):.2f} bounds, "
                                   f"{np.isnan(out[r]).sum()} NaN")
            assert (np.abs(lse[r] - wl) <= lb).all(), f"row {r} lse: {np.abs(lse[r] - wl).max()} over {lb.min()}"


WIDE = 1200
WIDTHS = pytest.mark.parametrize("width", [0, WIDE])
LENGTHS = [1, 63, 64, 65, 0, 127, 128, 200, 2, 333]


@WIDTHS
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,next_n", [(1, 1), (3, 1), (16, 1), (17, 1), (16, 2), (32, 1), (24, 3), (64, 1),
                                          (100, 1), (128, 1), (128, 2)])
def test_paged_decode(gpu, heads, next_n, dtype, width):
    """Head counts that fill pair tiles and ones that do not, lengths around
    page ends, verify rows (row j sees L + j keys), an empty request."""
    announce(f"paged_attention heads={heads} next_n={next_n} {dtype}")
    ends = [n + j if n else 0 for n in LENGTHS for j in range(next_n)]
    b = Batch(100 + heads + next_n, heads, [next_n] * len(LENGTHS), ends, dtype=dtype, width=width)
    b.check(*b.run(gpu))


@WIDTHS
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [8, 16, 128])
def test_paged_long(gpu, heads, dtype, width):
    """Requests that many workgroups share, beside short ones."""
    announce(f"paged_attention long heads={heads} {dtype}")
    b = Batch(7, heads, [1] * 4, [9001, 5, 0, 4097], dtype=dtype, q_scale=2.0, width=2 * width)
    b.check(*b.run(gpu))


def growing(b, seed):
    """Keys whose scores grow along the request, by far more than 2^60 in the
    weights: every running maximum is passed many times."""
    flat = b.cache.view(-1, 576).float()
    for r in range(len(b.ends)):
        at = np.arange(int(b.ends[r]))
        # (requests without pages in common)
        flat[torch.from_numpy(b.slots(r, at))] *= torch.from_numpy(0.05 + 8.0 * at / max(1, len(at)))[:, None].float()
    b.cache = flat.to(b.cache.dtype).view(b.cache.shape)


@WIDTHS
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [16, 32, 64, 128])
def test_growing_scores(gpu, heads, dtype, width):
    announce(f"paged and sparse attention growing scores heads={heads} {dtype}")
    b = Batch(37, heads, [1] * 5, [3000, 900, 400, 64, 2100], dtype=dtype, q_scale=4.0, width=width)
    growing(b, 1)
    b.check(*b.run(gpu))
    lists = np.full((5, 3000), -1, np.int32)
    for r, n in enumerate(b.ends):
        lists[r, :n] = np.arange(n)
    out, lse = b.out()
    gpu.sparse_attention(b.q.to(DEV), b.cache.to(DEV), b.dev(b.table), b.dev(lists), 1, SCALE, out, lse)
    torch.cuda.synchronize()
    b.check(out, lse)


@WIDTHS
@pytest.mark.parametrize("mask", ["causal", "window", "document", "prefix", "empty"])
@pytest.mark.parametrize("heads", [4, 16, 48])
def test_paged_ragged_masks(gpu, heads, mask, width):
    """Ragged extend batches: pair tiles hold several rows with key ranges of
    their own; requests without rows; rows whose range is empty."""
    announce(f"paged_attention ragged {mask} heads={heads}")
    rows, prefix = [37, 0, 1, 70, 5], [0, 10, 64, 130, 500]
    pos = np.concatenate([np.arange(p, p + n) for n, p in zip(rows, prefix)])
    ends, starts = pos + 1, None
    if mask == "window":
        starts = np.maximum(0, ends - 33)
    elif mask == "document":
        starts = pos // 29 * 29
    elif mask == "prefix":
        total = np.repeat([p + n for n, p in zip(rows, prefix)], rows)
        ends = np.minimum(np.maximum(ends, 100), total)
    elif mask == "empty":
        starts = np.where(np.arange(len(pos)) % 3 == 0, ends + np.arange(len(pos)) % 5, np.maximum(0, ends - 70))
    b = Batch(31, heads, rows, ends, starts, width=width)
    b.check(*b.run(gpu))


@WIDTHS
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("softcap,bias,given", [(20.0, False, False), (0.0, True, False), (30.0, True, True),
                                                (0.5, True, True)])
def test_paged_scores(gpu, softcap, bias, given, dtype, width):
    """Capped scores and the distance bias, on keys before and after the row."""
    announce(f"paged_attention softcap={softcap} bias={bias} {dtype}")
    heads, rows, prefix = 16, [9, 30, 2], [0, 300, 70]
    pos = np.concatenate([np.arange(p, p + n) for n, p in zip(rows, prefix)])
    total = np.repeat([p + n for n, p in zip(rows, prefix)], rows)
    ends = np.minimum(pos + 12, total) if given else pos + 1
    b = Batch(41, heads, rows, ends, dtype=dtype, q_scale=3.0, width=width)
    slopes = (2.0 ** (-8.0 * np.arange(1, heads + 1) / heads)).astype(np.float32) if bias else None
    positions = pos.astype(np.int32) if given else None
    out, lse = b.run(gpu, softcap=softcap, slopes=b.dev(slopes), row_positions=b.dev(positions))
    b.check(out, lse, softcap, slopes, positions)


def test_rows_behind_the_batch_stay(gpu):
    """A ragged batch padded with rows of no request: they are left alone."""
    announce("paged_attention padded ragged batch")
    b = Batch(51, 16, [3, 8], np.arange(100, 111))
    out, lse = b.out(4)
    pad = torch.zeros(4, 16, 576, dtype=torch.bfloat16)
    lens = b.dev(np.concatenate([b.ends, [50] * 4]).astype(np.int32))
    gpu.paged_attention(torch.cat([b.q, pad]).to(DEV), b.cache.to(DEV), b.dev(b.table), lens, 0, SCALE, out, lse,
                        cu_q=b.dev(b.first.astype(np.int32)))
    torch.cuda.synchronize()
    b.check(out[:11], lse[:11])
    assert (out[11:] == 5).all() and (lse[11:] == 5).all()
    idx = b.dev(np.tile(np.arange(20, dtype=np.int32), (15, 1)))
    out, lse = b.out(4)
    cache = torch.nan_to_num(b.cache).to(DEV)
    gpu.sparse_attention(torch.cat([b.q, pad]).to(DEV), cache, b.dev(b.table), idx, 0, SCALE, out, lse,
                         cu_q=b.dev(b.first.astype(np.int32)))
    torch.cuda.synchronize()
    b.cache = cache.cpu()
    b.check(out[:11], lse[:11], picked=[np.arange(20)] * 11)
    assert (out[11:] == 5).all() and (lse[11:] == 5).all()


@WIDTHS
@pytest.mark.parametrize("heads", [4, 16])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_hidden_nan_next_to_rows_that_see_it(gpu, dtype, heads, width):
    """Keys with NaN and infinities that some rows of a pair tile see and
    others do not: the others stay clean, the ones that see a NaN are NaN."""
    announce(f"paged_attention hidden NaN {dtype}")
    ends = np.arange(90, 98)
    b = Batch(61, heads, [8], ends, dtype=dtype, width=8 * width)
    flat = b.cache.view(-1, 576)
    slot = b.slots(0, np.arange(98))
    flat[slot[93], 7] = float("nan")     # seen by rows with end >= 94
    flat[slot[95], 560] = float("nan")
    flat[slot[96], 200] = float("inf")
    out, lse = b.run(gpu)
    b.check(out, lse, rows=range(4))
    assert torch.isnan(out[4:]).all() and torch.isnan(lse[4:]).all()


@WIDTHS
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [200, 560])
def test_infinity_under_a_cap(gpu, dtype, dim, width):
    """A capped score is finite, also that of a key with an infinity: the rows
    that see the key are NaN all the same, whichever part of a key holds it and
    whether or not other rows of the pair tile see the key too."""
    announce(f"paged_attention capped infinity {dtype} dim {dim}")
    for ends in (np.arange(90, 98), np.arange(120, 128)):
        b = Batch(63, 16, [8], ends, dtype=dtype, width=8 * width)
        b.cache.view(-1, 576)[b.slots(0, np.array([96]))[0], dim] = float("inf")
        out, lse = b.run(gpu, softcap=20.0)
        seen = ends > 96
        b.check(out, lse, softcap=20.0, rows=np.flatnonzero(~seen))
        assert torch.isnan(out[seen]).all() and torch.isnan(lse[seen]).all()


@WIDTHS
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,requests,next_n,prefix", [(16, 5, 1, 1), (16, 9, 2, 4), (128, 3, 1, 7), (5, 33, 1, 2),
                                                          (40, 2, 4, 40)])
def test_shared_prefix(gpu, heads, requests, next_n, prefix, dtype, width):
    """Requests with tails of none, one and many keys behind the prefix, one
    that ends inside it, and an empty one."""
    announce(f"shared_prefix_attention heads={heads} requests={requests} prefix={prefix} {dtype}")
    tails = [0, 1, 64, 200, 63, 129]
    ends = np.concatenate([prefix * 64 + tails[i % 6] - np.arange(next_n)[::-1] for i in range(requests)])
    ends[:next_n] = prefix * 64 - 30
    if requests > 3:
        ends[2 * next_n:3 * next_n] = 0
    b = Batch(71, heads, [next_n] * requests, ends, shared=prefix, dtype=dtype, width=width)
    out, lse = b.out()
    gpu.shared_prefix_attention(b.q.to(DEV), b.cache.to(DEV), b.dev(b.table), b.dev(b.ends.astype(np.int32)), next_n,
                                prefix, SCALE, out, lse)
    torch.cuda.synchronize()
    b.check(out, lse)


@WIDTHS
def test_shared_prefix_masks_and_scores(gpu, width):
    """Windows that begin inside, at the end of and behind the prefix; caps and
    slopes; a table that holds nothing but the prefix."""
    announce("shared_prefix_attention masks")
    heads, prefix = 16, 3
    ends = np.array([250, 260, 200, 192, 300, 193])
    starts = np.array([100, 192, 195, 0, 299, 64])
    b = Batch(81, heads, [1] * 6, ends, starts, shared=prefix, width=width)
    slopes = np.linspace(0.01, 0.5, heads).astype(np.float32)
    pos = (ends + 3).astype(np.int32)
    out, lse = b.out()
    gpu.shared_prefix_attention(b.q.to(DEV), b.cache.to(DEV), b.dev(b.table), b.dev(ends.astype(np.int32)), 1, prefix,
                                SCALE, out, lse, row_starts=b.dev(starts.astype(np.int32)), softcap=25.0,
                                slopes=b.dev(slopes), row_positions=b.dev(pos))
    torch.cuda.synchronize()
    b.check(out, lse, 25.0, slopes, pos)
    b = Batch(82, heads, [2] * 5, np.arange(183, 193), shared=3)
    out, lse = b.out()
    gpu.shared_prefix_attention(b.q.to(DEV), b.cache.to(DEV), b.dev(b.table), b.dev(b.ends.astype(np.int32)), 2, 3,
                                SCALE, out, lse)
    torch.cuda.synchronize()
    b.check(out, lse)


def selections(b, k, seed):
    """Lists of k entries per row: distinct visible keys in random order, -1
    and out-of-range padding anywhere, one row of padding only."""
    rng = np.random.default_rng(seed)
    lists, picked = np.full((len(b.ends), k), -1, np.int32), []
    for r, end in enumerate(b.ends):
        n = 0 if r == 1 else min(int(end), k if r % 2 else rng.integers(1, k + 1))
        chosen = rng.permutation(int(end))[:n]
        places = np.sort(rng.permutation(k)[:n])
        lists[r, places] = chosen
        holes = np.setdiff1d(np.arange(k), places)
        lists[r, holes] = rng.choice([-1, -7, b.max_pages * 64, 2 ** 31 - 1, -2 ** 31], len(holes))
        picked.append(chosen)
    return lists, picked


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,k", [(1, 1), (16, 5), (16, 64), (20, 100), (32, 65), (64, 512), (128, 300)])
def test_sparse(gpu, heads, k, dtype):
    announce(f"sparse_attention heads={heads} k={k} {dtype}")
    ends = np.array([400, 70, 1, 1000, 64, 63, 333])
    b = Batch(91 + k, heads, [1] * 7, ends, dtype=dtype)
    lists, picked = selections(b, k, k)
    out, lse = b.out()
    gpu.sparse_attention(b.q.to(DEV), b.cache.to(DEV), b.dev(b.table), b.dev(lists), 1, SCALE, out, lse)
    torch.cuda.synchronize()
    b.check(out, lse, picked=picked)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,rows", [(128, 24), (50, 40)])
@pytest.mark.parametrize("scores", [False, True])
def test_sparse_large_tiles(gpu, heads, rows, scores, dtype):
    """Selections that take 128- and 64-pair tiles: long lists, mostly padding,
    whole steps of it among them; with caps and slopes, too."""
    announce(f"sparse_attention large tiles heads={heads} {dtype} scores={scores}")
    k = 8192
    b = Batch(99, heads, [rows], np.arange(rows) * 31 + 200, dtype=dtype, q_scale=2.0)
    rng = np.random.default_rng(8)
    lists = np.full((rows, k), -1, np.int32)
    picked = []
    for r, end in enumerate(b.ends):
        n = 0 if r == 3 else rng.integers(1, min(int(end), 400) + 1)
        chosen = rng.permutation(int(end))[:n]
        first = rng.integers(0, 7000)
        lists[r, np.sort(first + rng.permutation(1100)[:n])] = chosen
        picked.append(chosen)
    slopes = np.linspace(0.01, 0.5, heads).astype(np.float32) if scores else None
    pos = (b.ends + 5).astype(np.int32) if scores else None
    cap = 20.0 if scores else 0.0
    out, lse = b.out()
    gpu.sparse_attention(b.q.to(DEV), b.cache.to(DEV), b.dev(b.table), b.dev(lists), rows, SCALE, out, lse,
                         softcap=cap, slopes=b.dev(slopes), row_positions=b.dev(pos))
    torch.cuda.synchronize()
    b.check(out, lse, cap, slopes, pos, picked=picked)


@pytest.mark.parametrize("heads,rows", [(16, 2), (40, 2), (128, 2), (128, 300)])
def test_sparse_long_lists(gpu, heads, rows):
    """Lists longer than the keys that are resolved at a time, for few rows
    (cut into parts) and for many (whole rows)."""
    announce(f"sparse_attention long lists heads={heads} rows={rows}")
    b = Batch(97, heads, [rows], [6000 - r for r in range(rows)])
    rng = np.random.default_rng(3)
    lists = np.stack([rng.permutation(5600)[:5000] for _ in range(rows)]).astype(np.int32)
    lists[rng.random(lists.shape) < 0.05] = -1
    picked = [row[row >= 0] for row in lists]
    out, lse = b.out()
    gpu.sparse_attention(b.q.to(DEV), b.cache.to(DEV), b.dev(b.table), b.dev(lists), rows, SCALE, out, lse)
    torch.cuda.synchronize()
    b.check(out, lse, picked=picked, rows=range(rows) if rows < 10 else [0, 1, 77, 255, 256, 299])
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("ragged", [False, True])
def test_sparse_rows_and_scores(gpu, ragged):
    """Several rows per request with lists of their own, caps and slopes, a key
    listed twice (which counts twice)."""
    announce(f"sparse_attention rows ragged={ragged}")
    rows = [3, 0, 5, 1] if ragged else [3, 3, 3]
    n = sum(rows)
    heads, k = 16, 70
    b = Batch(95, heads, rows, np.arange(n) * 20 + 90)
    lists, picked = selections(b, k, 4)
    lists[0, :2] = 17
    picked[0] = lists[0][(lists[0] >= 0) & (lists[0] < b.max_pages * 64)]
    b.cache = torch.nan_to_num(b.cache)
    slopes = np.linspace(0.01, 0.5, heads).astype(np.float32)
    pos = (b.ends - 1).astype(np.int32)
    out, lse = b.out()
    gpu.sparse_attention(b.q.to(DEV), b.cache.to(DEV), b.dev(b.table), b.dev(lists), b.uniform(), SCALE, out, lse,
                         cu_q=b.dev(b.first.astype(np.int32)) if ragged else None, softcap=15.0,
                         slopes=b.dev(slopes), row_positions=b.dev(pos))
    torch.cuda.synchronize()
    b.check(out, lse, 15.0, slopes, pos, picked=picked)


def test_many_requests(gpu):
    """More pair tiles than the work list takes in one step, most of them short."""
    announce("paged_attention 1500 requests")
    rng = np.random.default_rng(2)
    ends = rng.integers(0, 130, 1500)
    ends[700] = 3000
    b = Batch(101, 2, [1] * 1500, ends)
    out, lse = b.run(gpu)
    b.check(out, lse, rows=[0, 1, 255, 256, 257, 511, 699, 700, 701, 1023, 1024, 1498, 1499])
    assert torch.isfinite(out).all()


def test_far_pages(gpu):
    """Pages beyond 4 GiB of cache, and lengths past the table (clamped)."""
    announce("paged, shared and sparse attention far pages")
    pages = 60000  # 4.4 GB
    cache = torch.zeros(pages, 64, 576, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(9)
    table = torch.tensor([[59999, 58254, 3, 59990]], dtype=torch.int32)
    keys = torch.randn(4, 64, 576, generator=g).bfloat16()
    cache[table[0].long().to(DEV)] = keys.to(DEV)
    q = torch.randn(1, 16, 576, generator=g).bfloat16()
    out = torch.empty(1, 16, 512, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(1, 16, device=DEV)
    want, wl, ob, lb = L.attend_row(q[0].double().numpy(), keys.view(256, 576).double().numpy(), np.arange(256), SCALE)
    lens = torch.tensor([2 ** 31 - 1], dtype=torch.int32, device=DEV)
    idx = torch.arange(256, dtype=torch.int32, device=DEV).view(1, -1)
    for call in (lambda: gpu.paged_attention(q.to(DEV), cache, table.to(DEV), lens, 1, SCALE, out, lse),
                 lambda: gpu.shared_prefix_attention(q.to(DEV), cache, table.to(DEV), lens, 1, 2, SCALE, out, lse),
                 lambda: gpu.sparse_attention(q.to(DEV), cache, table.to(DEV), idx, 1, SCALE, out, lse)):
        out.fill_(9)
        call()
        torch.cuda.synchronize()
        assert (np.abs(out[0].double().cpu().numpy() - want) <= ob).all()
        assert (np.abs(lse[0].double().cpu().numpy() - wl) <= lb).all()


def all_calls(gpu, b, lists, prefix, workspace=None, sizes=None):
    """One call of each operator on the batch; returns their outputs."""
    q, cache, table = b.q.to(DEV), b.cache.to(DEV), b.dev(b.table)
    ends, idx = b.dev(b.ends.astype(np.int32)), b.dev(lists)
    outs = [b.out() for _ in range(3)]

    def calls():
        gpu.paged_attention(q, cache, table, ends, 1, SCALE, *outs[0], workspace=workspace)
        gpu.shared_prefix_attention(q, cache, table, ends, 1, prefix, SCALE, *outs[1], workspace=workspace)
        gpu.sparse_attention(q, cache, table, idx, 1, SCALE, *outs[2], workspace=workspace)
    return calls, outs


def test_graphs_share_a_workspace(gpu):
    """Two captured graphs with one workspace, replayed in turn with eager calls
    in between: every replay gives the eager bits.  Also on another stream."""
    announce("attention graphs")
    prefix = 2
    batches = [Batch(111 + i, 16, [1] * 5, [128 + 900 * i, 140, 700, 129, 2000 - i], shared=prefix) for i in range(2)]
    need = max(max(gpu.attention_workspace_bytes(5, 16, 5), gpu.shared_prefix_workspace_bytes(5, 16, 5)), 256)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV).fill_(0xA5)
    graphs, expected = [], []
    for b in batches:
        lists, _ = selections(b, 150, 6)
        calls, outs = all_calls(gpu, b, lists, prefix, ws)
        calls()
        torch.cuda.synchronize()
        expected.append([[x.clone() for x in o] for o in outs])
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            calls()
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls()
        graphs.append((g, outs, calls))
    for turn in range(4):
        for (g, outs, calls), want in zip(graphs, expected):
            for o in outs:
                for x in o:
                    x.fill_(3.0)
            ws.fill_(turn)
            g.replay()
            torch.cuda.synchronize()
            for o, w in zip(outs, want):
                for x, y in zip(o, w):
                    assert torch.equal(x, y), f"replay {turn}"
            calls()
            torch.cuda.synchronize()
            for o, w in zip(outs, want):
                for x, y in zip(o, w):
                    assert torch.equal(x, y), f"eager {turn}"


def test_two_streams_at_once(gpu):
    """Calls on two streams in flight together, each with the workspace that the
    call takes for itself, give the bits of calls alone."""
    announce("attention on two streams")
    batches = [Batch(131 + i, 16 + 112 * i, [1] * 6, [1500, 30, 700, 2500, 129, 64], shared=0) for i in range(2)]
    runs = []
    for b in batches:
        lists, _ = selections(b, 300, 9)
        args = [b.q.to(DEV), b.cache.to(DEV), b.dev(b.table), b.dev(b.ends.astype(np.int32)), b.dev(lists)]
        alone = [b.out() for _ in range(2)]
        gpu.paged_attention(*args[:4], 1, SCALE, *alone[0])
        gpu.sparse_attention(*args[:3], args[4], 1, SCALE, *alone[1])
        runs.append((args, alone, [b.out() for _ in range(2)], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for args, _, outs, stream in runs:
            with torch.cuda.stream(stream):
                gpu.paged_attention(*args[:4], 1, SCALE, *outs[0])
                gpu.sparse_attention(*args[:3], args[4], 1, SCALE, *outs[1])
    torch.cuda.synchronize()
    for _, alone, outs, _ in runs:
        for want, got in zip(alone, outs):
            assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_forms_agree(gpu):
    """The three operators on the same keys agree within the sum of their
    bounds, a call without lse or workspace gives the same bits, and two calls
    give the same bits."""
    announce("attention forms agree")
    b = Batch(121, 32, [1] * 3, [300, 300, 300], shared=2)
    lists = np.stack([np.random.default_rng(r).permutation(300) for r in range(3)]).astype(np.int32)
    calls, outs = all_calls(gpu, b, lists, 2)
    calls()
    torch.cuda.synchronize()
    for out, lse in outs:
        b.check(out, lse)
    first = [o[0].clone() for o in outs]
    calls()
    torch.cuda.synchronize()
    for o, f in zip(outs, first):
        assert torch.equal(o[0], f)
    alone = torch.empty_like(outs[0][0])
    gpu.paged_attention(b.q.to(DEV), b.cache.to(DEV), b.dev(b.table), b.dev(b.ends.astype(np.int32)), 1, SCALE, alone,
                        events=(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)))
    torch.cuda.synchronize()
    assert torch.equal(alone, outs[0][0])


def test_indexer_chain(gpu):
    """The operators as one decode step: index keys and latent rows appended to
    their pages, logits with their histogram, top-k, attention over the
    selection -- against the oracle on the caches that were written, and for a
    context no longer than k against attention over all keys."""
    announce("append -> logits -> top-k -> sparse attention")
    heads, k = 16, 256
    lens = [700, 256, 100]
    g = torch.Generator().manual_seed(13)
    total = sum(lens)
    need = [-(-n // 64) for n in lens]
    perm = torch.randperm(sum(need) + 2, generator=g).int()
    table = torch.zeros(3, max(need), dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    pos = torch.cat([torch.arange(n) for n in lens]).int()
    req = torch.repeat_interleave(torch.arange(3), torch.tensor(lens))
    slots = (table[req, (pos // 64).long()] * 64 + pos % 64).int()
    angle = torch.arange(1024).double()[:, None] * 10000.0 ** (-torch.arange(32).double() / 32)
    rope = torch.cat([angle.cos(), angle.sin()], 1).float().to(DEV)
    keys = torch.randn(total, 128, generator=g).bfloat16().to(DEV)
    rows = torch.randn(total, 576, generator=g).bfloat16().to(DEV)
    P = len(perm)
    kv = torch.zeros(P, 64, 128, dtype=torch.uint8, device=DEV)
    sc = torch.zeros(P, 64, device=DEV)
    latent = torch.full((P, 64, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
    gpu.index_k_append(keys, pos.to(DEV), slots.to(DEV), rope, kv, sc)
    gpu.latent_append(rows, pos.to(DEV), slots.to(DEV), rope, latent, interleaved=True)
    q8 = torch.randn(3, 32, 128, generator=g).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    w = torch.rand(3, 32, generator=g).to(DEV)
    bt, ctx = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    logits = torch.empty(3, 704, device=DEV)
    hist = torch.zeros(3, 1024, dtype=torch.int32, device=DEV)
    gpu.indexer_logits(q8, kv, sc, w, bt, ctx, 1, logits, hist)
    idx = torch.empty(3, k, dtype=torch.int32, device=DEV)
    gpu.topk_rows(logits, hist, ctx, k, gpu.KEY_FP32, idx)
    q = torch.randn(3, heads, 576, generator=g).bfloat16()
    out = torch.empty(3, heads, 512, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(3, heads, device=DEV)
    gpu.sparse_attention(q.to(DEV), latent, bt, idx, 1, SCALE, out, lse)
    dense, dense_lse = torch.empty_like(out), torch.empty_like(lse)
    gpu.paged_attention(q.to(DEV), latent, bt, ctx, 1, SCALE, dense, dense_lse)
    torch.cuda.synchronize()
    want_idx = O.topk_rows(logits.cpu().numpy(), np.array(lens), k, O.KEY_FP32)
    cache = latent.view(-1, 576).double().cpu().numpy()
    for r in range(3):
        chosen = idx[r].cpu().numpy()
        chosen = np.sort(chosen[chosen >= 0])
        assert np.array_equal(chosen, want_idx[r][want_idx[r] >= 0])
        for got, got_lse, at in ((out, lse, chosen), (dense, dense_lse, np.arange(lens[r]))):
            where = table[r].numpy()[at // 64].astype(np.int64) * 64 + at % 64
            want, wl, ob, lb = L.attend_row(q[r].double().numpy(), cache[where], at, SCALE)
            assert (np.abs(got[r].double().cpu().numpy() - want) <= ob).all()
            assert (np.abs(got_lse[r].double().cpu().numpy() - wl) <= lb).all()
