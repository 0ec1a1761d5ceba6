"""Release, fork, compaction and copies of cache pages on the GPU against the plain
oracle, number by number: pools of one page and of many, ragged lengths, pages held
by several requests, pools without a free page, results in place and apart, and the
calls together as a serving loop makes them, eager and captured."""
import numpy as np
import pytest
import torch

import oracle as O
from tests.gpu_harness import DEV, announce

pytestmark = pytest.mark.gpu
P = O.pages
I32 = dict(dtype=torch.int32, device=DEV)


def dev(x):
    return torch.tensor(np.asarray(x), **I32)


def make_pool(seed, requests, longest, spare, idle=0, shared=0.3, extra_columns=1):
    """(table, lens, refs): requests without tokens among them, pages held twice."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(1, longest + 1, requests)
    lens[rng.permutation(requests)[:idle]] = 0
    need = -(-lens // 64)
    pages = max(1, int(need.sum()) + spare)
    order = rng.permutation(pages)
    # columns behind a request's pages hold anything
    table = rng.integers(-3, pages + 3, (requests, -(-longest // 64) + extra_columns))
    refs, used = np.zeros(pages, np.int64), 0
    for b in range(requests):
        n = 0
        if b and rng.random() < shared:
            other = rng.integers(0, b)
            n = int(min(lens[b], lens[other]) // 64)
            table[b, :n] = table[other, :n]
        table[b, n:need[b]] = order[used:used + need[b] - n]
        used += need[b] - n
        np.add.at(refs, table[b, :need[b]], 1)
    return table, lens, refs


def same(got, want):
    assert np.array_equal(got.cpu().numpy(), np.asarray(want))


POOLS = [(1, 1, 0, 0), (1, 64, 3, 0), (2, 65, 0, 1), (7, 300, 2, 3), (64, 1000, 40, 20), (300, 130, 0, 100),
         (37, 5000, 700, 9), (4096, 70, 100, 2000)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("requests,longest,spare,idle", POOLS)
def test_release(gpu, requests, longest, spare, idle, in_place):
    announce(f"release_pages {requests} requests in_place={in_place}")
    table, lens, refs = make_pool(1, requests, longest, spare, idle)
    ended = np.random.default_rng(2).integers(0, 3, requests) * (np.arange(requests) % 3 != 1) - (requests == 1)
    t, a, r, m = dev(table), dev(lens), dev(refs), dev(ended)
    new_lens, new_refs = (a, r) if in_place else (torch.full_like(a, -9), torch.full_like(r, -9))
    gpu.release_pages(t, a, m, r, new_lens, new_refs)
    torch.cuda.synchronize()
    want_lens, want_refs = P.release(table.tolist(), lens.tolist(), ended.tolist(), refs.tolist())
    same(new_lens, want_lens)
    same(new_refs, want_refs)
    same(t, table)


def fork(gpu, table, lens, parents, refs, in_place=False, workspace=None):
    t, a, r, p = dev(table), dev(lens), dev(refs), dev(parents)
    n = len(lens)
    new_lens, new_refs = (a, r) if in_place else (torch.full_like(a, -9), torch.full_like(r, -9))
    lists = [torch.full((n,), -9, **I32) for _ in range(3)]
    counts = torch.full((2,), -9, **I32)
    gpu.fork_pages(t, a, p, r, new_lens, new_refs, *lists, counts, workspace=workspace)
    torch.cuda.synchronize()
    want = P.fork(table.tolist(), lens.tolist(), parents.tolist(), refs.tolist())
    for got, w in zip((t, new_lens, new_refs, *lists, counts), want):
        same(got, w)
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("requests,longest,spare,idle", POOLS)
def test_fork(gpu, requests, longest, spare, idle, in_place):
    announce(f"fork_pages {requests} requests spare={spare} in_place={in_place}")
    table, lens, refs = make_pool(3, requests, longest, spare, idle)
    # parents of every kind: none, out of range, busy children, requests that are forked themselves
    parents = np.random.default_rng(4).integers(-2, requests + 2, requests)
    want = fork(gpu, table, lens, parents, refs, in_place)
    if requests == 300:
        assert want[-1][1] > 0  # some went without


def test_fork_of_lengths_beyond_the_table(gpu):
    announce("fork_pages clamped lengths")
    table = np.arange(12).reshape(3, 4)
    refs = np.concatenate([np.ones(8, int), np.zeros(8, int)])
    fork(gpu, table, np.array([2 ** 31 - 1, -5, 0]), np.array([-1, 0, 0]), refs)
    fork(gpu, table, np.array([-(2 ** 31), 100, 0]), np.array([1, -1, 0]), refs)


def test_fork_of_one_parent_many_times(gpu):
    """A parent whose last page is full (nothing to copy) and one whose page is begun."""
    announce("fork_pages many children")
    for length in (128, 129, 63, 64):
        n = 200
        table = np.full((n, 3), -1)
        table[0, :3] = [7, 3, 9]
        refs = np.zeros(220, int)
        refs[table[0, :-(-length // 64)]] = 1
        lens = np.zeros(n, int)
        lens[0] = length
        parents = np.zeros(n, int)
        parents[0] = -1
        fork(gpu, table, lens, parents, refs)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("free", ["none", "last", "some", "all"])
@pytest.mark.parametrize("pages", [8192, 8193, 40001])
def test_fork_in_pools_of_many_pages(gpu, pages, free, in_place):
    """Free pages far behind, too few of them, and none."""
    announce(f"fork_pages {pages} pages, free: {free}")
    rng = np.random.default_rng(pages)
    refs = {"none": np.ones(pages, int), "last": (np.arange(pages) < pages - 5) * 2,
            "some": (rng.random(pages) > 0.0005) * 1, "all": np.zeros(pages, int)}[free]
    table = rng.integers(0, pages, (60, 3))
    lens = np.where(np.arange(60) % 3 == 0, rng.integers(1, 190, 60), 0)
    parents = np.where(lens == 0, np.arange(60) // 3 * 3, -1)
    fork(gpu, table, lens, parents, refs, in_place)


@pytest.mark.parametrize("requests,columns", [(128, 64), (129, 64), (3, 5000)])
def test_release_and_compact_at_the_small_pools_limit(gpu, requests, columns):
    announce(f"release_pages, compact_pages table of {requests} x {columns}")
    table, lens, refs = make_pool(31, requests, (columns - 1) * 64, 10, idle=1, extra_columns=1)
    assert table.shape[1] == columns
    ended = (np.arange(requests) % 4 == 0) * 1
    a, r = dev(lens), dev(refs)
    gpu.release_pages(dev(table), a, dev(ended), r, a, r)
    lens, refs = P.release(table.tolist(), lens.tolist(), ended.tolist(), refs.tolist())
    same(a, lens)
    same(r, refs)
    t, src, dst, counts = dev(table), torch.empty_like(r), torch.empty_like(r), torch.empty(2, **I32)
    gpu.compact_pages(t, a, r, t, r, src, dst, counts)
    for got, w in zip((t, r, src, dst, counts), P.compact(table.tolist(), lens, refs)):
        same(got, w)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("requests,longest,spare,idle", POOLS)
def test_compact(gpu, requests, longest, spare, idle, in_place):
    announce(f"compact_pages {requests} requests in_place={in_place}")
    table, lens, refs = make_pool(5, requests, longest, spare, idle)
    ended = np.random.default_rng(6).random(requests) < 0.4
    lens, refs = P.release(table.tolist(), lens.tolist(), ended.tolist(), refs.tolist())
    t, a, r = dev(table), dev(lens), dev(refs)
    new_table, new_refs = (t, r) if in_place else (torch.full_like(t, -9), torch.full_like(r, -9))
    src, dst, counts = torch.full_like(r, -9), torch.full_like(r, -9), torch.full((2,), -9, **I32)
    gpu.compact_pages(t, a, r, new_table, new_refs, src, dst, counts)
    torch.cuda.synchronize()
    want = P.compact(table.tolist(), lens, refs)
    for got, w in zip((new_table, new_refs, src, dst, counts), want):
        same(got, w)
    same(a, lens)


@pytest.mark.parametrize("held", ["none", "all", "upper", "lower", "one"])
@pytest.mark.parametrize("pages", [1, 2, 4095, 4096, 4097, 20000])
def test_compact_of_pools_at_their_edges(gpu, pages, held):
    announce(f"compact_pages {pages} pages, held: {held}")
    refs = {"none": np.zeros(pages, int), "all": np.full(pages, 3), "upper": (np.arange(pages) >= pages // 2) * 2,
            "lower": (np.arange(pages) < pages // 3) * 1, "one": (np.arange(pages) == pages - 1) * 1}[held]
    table = np.random.default_rng(pages).integers(0, pages, (3, 2))
    lens = [128, 1, 0]
    r, src, dst = dev(refs), torch.full((pages,), -9, **I32), torch.full((pages,), -9, **I32)
    new_table, new_refs, counts = torch.full((3, 2), -9, **I32), torch.full_like(r, -9), torch.full((2,), -9, **I32)
    gpu.compact_pages(dev(table), dev(lens), r, new_table, new_refs, src, dst, counts)
    torch.cuda.synchronize()
    for got, w in zip((new_table, new_refs, src, dst, counts), P.compact(table.tolist(), lens, refs.tolist())):
        same(got, w)


def make_caches(pages, seed, kinds=((400,), (128,), (68,), (576,), ())):
    """One cache of each token size: 400, 128 and 68 bytes, 576 values of 16 bits, one float."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for shape in kinds:
        t = torch.randint(0, 256, (pages, 64, *shape), generator=g, dtype=torch.uint8)
        out.append((t.to(torch.bfloat16) if shape == (576,) else t.float() if shape == () else t).to(DEV))
    return out


def copied(caches, src, dst, tokens, n):
    want = [c.clone() for c in caches]
    for i in range(n):
        s, d, k = int(src[i]), int(dst[i]), 64 if tokens is None else max(0, min(64, int(tokens[i])))
        if 0 <= s < len(caches[0]) and 0 <= d < len(caches[0]):
            for w, c in zip(want, caches):
                w[d, :k] = c[s, :k]
    return want


@pytest.mark.parametrize("some", [False, True])
@pytest.mark.parametrize("count", [None, 0, 3, 1000])
@pytest.mark.parametrize("n", [1, 5, 40])
def test_copy(gpu, n, count, some):
    announce(f"copy_pages {n} count={count} tokens={some}")
    pages = 90
    caches = make_caches(pages, n)
    order = np.random.default_rng(n).permutation(pages)
    src, dst = order[:n].copy(), order[n:2 * n].copy()
    if n > 4:
        src[2], dst[3], src[4] = -1, pages, 2 ** 31 - 1
    tokens = np.random.default_rng(n + 1).integers(-2, 67, n) if some else None
    want = copied(caches, src, dst, tokens, n if count is None else min(n, count))
    gpu.copy_pages(caches if n == 1 else gpu.PageCaches(caches), dev(src), dev(dst),
                   tokens=dev(tokens) if some else None, count=None if count is None else dev([count]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(caches, want))


@pytest.mark.parametrize("layers", [127, 128, 129, 300])
def test_copy_in_many_caches(gpu, layers):
    announce(f"copy_pages {layers} caches")
    caches = [torch.randint(0, 256, (6, 64, 4 * (1 + i % 3)), dtype=torch.uint8, device=DEV) for i in range(layers)]
    src, dst = np.array([0, 5, 2]), np.array([3, 1, 4])
    want = copied(caches, src, dst, [64, 7, 1], 3)
    gpu.copy_pages(caches, dev(src), dev(dst), tokens=dev([64, 7, 1]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(caches, want))


def test_copy_behind_4_gib(gpu):
    """Pages whose bytes lie beyond 2^32."""
    announce("copy_pages far pages")
    pages = 2 ** 32 // (64 * 1152) + 40
    cache = torch.zeros(pages, 64, 576, dtype=torch.bfloat16, device=DEV)
    cache[pages - 1] = 3.0
    gpu.copy_pages([cache], dev([pages - 1]), dev([pages - 30]))
    torch.cuda.synchronize()
    assert (cache[pages - 30] == 3).all() and float(cache.float().sum()) == 2 * 3.0 * 64 * 576


def turnover(gpu, s):
    """A step of a serving loop, in place: requests end, others fork, the pool is made dense."""
    gpu.release_pages(s["table"], s["lens"], s["ended"], s["refs"], s["lens"], s["refs"])
    gpu.fork_pages(s["table"], s["lens"], s["parents"], s["refs"], s["lens"], s["refs"], s["fsrc"], s["fdst"],
                   s["tokens"], s["fcounts"], workspace=s["ws"])
    gpu.copy_pages(s["caches"], s["fsrc"], s["fdst"], tokens=s["tokens"])
    gpu.compact_pages(s["table"], s["lens"], s["refs"], s["table"], s["refs"], s["src"], s["dst"], s["counts"],
                      workspace=s["ws"])
    gpu.copy_pages(s["caches"], s["src"], s["dst"], count=s["counts"][1:])


def loop_state(gpu, table, lens, refs, caches):
    n, pages = len(lens), len(refs)
    s = dict(table=dev(table), lens=dev(lens), refs=dev(refs), ended=torch.zeros(n, **I32),
             parents=torch.full((n,), -1, **I32), fcounts=torch.zeros(2, **I32), counts=torch.zeros(2, **I32),
             src=torch.zeros(pages, **I32), dst=torch.zeros(pages, **I32), caches=gpu.PageCaches(caches),
             ws=torch.empty(gpu.pages_workspace_bytes(n, pages), dtype=torch.uint8, device=DEV))
    s.update({k: torch.zeros(n, **I32) for k in ("fsrc", "fdst", "tokens")})
    return s


def tokens_of(table, lens, cache):
    """What each request reads."""
    out = []
    for row, n in zip(table, lens):
        at = np.arange(n)
        out.append(cache[torch.as_tensor(np.asarray(row)[at // 64], dtype=torch.long), torch.as_tensor(at % 64)])
    return out


@pytest.mark.parametrize("captured", [False, True])
def test_steps_of_a_serving_loop(gpu, captured):
    """Six steps in place, eager or replayed from one graph: after each, the books are the
    oracle's, every request that stayed reads what it read, and a forked one what its
    parent reads."""
    announce(f"release, fork, copy, compact in a loop captured={captured}")
    rng = np.random.default_rng(11)
    table, lens, refs = make_pool(9, 40, 700, 120, idle=12)
    caches = make_caches(len(refs), 13, ((400,), (68,), ()))
    s = loop_state(gpu, table, lens, refs, caches)
    graph = None
    if captured:
        first = {k: s[k].clone() for k in ("table", "lens", "refs")}
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            turnover(gpu, s)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            turnover(gpu, s)
        for k, v in first.items():  # the warm-up moved pages
            s[k].copy_(v)
        for c, fresh in zip(caches, make_caches(len(refs), 13, ((400,), (68,), ()))):
            c.copy_(fresh)
    table, lens, refs = table.tolist(), lens.tolist(), refs.tolist()
    for _ in range(6):
        busy = [b for b, n in enumerate(lens) if n]
        ended = np.zeros(len(lens), int)
        ended[rng.permutation(busy)[:6]] = 1
        stay = [b for b in busy if not ended[b]]
        parents = np.where(rng.random(len(lens)) < 0.4, rng.choice(stay, len(lens)), -1)
        s["ended"].copy_(dev(ended))
        s["parents"].copy_(dev(parents))
        host = [c.cpu() for c in caches]
        before = [tokens_of(table, lens, c) for c in host]
        graph.replay() if captured else turnover(gpu, s)
        torch.cuda.synchronize()
        held_before = lens
        lens, refs = P.release(table, lens, ended.tolist(), refs)
        cleared = lens
        table, lens, refs, *_ = P.fork(table, lens, parents.tolist(), refs)
        table, refs, src, dst, counts = P.compact(table, lens, refs)
        same(s["table"], table)
        same(s["lens"], lens)
        same(s["refs"], refs)
        same(s["counts"], counts)
        for c, old in zip([c.cpu() for c in caches], before):
            now = tokens_of(table, lens, c)
            for b in range(len(lens)):
                if cleared[b]:
                    assert torch.equal(now[b], old[b])
                elif lens[b]:
                    assert torch.equal(now[b], old[parents[b]])


def test_calls_on_another_stream(gpu):
    announce("page calls on a side stream")
    table, lens, refs = make_pool(21, 20, 400, 30, idle=5)
    caches = make_caches(len(refs), 2, ((400,),))
    s = loop_state(gpu, table, lens, refs, caches)
    parents = np.full(20, -1)
    parents[np.flatnonzero(lens == 0)] = int(np.argmax(lens))
    s["parents"].copy_(dev(parents))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        turnover(gpu, s)
    side.synchronize()
    t, n, r, *_ = P.fork(table.tolist(), lens.tolist(), parents.tolist(), refs.tolist())
    t, r, *_ = P.compact(t, n, r)
    same(s["table"], t)
    same(s["refs"], r)
