"""Attention over the 4-bit latent cache on the GPU: every test of the 16-bit cache on
4-bit rows, against the same plain float64 implementation and the same bounds (the
values of 4-bit rows are exact in 16 bits), and what 4-bit rows have of their own --
powers of two at both ends, blocks of NaN, far pages, the chain from the append."""
import numpy as np
import pytest
import torch

import oracle as O
import tests.test_gpu_attention as base
import tests.test_gpu_attention_limits as limits
import tests.test_gpu_attention_range as ranges
import tests.test_gpu_attention_rms as rms
from tests.gpu_harness import DEV, announce
from tests.mxfp4_cache import Batch4, Packing, pack, unpack

pytestmark = pytest.mark.gpu
L = O.latent
SCALE, DTYPES = base.SCALE, base.DTYPES
SKIP = {"test_far_pages", "test_indexer_chain",          # below, on 4-bit pages
        "test_two_streams_at_once", "test_graphs_share_a_workspace"}


def cases_of(module):
    """(function, arguments) of every parametrised test of a module."""
    out = []
    for name, f in vars(module).items():
        if not name.startswith("test_") or name in SKIP or getattr(f, "__module__", "") != module.__name__:
            continue
        cases = [{}]
        for mark in getattr(f, "pytestmark", []):
            if mark.name != "parametrize":
                continue
            names = [n.strip() for n in mark.args[0].split(",")]
            rows = [v if len(names) > 1 else (v,) for v in mark.args[1]]
            cases = [{**c, **dict(zip(names, row))} for c in cases for row in rows]
        for c in cases:
            label = "-".join(str(v) for v in c.values())
            out.append(pytest.param(f, c, id=f"{name[5:]}[{label}]"))
    return out


@pytest.fixture
def four(gpu, monkeypatch):
    for module in (base, ranges, rms):
        monkeypatch.setattr(module, "Batch", Batch4)
    return Packing(gpu)


@pytest.mark.parametrize("test,case", cases_of(base))
def test_as_16_bit(four, test, case):
    announce(f"4-bit rows: {test.__name__} {case}")
    test(four, **case)


@pytest.mark.parametrize("test,case", cases_of(ranges))
def test_as_16_bit_range(four, test, case):
    announce(f"4-bit rows: {test.__name__} {case}")
    test(four, **case)


@pytest.mark.parametrize("test,case", cases_of(rms))
def test_as_16_bit_rms(four, test, case):
    announce(f"4-bit rows: {test.__name__} {case}")
    test(four, **case)


@pytest.mark.parametrize("case", ["selections", "pages of 1 head", "pages of 17 heads"])
def test_as_16_bit_most_rows(gpu, monkeypatch, case):
    """As many rows and requests as a call takes."""
    announce(f"4-bit rows: most rows, {case}")
    plain = limits.caches

    def rounded(*args):
        g, cache, table = plain(*args)
        return g, unpack(pack(cache), cache.dtype), table

    monkeypatch.setattr(limits, "caches", rounded)
    if case == "selections":
        limits.test_most_ragged_rows_over_selections(Packing(gpu))
    else:
        limits.test_most_requests_over_pages(Packing(gpu), int(case.split()[2]), 15)


def test_packing_is_the_oracles(gpu):
    announce("packing of the tests")
    x = torch.randn(50, 576, generator=torch.Generator().manual_seed(1)).bfloat16()
    x[3, 5], x[4, 40], x[5, :64] = float("nan"), float("inf"), 0
    rows = pack(x).numpy()
    want = L.mxfp4_key(x[:, :512].float().numpy())
    keep = ~((want[:, 256:] == 0) & (rows[:, 256:272] != 0))  # a block of zeros may have any power
    assert np.array_equal(rows[:, :256], want[:, :256]) and keep.sum() == keep.size - 2
    assert np.array_equal(rows[:, 256:272][keep], want[:, 256:][keep])
    v = unpack(torch.from_numpy(rows), torch.bfloat16).double().numpy()
    assert np.array_equal(v, L.latent_mxfp4_values(rows, "bf16"), equal_nan=True)


@pytest.mark.parametrize("form", ["paged", "shared", "sparse"])
@pytest.mark.parametrize("heads", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype,powers", [("bf16", (0, 1, 3, 60, 127, 200, 240)),
                                          ("fp16", (101, 103, 110, 127, 138, 140))])
def test_powers_of_two_at_both_ends(gpu, dtype, powers, heads, form):
    """Every code under powers from the least to nearly the largest that stay in the
    type, one power a request; the queries see the latent part through the rotated
    dimensions alone, so that scores are small.  Products with values below the type's
    normal range may lose what lies below float32's: 2^-126 for each key; outputs below
    it have steps of 2^-24 and 2^-133."""
    announce(f"{form} attention mxfp4 powers {dtype} heads={heads}")
    n, lens = len(powers), [70 + 5 * i for i in range(len(powers))]
    g = torch.Generator().manual_seed(heads)
    need = [-(-x // 64) for x in lens]
    table = np.full((n, max(need) if heads < 64 else 600), 0, np.int32)
    table[:, 0] = 0  # shared: one page in common
    at = 1
    for i, k in enumerate(need):
        table[i, 1 if form == "shared" else 0:k] = np.arange(at, at + k - (form == "shared"))
        at += k
    rows = torch.randint(0, 256, (at, 64, 400), generator=g, dtype=torch.uint8)
    rows[..., 272:] = torch.randn(at, 64, 64, generator=g).to(DTYPES[dtype]).view(torch.uint8)
    for i in range(n):
        for p in table[i, :need[i]]:
            rows[p, :, 256:272] = powers[i]
    if form == "shared":
        rows[0, :, 256:272] = powers[0]
    q = torch.zeros(n, heads, 576, dtype=DTYPES[dtype])
    q[:, :, 512:] = torch.randn(n, heads, 64, generator=g)
    out = torch.empty(n, heads, 512, dtype=DTYPES[dtype], device=DEV)
    lse = torch.empty(n, heads, device=DEV)
    dev = lambda x: torch.as_tensor(x).to(DEV)
    ends = dev(np.array(lens, np.int32))
    if form == "paged":
        gpu.paged_attention_mxfp4(dev(q), dev(rows), dev(table), ends, 1, SCALE, out, lse)
    elif form == "shared":
        gpu.shared_prefix_attention_mxfp4(dev(q), dev(rows), dev(table), ends, 1, 1, SCALE, out, lse)
    else:
        idx = np.full((n, 128), -1, np.int32)
        for i, k in enumerate(lens):
            idx[i, :k] = np.arange(k)
        gpu.sparse_attention_mxfp4(dev(q), dev(rows), dev(table), dev(idx), 1, SCALE, out, lse)
    torch.cuda.synchronize()
    values = L.latent_mxfp4_values(rows.view(-1, 400).numpy(), dtype)
    if dtype == "fp16":  # keys are taken in the queries' type, which holds 2^-25 (a power below 104) rounded
        with np.errstate(over="ignore"):
            values = values.astype(np.float16).astype(np.float64)
    for i, k in enumerate(lens):
        s = np.arange(k)
        keys = values[table[i, s // 64].astype(np.int64) * 64 + s % 64]
        want, wl, ob, lb = L.attend_row(q[i].double().numpy(), keys, s, SCALE, dtype=dtype)
        room = ob + k * 2.0 ** -126 + (2.0 ** -25 if dtype == "fp16" else 2.0 ** -134)
        assert (np.abs(out[i].double().cpu().numpy() - want) <= room).all(), f"power {powers[i]}"
        assert (np.abs(lse[i].double().cpu().numpy() - wl) <= lb).all()


@pytest.mark.parametrize("heads,width", [(16, 1), (32, 600), (64, 600), (128, 600)])
def test_blocks_of_nan(gpu, heads, width):
    """The byte 255 makes a row that sees the key NaN, whatever its codes and whatever
    the queries are at the block's dimensions, and no other."""
    announce(f"paged_attention_mxfp4 NaN block heads={heads}")
    g = torch.Generator().manual_seed(3)
    cache = torch.randn(3, 64, 576, generator=g).bfloat16()
    rows = pack(cache)
    rows[1, 20, 256 + 7] = 255
    rows[1, 20, 16 * 7:16 * 8] = 0  # codes of zero
    table = torch.zeros(2, width, dtype=torch.int32)
    table[0, 0], table[1, 0] = 1, 2
    q = torch.randn(2, heads, 576, generator=g).bfloat16()
    q[:, :, 32 * 7:32 * 8] = 0
    for end, bad in ((20, False), (21, True), (60, True)):
        out = torch.empty(2, heads, 512, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(2, heads, device=DEV)
        gpu.paged_attention_mxfp4(q.to(DEV), rows.to(DEV), table.to(DEV),
                                  torch.tensor([end, 50], dtype=torch.int32, device=DEV), 1, SCALE, out, lse)
        torch.cuda.synchronize()
        assert bool(torch.isnan(out[0]).all()) == bad and bool(torch.isnan(lse[0]).all()) == bad
        assert torch.isfinite(out).all(2).all(1).tolist() == [not bad, True]


def test_far_pages(gpu):
    """Pages beyond 4 GiB of cache, and lengths past the table (clamped)."""
    announce("paged, shared and sparse attention mxfp4 far pages")
    pages = 2 ** 32 // (64 * 400) + 300
    cache = torch.zeros(pages, 64, 400, dtype=torch.uint8, device=DEV)
    g = torch.Generator().manual_seed(9)
    table = torch.tensor([[pages - 1, pages - 200, 3, pages - 9]], dtype=torch.int32)
    plain = torch.randn(4, 64, 576, generator=g).bfloat16()
    rows = pack(plain)
    # written by the append, at the position whose angles are zero
    slots = (table[0][:, None] * 64 + torch.arange(64)).flatten().int()
    at = torch.zeros(256, dtype=torch.int32, device=DEV)
    still = torch.cat([torch.ones(1, 32), torch.zeros(1, 32)], 1).to(DEV)
    gpu.latent_append_mxfp4(plain.view(256, 576).to(DEV), at, slots.to(DEV), still, cache)
    assert torch.equal(cache[table[0].long().to(DEV)].cpu(), rows)
    keys = L.latent_mxfp4_values(rows.view(-1, 400).numpy(), "bf16")
    for heads in (16, 128):
        q = torch.randn(1, heads, 576, generator=g).bfloat16()
        out = torch.empty(1, heads, 512, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(1, heads, device=DEV)
        want, wl, ob, lb = L.attend_row(q[0].double().numpy(), keys, np.arange(256), SCALE)
        lens = torch.tensor([2 ** 31 - 1], dtype=torch.int32, device=DEV)
        idx = torch.arange(256, dtype=torch.int32, device=DEV).view(1, -1)
        dq, dt = q.to(DEV), table.to(DEV)
        for call in (lambda: gpu.paged_attention_mxfp4(dq, cache, dt, lens, 1, SCALE, out, lse),
                     lambda: gpu.shared_prefix_attention_mxfp4(dq, cache, dt, lens, 1, 2, SCALE, out, lse),
                     lambda: gpu.sparse_attention_mxfp4(dq, cache, dt, idx, 1, SCALE, out, lse)):
            out.fill_(9)
            call()
            torch.cuda.synchronize()
            assert (np.abs(out[0].double().cpu().numpy() - want) <= ob).all()
            assert (np.abs(lse[0].double().cpu().numpy() - wl) <= lb).all()


@pytest.mark.parametrize("heads", [16, 64, 128])
@pytest.mark.parametrize("scale", [-0.05, 0.0, 1e-30])
def test_scales(four, heads, scale):
    """A factor that turns the scores' order round, and ones that make them all alike."""
    announce(f"attention mxfp4 scale={scale} heads={heads}")
    b = Batch4(151, heads, [1] * 4, [300, 65, 1, 900], width=600)
    lists = np.full((4, 960), -1, np.int32)
    for r, n in enumerate(b.ends):
        lists[r, :n] = np.arange(n)
    q, rows, table = b.q.to(DEV), b.cache.to(DEV), b.dev(b.table)
    for call, keys in (("paged_attention", b.ends.astype(np.int32)), ("sparse_attention", lists)):
        out, lse = b.out()
        getattr(four, call)(q, rows, table, b.dev(keys), 1, scale, out, lse)
        torch.cuda.synchronize()
        for r, n in enumerate(b.ends):
            at = np.arange(n)
            keys_r = b.cache.view(-1, 576)[torch.from_numpy(b.slots(r, at))].double().numpy()
            want, wl, ob, lb = L.attend_row(b.q[r].double().numpy(), keys_r, at, scale)
            assert (np.abs(out[r].double().cpu().numpy() - want) <= ob + n * 2.0 ** -110 * 8).all()
            assert (np.abs(lse[r].double().cpu().numpy() - wl) <= lb).all()


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("heads,rows,k", [(16, 300, 700), (32, 300, 700), (64, 300, 5000), (128, 200, 2300)])
def test_padded_selections_of_many(gpu, heads, rows, k, ragged):
    """Selections that are counted before they are shared out: full lists, lists that end
    early, one key at either end, keys behind long padding, none."""
    announce(f"sparse_attention_mxfp4 padded heads={heads} rows={rows} k={k}")
    counts = [rows // 3, 0, rows - rows // 3] if ragged else [rows]
    b = Batch4(161, heads, counts, np.full(rows, 6000))
    rng = np.random.default_rng(k)
    lists, picked = np.full((rows, k), -1, np.int32), []
    for r in range(rows):
        kind, n = r % 7, int(rng.integers(1, 200))
        places = {0: np.arange(k), 1: np.arange(n), 2: [0], 3: [k - 1], 4: np.arange(k - n, k), 5: [],
                  6: np.sort(rng.permutation(k)[:n])}[kind]
        chosen = rng.permutation(6000)[:len(places)]
        lists[r, np.asarray(places, int)] = chosen
        if kind != 0:
            holes = np.setdiff1d(np.arange(k), places)
            lists[r, holes] = rng.choice([-1, b.max_pages * 64, 2 ** 31 - 1, -2 ** 31], len(holes))
        picked.append(chosen)
    out, lse = b.out()
    gpu.sparse_attention_mxfp4(b.q.to(DEV), pack(b.cache).to(DEV), b.dev(b.table), b.dev(lists), 0 if ragged else rows,
                               SCALE, out, lse, cu_q=b.dev(b.first.astype(np.int32)) if ragged else None)
    torch.cuda.synchronize()
    b.check(out, lse, picked=picked, rows=list(range(14)) + [rows // 3 - 1, rows // 3, rows - 7, rows - 6, rows - 5,
                                                             rows - 4, rows - 3, rows - 2, rows - 1])
    some = torch.tensor([len(p) > 0 for p in picked])
    assert torch.isfinite(lse.cpu()[some]).all() and (lse.cpu()[~some] == -torch.inf).all()


def all_calls(gpu, b, prefix, workspace=None):
    q, rows, table = b.q.to(DEV), pack(b.cache).to(DEV), b.dev(b.table)
    lists, _ = base.selections(b, 300, 6)
    ends, idx = b.dev(b.ends.astype(np.int32)), b.dev(lists)
    outs = [b.out() for _ in range(3)]

    def calls():
        gpu.paged_attention_mxfp4(q, rows, table, ends, 1, SCALE, *outs[0], workspace=workspace)
        gpu.shared_prefix_attention_mxfp4(q, rows, table, ends, 1, prefix, SCALE, *outs[1], workspace=workspace)
        gpu.sparse_attention_mxfp4(q, rows, table, idx, 1, SCALE, *outs[2], workspace=workspace)
    return calls, [x for o in outs for x in o]


@pytest.mark.parametrize("heads", [16, 48, 128])
def test_graphs_share_a_workspace(gpu, heads):
    """Two captured graphs with one workspace, replayed in turn with eager calls in
    between: every replay gives the eager bits."""
    announce(f"attention mxfp4 graphs heads={heads}")
    batches = [base.Batch(111 + i, heads, [1] * 5, [128 + 900 * i, 140, 700, 129, 2000 - i], shared=2)
               for i in range(2)]
    need = max(gpu.attention_workspace_bytes(5, heads, 5), gpu.shared_prefix_workspace_bytes(5, heads, 5))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV).fill_(0xA5)
    graphs = []
    for b in batches:
        calls, outs = all_calls(gpu, b, 2, ws)
        calls()
        torch.cuda.synchronize()
        want = [x.clone() for x in outs]
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            calls()
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls()
        graphs.append((g, outs, calls, want))
    for turn in range(4):
        for g, outs, calls, want in graphs:
            for again in (g.replay, calls):
                for x in outs:
                    x.fill_(3.0)
                ws.fill_(turn)
                again()
                torch.cuda.synchronize()
                assert all(torch.equal(x, y) for x, y in zip(outs, want)), f"turn {turn}"


def test_two_streams_at_once(gpu):
    """Calls in flight together, each with the workspace that it takes for itself."""
    announce("attention mxfp4 on two streams")
    runs = []
    for i in range(2):
        b = base.Batch(131 + i, 16 + 112 * i, [1] * 6, [1500, 200, 700, 2500, 129, 130], shared=2)
        calls, outs = all_calls(gpu, b, 2)
        calls()
        torch.cuda.synchronize()
        runs.append((calls, outs, [x.clone() for x in outs], torch.cuda.Stream()))
    for _ in range(5):
        for calls, _, _, stream in runs:
            with torch.cuda.stream(stream):
                calls()
    torch.cuda.synchronize()
    for _, outs, want, _ in runs:
        assert all(torch.equal(x, y) for x, y in zip(outs, want))


@pytest.mark.parametrize("heads", [16, 128])
def test_same_as_over_16_bits(gpu, heads):
    """The cache in 4 bits and the same values in 16: equal within both bounds."""
    announce(f"attention mxfp4 against 16 bits heads={heads}")
    b = Batch4(141, heads, [1] * 4, [900, 64, 333, 2000])
    out, lse = b.run(Packing(gpu))
    other, other_lse = b.run(gpu)
    b.check(out, lse)
    b.check(other, other_lse)


def test_serving_chain(gpu):
    """The operators as they are used: positions on three axes composed, index keys and
    4-bit latent rows appended, queries rotated and cast, logits, top-k, attention over
    the selection; then a request is forked, its child goes on by itself in the copied
    page, the pool is made dense, and every request still reads its own keys -- against
    the oracle on the caches that were written."""
    announce("rotate, append, logits, top-k, sparse attention, fork, compact, paged attention")
    heads, k, lens = 16, 128, [700, 256, 100, 0]
    g = torch.Generator().manual_seed(13)
    need = [-(-n // 64) for n in lens]
    pages = sum(need) + 9
    perm = torch.randperm(pages, generator=g).int()
    table = torch.zeros(4, max(need) + 1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        refs[perm[at:at + n].long()] = 1
        at += n
    dev = lambda x: torch.as_tensor(x).to(DEV)
    pos = torch.cat([torch.arange(n) for n in lens]).int()
    req = torch.repeat_interleave(torch.arange(4), torch.tensor(lens))
    slots = (table[req, (pos // 64).long()] * 64 + pos % 64).int()
    angle = torch.arange(1024).double()[:, None] * 10000.0 ** (-torch.arange(32).double() / 32)
    rope = torch.cat([angle.cos(), angle.sin()], 1).float()
    axis_of = [0] * 8 + [1] * 12 + [2] * 12
    amap = gpu.axis_map(axis_of)
    axes = torch.stack([pos // 40, pos % 8, pos // 8 % 5]).int()
    total = sum(lens)
    keys, rows = torch.randn(total, 128, generator=g).bfloat16(), torch.randn(total, 576, generator=g).bfloat16()
    kv = torch.zeros(pages, 64, 128, dtype=torch.uint8, device=DEV)
    sc = torch.zeros(pages, 64, device=DEV)
    latent = torch.full((pages, 64, 400), 255, dtype=torch.uint8, device=DEV)
    turned = torch.empty(total, 64, device=DEV)
    index = torch.arange(total, dtype=torch.int32, device=DEV)
    gpu.axis_rotations(dev(axes), amap, dev(rope), turned)
    gpu.index_k_append(dev(keys), index, dev(slots), turned, kv, sc)
    gpu.latent_append_mxfp4(dev(rows), index, dev(slots), turned, latent)
    # queries: one row per request with keys, at its last position
    last = torch.tensor([699, 955, 1055])
    qi, ql = torch.randn(3, 32, 128, generator=g).bfloat16(), torch.randn(3, heads, 576, generator=g).bfloat16()
    q8, q = torch.empty(3, 32, 128, dtype=torch.uint8, device=DEV), dev(ql)
    at_q = dev(axes[:, last].contiguous())
    gpu.rotate_index_queries(dev(qi), at_q, dev(rope), q8, amap)
    gpu.rotate_queries(q[:, :, 512:], at_q, dev(rope), q[:, :, 512:], amap)
    w, ctx = torch.rand(3, 32, generator=g), dev(torch.tensor(lens[:3], dtype=torch.int32))
    logits, hist = torch.empty(3, 768, device=DEV), torch.zeros(3, 1024, dtype=torch.int32, device=DEV)
    bt = dev(table)
    gpu.indexer_logits(q8, kv, sc, dev(w), bt[:3].contiguous(), ctx, 1, logits, hist)
    idx = torch.empty(3, k, dtype=torch.int32, device=DEV)
    gpu.topk_rows(logits, hist, ctx, k, gpu.KEY_FP32, idx)
    out, lse = torch.empty(3, heads, 512, dtype=torch.bfloat16, device=DEV), torch.empty(3, heads, device=DEV)
    gpu.sparse_attention_mxfp4(q, latent, bt[:3].contiguous(), idx, 1, SCALE, out, lse)
    torch.cuda.synchronize()

    # the rotated parts are the definition's, on one rounding
    rows_at = L.axis_rows(rope.numpy(), axes.numpy(), axis_of)
    want_q = L.rotate(ql[:, :, 512:].double().numpy(), rows_at[last.numpy()][:, None], False)
    assert (np.abs(q[:, :, 512:].double().cpu().numpy() - want_q) <= 2.0 ** -8 * np.abs(want_q) + 2.0 ** -40).all()
    want_qi = L.index_key(qi.float().numpy(), rows_at[last.numpy()][:, None], False)
    assert np.array_equal(q8.cpu().numpy(), L.e4m3_codes(want_qi))
    want_idx = O.topk_rows(logits.cpu().numpy(), np.array(lens[:3]), k, O.KEY_FP32)

    def check(got, got_lse, cache, tab, r, query, chosen):
        where = tab[r][chosen // 64].astype(np.int64) * 64 + chosen % 64
        want, wl, ob, lb = L.attend_row(query, cache[where], chosen, SCALE)
        assert (np.abs(got.double().cpu().numpy() - want) <= ob).all()
        assert (np.abs(got_lse.double().cpu().numpy() - wl) <= lb).all()

    qd = q.double().cpu().numpy()
    cache = L.latent_mxfp4_values(latent.cpu().numpy().reshape(-1, 400), "bf16")
    for r in range(3):
        chosen = np.sort(idx[r].cpu().numpy())
        chosen = chosen[chosen >= 0]
        assert np.array_equal(chosen, want_idx[r][want_idx[r] >= 0])
        check(out[r], lse[r], cache, table.numpy(), r, qd[r], chosen)

    # request 3 forks request 0 (700 tokens, the last page begun); 1 ends; both 0 and 3 go on by a token
    i32 = dict(dtype=torch.int32, device=DEV)
    lens_d, refs_d = dev(torch.tensor(lens, dtype=torch.int32)), dev(refs)
    lists, counts = [torch.empty(4, **i32) for _ in range(3)], torch.empty(2, **i32)
    gpu.release_pages(bt, lens_d, torch.tensor([0, 1, 0, 0], **i32), refs_d, lens_d, refs_d)
    gpu.fork_pages(bt, lens_d, torch.tensor([-1, -1, -1, 0], **i32), refs_d, lens_d, refs_d, *lists, counts)
    caches = gpu.PageCaches([kv, sc, latent])
    gpu.copy_pages(caches, lists[0], lists[1], tokens=lists[2])
    torch.cuda.synchronize()
    t = bt.cpu()
    new = torch.randn(2, 576, generator=g).bfloat16()
    slot = torch.stack([t[0, 10] * 64 + 700 % 64, t[3, 10] * 64 + 700 % 64]).int()
    assert t[0, 10] != t[3, 10] and torch.equal(t[0, :10], t[3, :10])
    gpu.latent_append_mxfp4(dev(new), torch.tensor([700, 700], **i32), dev(slot), dev(rope), latent)
    lens_d += torch.tensor([1, 0, 0, 1], **i32)
    src, dst, counts = torch.empty(pages, **i32), torch.empty(pages, **i32), torch.empty(2, **i32)
    before = L.latent_mxfp4_values(latent.cpu().numpy().reshape(-1, 400), "bf16")
    gpu.compact_pages(bt, lens_d, refs_d, bt, refs_d, src, dst, counts)
    gpu.copy_pages(caches, src, dst, count=counts[1:])
    q4 = torch.stack([q[0], q[1], q[2], q[0]])
    out, lse = torch.empty(4, heads, 512, dtype=torch.bfloat16, device=DEV), torch.empty(4, heads, device=DEV)
    gpu.paged_attention_mxfp4(q4, latent, bt, lens_d, 1, SCALE, out, lse)
    torch.cuda.synchronize()
    held, moves = counts.tolist()
    assert held == 10 + 1 + 1 + 2 and moves > 0 and int(bt[[0, 2, 3]].max()) < pages
    after, tab = L.latent_mxfp4_values(latent.cpu().numpy().reshape(-1, 400), "bf16"), bt.cpu().numpy()
    for r, n in ((0, 701), (2, 100), (3, 701)):
        s = np.arange(n)
        where = tab[r][s // 64].astype(np.int64) * 64 + s % 64
        old = t.numpy()[r][s // 64].astype(np.int64) * 64 + s % 64
        assert (tab[r][:-(-n // 64)] < held).all() and np.array_equal(after[where], before[old])
        check(out[r], lse[r], after, tab, r, q4[r].double().cpu().numpy(), s)
    assert (out[1] == 0).all() and (lse[1] == -np.inf).all()
