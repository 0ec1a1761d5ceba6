"""The attention and the appends at the ends of what the header allows, and as a
captured decode step: as many rows as a call takes, ragged and uniform, and a
graph of appends and attention whose workspaces the calls take for themselves."""
import numpy as np
import pytest
import torch

from tests.gpu_harness import DEV, announce
from tests.test_gpu_attention import SCALE

pytestmark = pytest.mark.gpu
U, E = 2.0 ** -8, 2.0 ** -24  # half a step of bfloat16 and float32


def check_rows(q, keys, hidden, out, lse):
    """q [n, heads, 576], keys [n, k, 576], hidden [n, k]; scores of magnitude 8 at
    most (asserted), whose float32 sums, factors and exponentials are off by less
    than 2^-16; the weights by U each in numerator and divisor, 64 float32
    roundings of the sums, the output by its own rounding."""
    q, keys = q.double(), keys.double()
    z = SCALE * torch.stack([(q[:, h, None] * keys).sum(2) for h in range(q.shape[1])], 1)
    assert z.abs().max() < 8
    z = z.masked_fill(hidden[:, None], -torch.inf)
    want_lse = torch.logsumexp(z, 2)
    p = torch.where(hidden[:, None], 0.0, torch.exp(z - torch.where(want_lse.isinf(), 0.0, want_lse)[..., None]))
    v = keys[..., :512]
    want = sum(p[:, :, s, None] * v[:, None, s] for s in range(keys.shape[1]))
    off = sum(p[:, :, s, None] * (v[:, None, s] - want).abs() for s in range(keys.shape[1]))
    size = sum(p[:, :, s, None] * v[:, None, s].abs() for s in range(keys.shape[1]))
    inner = (1.01 * U + 2 * 2.0 ** -16) * off + 64 * E * size
    assert ((out.double() - want).abs() <= inner + U * (want.abs() + inner)).all()
    empty = hidden.all(1)
    assert (lse[empty] == -torch.inf).all() and (out[empty] == 0).all()
    assert ((lse.double() - want_lse)[~empty].abs() <= 2.0 ** -16 + 16 * E * 8).all()


def caches(pages, requests, max_pages, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    cache = torch.randn(pages, 64, 576, device=DEV, generator=g).bfloat16()
    table = torch.randint(0, pages, (requests, max_pages), device=DEV, generator=g).int()
    return g, cache, table


def test_most_ragged_rows_over_selections(gpu):
    """65535 rows of 4096 requests, a third of them without rows."""
    announce("sparse_attention 65535 ragged rows")
    rows, requests, heads, k = 65535, 4096, 2, 3
    g, cache, table = caches(300, requests, 4, 1)
    q = (torch.randn(rows, heads, 576, device=DEV, generator=g) * 0.7).bfloat16()
    idx = torch.randint(-60, 256, (rows, k), device=DEV, generator=g).int()
    counts = np.random.default_rng(2).multinomial(rows - 40, np.r_[np.full(2730, 1 / 2730), np.zeros(requests - 2730)])
    np.random.default_rng(3).shuffle(counts)
    cu = torch.from_numpy(20 + np.r_[0, np.cumsum(counts)]).int().to(DEV)
    out = torch.full((rows, heads, 512), 5.0, device=DEV, dtype=torch.bfloat16)
    lse = torch.full((rows, heads), 5.0, device=DEV)
    gpu.sparse_attention(q, cache, table, idx, 0, SCALE, out, lse, cu_q=cu)
    torch.cuda.synchronize()
    for x in (out, lse):
        assert (x[:20] == 5).all() and (x[-20:] == 5).all()
    owner = torch.repeat_interleave(torch.arange(requests), torch.from_numpy(counts)).to(DEV)
    for a in range(20, rows - 20, 8192):
        b = min(a + 8192, rows - 20)
        at = idx[a:b].long()
        page = table[owner[a - 20:b - 20, None], at.clamp(min=0) // 64].long()
        check_rows(q[a:b], cache[page, at.clamp(min=0) % 64], at < 0, out[a:b], lse[a:b])


@pytest.mark.parametrize("heads,next_n", [(1, 15), (17, 15)])
def test_most_requests_over_pages(gpu, heads, next_n):
    """4096 requests of 15 rows (one short of the row limit), short contexts,
    windows of at most six keys."""
    announce(f"paged_attention 4096 requests of {next_n} rows, {heads} heads")
    requests, rows = 4096, 4096 * next_n
    g, cache, table = caches(300, requests, 3, 4)
    q = (torch.randn(rows, heads, 576, device=DEV, generator=g) * 0.7).bfloat16()
    ends = torch.randint(0, 193, (rows,), device=DEV, generator=g).int()
    starts = ends - torch.randint(0, 7, (rows,), device=DEV, generator=g).int()
    out = torch.full((rows, heads, 512), 5.0, device=DEV, dtype=torch.bfloat16)
    lse = torch.full((rows, heads), 5.0, device=DEV)
    gpu.paged_attention(q, cache, table, ends, next_n, SCALE, out, lse, row_starts=starts)
    torch.cuda.synchronize()
    owner = torch.arange(rows, device=DEV) // next_n
    for a in range(0, rows, 4096):
        b = min(a + 4096, rows)
        at = starts[a:b, None].clamp(min=0).long() + torch.arange(6, device=DEV)
        hidden = at >= ends[a:b, None]
        at = at.clamp(max=191)
        page = table[owner[a:b, None], at // 64].long()
        check_rows(q[a:b], cache[page, at % 64], hidden, out[a:b], lse[a:b])


def test_many_appended_tokens(gpu):
    """2^20 + 3 tokens in a call: far token numbers, every slot once."""
    announce("appends of 2^20 + 3 tokens")
    tokens, pages = (1 << 20) + 3, (1 << 14) + 1
    g = torch.Generator(DEV).manual_seed(6)
    kv = torch.randn(tokens, 576, device=DEV, generator=g).bfloat16()
    slots = torch.randperm(pages * 64, device=DEV, generator=g)[:tokens].int()
    at = torch.zeros(tokens, dtype=torch.int32, device=DEV)
    rope = torch.cat([torch.ones(1, 32), torch.zeros(1, 32)], 1).to(DEV)  # no rotation
    cache = torch.zeros(pages, 64, 576, dtype=torch.bfloat16, device=DEV)
    gpu.latent_append(kv, at, slots, rope, cache)
    want = torch.zeros_like(cache.view(-1, 576))
    want[slots.long()] = kv
    assert torch.equal(cache.view(-1, 576), want)
    k = kv[:, :128]  # rows 576 apart
    codes = torch.zeros(pages, 64, 128, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(pages, 64, device=DEV)
    gpu.index_k_append(k, at, slots, rope, codes, scales)
    scale = k.float().abs().amax(1) / torch.full((), 448.0, device=DEV)
    assert torch.equal(scales.view(-1)[slots.long()], scale)
    got = codes.view(-1, 128)[slots.long()].view(torch.float8_e4m3fn).float()
    assert torch.equal(got, (k.float() / scale[:, None]).to(torch.float8_e4m3fn).float())


def test_captured_decode_steps(gpu):
    """A decode step -- latent rows appended, attention over pages, prefix and
    selection -- captured once without workspaces of the caller's, replayed with
    new rows and lengths in its buffers, eager work in between: every replay
    gives the eager bits."""
    announce("captured decode step")
    requests, heads = 5, 16
    g, cache, table = caches(40, requests, 6, 8)
    table = torch.randperm(40, device=DEV, generator=g)[:30].view(requests, 6).int()
    table[:, 0] = table[0, 0]
    rope = torch.randn(400, 64, device=DEV, generator=g)
    kv = torch.zeros(requests, 576, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(requests, heads, 576, dtype=torch.bfloat16, device=DEV)
    pos, slots, lens = (torch.zeros(requests, dtype=torch.int32, device=DEV) for _ in range(3))
    idx = torch.zeros(requests, 100, dtype=torch.int32, device=DEV)
    outs = [torch.zeros(requests, heads, 512, dtype=torch.bfloat16, device=DEV) for _ in range(3)]

    def step():
        gpu.latent_append(kv, pos, slots, rope, cache)
        gpu.paged_attention(q, cache, table, lens, 1, SCALE, outs[0])
        gpu.shared_prefix_attention(q, cache, table, lens, 1, 1, SCALE, outs[1])
        gpu.sparse_attention(q, cache, table, idx, 1, SCALE, outs[2])

    def fill(i):
        h = torch.Generator(DEV).manual_seed(100 + i)
        kv.copy_(torch.randn(kv.shape, device=DEV, generator=h))
        q.copy_(torch.randn(q.shape, device=DEV, generator=h))
        pos.copy_(torch.randint(64, 384, (requests,), device=DEV, generator=h))
        slots.copy_(table[torch.arange(requests, device=DEV), (pos // 64).long()] * 64 + pos % 64)
        lens.copy_(pos + 1)
        idx.copy_(torch.randint(-5, 384, idx.shape, device=DEV, generator=h) % lens[:, None])

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    before = cache.clone()
    for i in range(1, 5):
        fill(i)
        cache.copy_(before)
        step()
        torch.cuda.synchronize()
        want, want_cache = [o.clone() for o in outs], cache.clone()
        cache.copy_(before)
        for o in outs:
            o.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cache, want_cache)
        for o, w in zip(outs, want):
            assert torch.equal(o, w), f"replay {i}"
        before = want_cache
