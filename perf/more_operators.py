"""Timed cases of the latent cache in 4 bits, of the care of cache pages and of rotary
positions with several axes.

Four operators: the append that writes rows into the 4-bit latent cache, attention over
that cache (a request's pages, pages that a batch shares, the keys that the top-k
selected), the rotation of queries by positions of one or several axes, and the pages'
turnover (requests released and forked, a pool compacted) with the copies that it takes
in the caches of all layers.

``run`` computes a case in its plain form (elementary torch operations in 32 bits, 64
where a rounding border decides) or, with ``own`` set, through the library's entry
points; ``exact`` holds each operator's definition in 64 bits.
"""

import math

import numpy as np
import torch

own = False

PAGE = 64          # tokens per cache page
LATENT = 512       # latent part of a cache row: the values
ROPE = 64          # rotated part
ROW = LATENT + ROPE
CODES = LATENT // 2    # bytes of a 4-bit row: two E2M1 codes each, ...
BLOCKS = LATENT // 32  # ... a power of two for every 32 dimensions, and the rotated part in 16 bits
ROW4 = CODES + BLOCKS + 2 * ROPE
INDEX_HEADS, INDEX_DIM = 32, 128
SCALE = 192 ** -0.5   # 128 unrotated + 64 rotated query dimensions per head
ROTATED_POSITIONS = 1 << 17
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E2M1 = [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
# angles of each axis, in turn: text positions; time, height and width of image and video tokens
SECTIONS = {1: [32], 2: [16, 16], 3: [8, 12, 12], 4: [2, 10, 10, 10]}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # a verify step of 16 requests with 4 tokens each, the batch padded to 72
        dict(name="append, 72", op="append", tokens=72, padding=8, dtype="bf16", interleaved=True, run_of=4, axes=1),
        # an extend chunk of video tokens, one token short of full pages
        dict(name="append, 8191 of video", op="append", tokens=8191, padding=0, dtype="fp16", interleaved=False,
             run_of=2048, axes=3),
        # the shortest useful decode: one request just past its first page
        dict(name="paged, 1 of 65", op="attend", over="pages", heads=16, requests=1, rows=1, shortest=65, longest=65,
             dtype="bf16", softcap=0.0, bias=False, mask="causal", span=0),
        # a decode batch of very different lengths, capped scores with a distance bias, one padded request
        dict(name="paged, 64 varied", op="attend", over="pages", heads=16, requests=64, rows=1, shortest=0,
             longest=32768, dtype="fp16", softcap=50.0, bias=True, mask="causal", span=0),
        # a batch that continues one 32K prompt, all heads on this GPU
        dict(name="shared, 8 on 32K", op="attend", over="prefix", heads=128, requests=8, rows=1, prefix_pages=512,
             shortest=100, longest=2000, dtype="bf16", softcap=0.0, bias=False),
        # the headline decode step: 8 requests of 128K keys, 2048 selected each
        dict(name="sparse, 8 of 128K", op="attend", over="selection", heads=128, requests=8, rows=1, selected=2048,
             shortest=131072, longest=131072, dtype="bf16", softcap=0.0, bias=False),
        # extend rows of four requests; the short request's rows see fewer keys than are asked for
        dict(name="sparse, extend 512", op="attend", over="selection", heads=128, requests=4, rows=128, selected=2048,
             shortest=128, longest=30976, dtype="bf16", softcap=0.0, bias=False),
        # the queries of one decode step, each head's rotated part put beside its latent part
        dict(name="rotate, 8 rows", op="rotate", what="queries", tokens=8, heads=128, dtype="bf16", interleaved=True,
             axes=1),
        # the queries of an extend chunk of video tokens
        dict(name="rotate, 4096 of video", op="rotate", what="queries", tokens=4096, heads=128, dtype="bf16",
             interleaved=False, axes=3),
        # the indexer's queries of an extend chunk, to the 8-bit codes that it reads
        dict(name="rotate index, 4001", op="rotate", what="index", tokens=4001, heads=INDEX_HEADS, dtype="fp16",
             interleaved=False, axes=1),
        # samples of a few prompts start as others end
        dict(name="turnover, 64 requests", op="pages", step="turnover", requests=64, released=12, forked=24,
             longest=1500, spare=64, layers=8),
        # a pool whose requests came and went is made dense, to give its upper half away
        dict(name="compact, 1500 pages", op="pages", step="compact", requests=100, released=40, forked=0,
             longest=1900, spare=20, layers=8),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "attend", "attend", "attend", "attend", "rotate", "pages"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "append":
        tokens = log(1, 16384)
        return dict(op=op, tokens=tokens, padding=min(tokens - 1, rng.choice([0, 0, 1, 7])), dtype=dtype,
                    interleaved=rng.random() < 0.5, run_of=rng.choice([1, 4, 512]), axes=rng.choice([1, 1, 2, 3, 4]))
    if op == "rotate":
        what = rng.choice(["queries", "index"])
        heads = INDEX_HEADS if what == "index" else rng.choice([1, 7, 16, 32, 128])
        if what == "index":
            dtype = rng.choice(["bf16", "fp16", "fp32"])
        return dict(op=op, what=what, tokens=log(1, 8192 * 64 // max(heads, 64)), heads=heads, dtype=dtype,
                    interleaved=rng.random() < 0.5, axes=rng.choice([1, 2, 3, 4]))
    if op == "pages":
        requests = log(2, 200)
        step = rng.choice(["turnover", "compact"])
        released = rng.randint(0, requests // 2)
        return dict(op=op, step=step, requests=requests, released=released,
                    forked=rng.randint(0, requests // 3) if step == "turnover" else 0, longest=log(1, 1500),
                    spare=rng.choice([0, 3, 50]), layers=rng.choice([1, 2, 5]))
    heads = rng.choice([1, 8, 16, 16, 24, 32, 64, 128, 128])
    over = rng.choice(["pages", "pages", "prefix", "selection", "selection"])
    case = dict(op=op, over=over, heads=heads, dtype=dtype, softcap=rng.choice([0.0, 0.0, 30.0]),
                bias=rng.random() < 0.3)
    if over == "pages":
        mask = rng.choice(["causal", "document", "prefix", "window"])
        requests, rows = log(1, 64), rng.choice([1, 1, 2, 4, log(5, 400)])
        most = max(64, min(32768, int(1.5e9 / (requests * rows * heads * 8))))
        longest = log(min(64, most), most)
        case.update(requests=requests, rows=rows, mask=mask, span=log(30, 3000),
                    shortest=rng.choice([0, 1, log(1, longest), longest]), longest=longest)
    elif over == "prefix":
        requests, rows = log(2, 64), rng.choice([1, 1, 2, 4])
        most = max(1, min(1024, int(5e5 / (requests * rows * heads))))
        longest = log(1, 2500)
        case.update(requests=requests, rows=rows, prefix_pages=log(1, most), shortest=rng.choice([1, log(1, longest)]),
                    longest=longest)
    else:
        requests, rows = log(1, 16), rng.choice([1, 1, 4, log(5, 32)])
        case.update(requests=requests, rows=rows, selected=rng.choice([2048, 512, log(1, 2048)]),
                    shortest=rows + rng.choice([0, 0, 500]), longest=rows + log(501, 32768))
    return case


# --------------------------------------------------------------------------- inputs

def _rotation(device):
    """[positions, 64]: the cosines of 32 angles, then their sines."""
    at = torch.arange(ROTATED_POSITIONS, dtype=torch.float64, device=device)
    angle = at[:, None] * 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device=device) / ROPE)
    return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()


def _axis_of(axes):
    """The axis of each of the 32 angles."""
    return [a for a, n in enumerate(SECTIONS[axes]) for _ in range(n)]


def _axis_positions(case, first, device, g):
    """[axes, tokens] from the tokens' places in the text: time goes on with it, the others
    walk over rows and columns of frames."""
    place = first.long()
    if case["axes"] == 1:
        return place[None].int()
    others = [(place // 31 ** i + 17 * i) % 96 for i in range(1, case["axes"])]
    return torch.stack([place // 64] + others).int().contiguous()


def _mxfp4(x):
    """Packed codes [..., 256] and power bytes [..., 16] of float32 rows [..., 512]."""
    blocks = x.view(*x.shape[:-1], BLOCKS, 32)
    power = (torch.frexp(blocks.abs().amax(-1)).exponent - 3).clamp(-127, 127)
    z = torch.ldexp(blocks, -power[..., None]).view(x.shape)
    # steps of 1/2 below 2, of 1 below 4, of 2 above; ties go to the even code
    m = z.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    m = (torch.round(m / step) * step).clamp(max=6.0)
    code = torch.where(m <= 2, 2 * m, torch.where(m <= 4, m + 2, m / 2 + 4)).to(torch.uint8)
    code = code + 8 * torch.signbit(z).to(torch.uint8)
    return code[..., 0::2] + 16 * code[..., 1::2], (power + 127).to(torch.uint8)


def _parts(rows, dtype, pair):
    """Packed rows [n, 400] as float32 [n, 512] and the rotated part [n, 64]."""
    codes = pair[rows[:, :CODES].int()].view(-1, BLOCKS, 32)
    power = torch.exp2(rows[:, CODES:CODES + BLOCKS].float() - 127)
    return (codes * power[:, :, None]).view(-1, LATENT), rows[:, CODES + BLOCKS:].contiguous().view(TYPES[dtype])


def _values(rows, dtype, pair):
    """float32 [n, 576]."""
    latent, rotated = _parts(rows, dtype, pair)
    return torch.cat([latent, rotated.float()], 1)


def _pair_table(device):
    value, code = torch.tensor(E2M1, device=device), torch.arange(256, device=device)
    return torch.stack([value[code % 16], value[code // 16]], 1)


def _append_state(case, seed, device):
    g = torch.Generator(device).manual_seed(seed)
    tokens, live, run_of = case["tokens"], case["tokens"] - case["padding"], case["run_of"]
    # the rows are cut out of a wider projection's output; some dimensions are larger than others
    wide = torch.randn(tokens, 1536 + ROW, device=device, generator=g)
    wide *= torch.exp(torch.randn(1536 + ROW, device=device, generator=g))
    runs = -(-live // run_of)
    pages_of = -(-(run_of + PAGE - 1) // PAGE)
    pages = runs * pages_of + 3
    table = torch.randperm(pages, device=device, generator=g)[:runs * pages_of].view(runs, pages_of)
    first = torch.randint(0, PAGE, (runs,), device=device, generator=g)
    history = torch.randint(0, (ROTATED_POSITIONS - run_of) // PAGE, (runs,), device=device, generator=g) * PAGE
    i = torch.arange(live, device=device)
    r, j = i // run_of, i % run_of
    at = first[r] + j
    slots = torch.full((tokens,), -1, dtype=torch.int32, device=device)
    slots[:live] = (table[r, at // PAGE] * PAGE + at % PAGE).int()
    place = torch.zeros(tokens, dtype=torch.int64, device=device)
    place[:live] = (history[r] + first[r] + j).clamp(max=ROTATED_POSITIONS - 1)
    s = dict(case=case, rows=wide.to(TYPES[case["dtype"]])[:, 1536:], slots=slots, rope=_rotation(device),
             positions=_axis_positions(case, place, device, g), pair=_pair_table(device),
             axis_of=torch.tensor(_axis_of(case["axes"]), device=device),
             where=slots[:live].long(), tokens=torch.arange(tokens, dtype=torch.int32, device=device),
             table=torch.empty(tokens, ROPE, device=device),
             pages=torch.zeros(pages, PAGE, ROW4, dtype=torch.uint8, device=device))
    if own:
        import paged_mqa_logits_indexer_amd as lib
        s["axis_map"] = lib.axis_map(_axis_of(case["axes"]))
    return s


def _rotate_state(case, seed, device):
    g = torch.Generator(device).manual_seed(seed)
    tokens, heads, dtype = case["tokens"], case["heads"], TYPES[case["dtype"]]
    place = torch.randint(0, ROTATED_POSITIONS - tokens, (1,), device=device, generator=g)
    place = place + torch.arange(tokens, device=device)
    dim = INDEX_DIM if case["what"] == "index" else 192
    q = torch.randn(tokens, heads, dim, device=device, generator=g)
    q *= 0.3 + 3.0 * torch.rand(tokens, heads, 1, device=device, generator=g)
    s = dict(case=case, rope=_rotation(device), positions=_axis_positions(case, place, device, g),
             axis_of=torch.tensor(_axis_of(case["axes"]), device=device))
    if case["what"] == "index":
        s["q"] = q.to(dtype)
        s["out"] = torch.empty(tokens, heads, INDEX_DIM, dtype=torch.uint8, device=device)
    else:
        # the rotated part of the projection, and its place behind the latent part of the attention's queries
        s["q"] = q.to(dtype)[:, :, 128:]
        s["out"] = torch.zeros(tokens, heads, ROW, dtype=dtype, device=device)[:, :, LATENT:]
    if own:
        import paged_mqa_logits_indexer_amd as lib
        s["axis_map"] = lib.axis_map(_axis_of(case["axes"]))
    return s


def _page_lengths(case):
    """Tokens of the requests in use, spread evenly over their logarithm."""
    n = case["requests"] - case["forked"]
    return np.array([min(case["longest"], int(math.exp((i + 0.5) / n * math.log(case["longest"] + 1))))
                     for i in range(n)])


def _pages_state(case, seed, device):
    """A pool in use: requests' pages all over it, some prompts' first pages held by two requests,
    some requests ended."""
    rng = np.random.default_rng(seed)
    n, longest = case["requests"], case["longest"]
    lens = np.zeros(n, np.int64)
    idle, busy = np.split(rng.permutation(n), [case["forked"]])    # idle: no request yet, these are forked into
    lens[busy] = _page_lengths(case)
    busy.sort()
    need = -(-lens // PAGE)
    pages = int(need.sum()) + case["spare"]
    order = rng.permutation(pages)
    refs = np.zeros(pages, np.int64)
    table = rng.integers(0, pages, (n, -(-longest // PAGE) + 1))
    used = 0
    for b in busy:
        shared = 0
        if rng.random() < 0.3 and b != busy[0]:
            other = busy[rng.integers(0, np.searchsorted(busy, b))]
            shared = int(min(lens[b], lens[other]) // PAGE)
            table[b, :shared] = table[other, :shared]
        table[b, shared:need[b]] = order[used:used + need[b] - shared]
        used += need[b] - shared
        np.add.at(refs, table[b, :need[b]], 1)
    ended = np.zeros(n, np.int64)
    ended[rng.permutation(busy)[:case["released"]]] = 1
    staying = busy[ended[busy] == 0]
    parents = np.full(n, -1, np.int64)
    if len(staying) and len(idle):
        parents[idle] = rng.choice(staying, len(idle))
    if case["step"] == "compact":
        # the requests that ended are gone already
        for b in np.flatnonzero(ended):
            np.subtract.at(refs, table[b, :need[b]], 1)
        lens = lens * (1 - ended)
    g = torch.Generator(device).manual_seed(seed)
    caches = []
    for _ in range(case["layers"]):
        caches.append(torch.randint(0, 256, (pages, PAGE, ROW4), dtype=torch.uint8, device=device, generator=g))
        caches.append(torch.randint(0, 256, (pages, PAGE, INDEX_DIM), dtype=torch.uint8, device=device, generator=g))
        caches.append(torch.rand(pages, PAGE, device=device, generator=g))
    i32 = dict(dtype=torch.int32, device=device)
    s = dict(case=case, caches=caches, block_table=torch.tensor(table, **i32), lens=torch.tensor(lens, **i32),
             refs=torch.tensor(refs, **i32), ended=torch.tensor(ended, **i32), parents=torch.tensor(parents, **i32))
    if own:
        import paged_mqa_logits_indexer_amd as lib
        size = n if case["step"] == "turnover" else pages
        s.update(handle=lib.PageCaches(caches), lens_between=torch.empty(n, **i32), refs_between=torch.empty(pages, **i32),
                 new_lens=torch.empty(n, **i32), new_refs=torch.empty(pages, **i32), src=torch.empty(size, **i32),
                 dst=torch.empty(size, **i32), tokens=torch.empty(size, **i32), counts=torch.empty(2, **i32),
                 new_table=torch.empty(n, table.shape[1], **i32),
                 workspace=torch.empty(lib.pages_workspace_bytes(n, pages), dtype=torch.uint8, device=device))
    return s


def _lengths(case):
    """Keys of each request, spread evenly over the logarithm of the case's range."""
    n, lo, hi = case["requests"], case["shortest"], case["longest"]
    if n == 1:
        return [hi]
    spread = [math.exp(math.log(max(lo, 1)) + (math.log(max(hi, 1)) - math.log(max(lo, 1))) * i / (n - 1))
              for i in range(n)]
    return [lo] + [int(round(x)) for x in spread[1:-1]] + [hi]


def _ragged(case):
    return case["over"] == "pages" and case["rows"] > 4


def _ragged_rows(case):
    """Rows of each request: decode and verify batches have the same for all, extend chunks differ."""
    n, rows = case["requests"], case["rows"]
    return [rows] * n if not _ragged(case) else [max(1, rows - (i * 37) % rows) for i in range(n)]


def _row_ranges(case):
    """(first key, end of keys, position) of every row of the batch, and rows per request."""
    counts, lens = _ragged_rows(case), _lengths(case)
    prefix = case.get("prefix_pages", 0) * PAGE
    starts, ends, positions = [], [], []
    for n, length in zip(counts, lens):
        length += prefix
        # the request's rows are its last tokens; a request without keys is padding
        p = np.arange(length - n, length) if length >= n else np.arange(n)
        end = p + 1 if length else np.zeros(n, np.int64)
        start = np.zeros(n, np.int64)
        mask, span = case.get("mask", "causal"), case.get("span", 0)
        if mask == "document" and length:
            start = p // span * span
        elif mask == "window" and length:
            start = np.maximum(0, end - span)
        elif mask == "prefix" and length:
            end = np.minimum(np.maximum(end, span), max(length, n))
        starts.append(start)
        ends.append(end)
        positions.append(p)
    return [np.concatenate(x) for x in (starts, ends, positions)] + [counts]


def _attend_state(case, seed, device):
    g = torch.Generator(device).manual_seed(seed)
    dtype, heads, requests = TYPES[case["dtype"]], case["heads"], case["requests"]
    start, end, position, counts = _row_ranges(case)
    rows = len(end)
    firsts = np.concatenate([[0], np.cumsum(counts)])
    longest = max(int(end.max()), 1)
    need = [max(1, -(-int(end[a:b].max()) // PAGE)) for a, b in zip(firsts[:-1], firsts[1:])]
    prefix = case.get("prefix_pages", 0)
    max_pages = -(-longest // PAGE)
    pages = sum(need) - prefix * (requests - 1) + 3
    perm = torch.randperm(pages, device=device, generator=g).int()
    table = torch.zeros(requests, max_pages, dtype=torch.int32, device=device)
    used = prefix
    for b, n in enumerate(need):
        table[b, :prefix] = perm[:prefix]
        table[b, prefix:n] = perm[used:used + n - prefix]
        used += n - prefix
    # latent rows whose dimensions differ in size
    size = torch.exp(0.5 * torch.randn(ROW, device=device, generator=g))
    cache = torch.empty(pages, PAGE, ROW4, dtype=torch.uint8, device=device)
    for a in range(0, pages, 2048):
        x = torch.randn(min(2048, pages - a), PAGE, ROW, device=device, generator=g) * size
        cache[a:a + 2048, :, :CODES], cache[a:a + 2048, :, CODES:CODES + BLOCKS] = _mxfp4(x[..., :LATENT].contiguous())
        cache[a:a + 2048, :, CODES + BLOCKS:] = x[..., LATENT:].to(dtype).contiguous().view(torch.uint8)
    # some rows are sharp and others flat
    q = torch.randn(rows, heads, ROW, device=device, generator=g)
    q *= 0.3 + 1.2 * torch.rand(rows, heads, 1, device=device, generator=g)
    i32 = dict(dtype=torch.int32, device=device)
    s = dict(case=case, q=q.to(dtype), cache=cache, table=table, ends=torch.tensor(end, **i32), starts=None,
             cu_q=torch.tensor(firsts, **i32) if _ragged(case) else None, positions=None, slopes=None,
             longest=longest, widest=max(counts), firsts=torch.tensor(firsts, device=device), indices=None,
             next_n=0 if _ragged(case) else case["rows"], prefix=prefix, pair=_pair_table(device),
             row_request=torch.repeat_interleave(torch.arange(requests), torch.tensor(counts)).to(device))
    if case.get("mask") in ("document", "window"):
        s["starts"] = torch.tensor(start, **i32)
    if case["bias"]:
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, heads + 1, device=device) / heads)
        s["positions"] = torch.tensor(position, **i32)
    if case["over"] == "selection":
        k = case["selected"]
        scores = torch.rand(rows, max(longest, k), device=device, generator=g)
        scores.masked_fill_(torch.arange(scores.shape[1], device=device) >= s["ends"][:, None], -1.0)
        best = scores.topk(k, dim=1)
        s["indices"] = torch.where(best.values < 0, -1, best.indices).int()
    s["out"] = torch.empty(rows, heads, LATENT, dtype=dtype, device=device)
    s["lse"] = torch.empty(rows, heads, device=device)
    if own:
        import paged_mqa_logits_indexer_amd as lib
        bytes_of = lib.shared_prefix_workspace_bytes if case["over"] == "prefix" else lib.attention_workspace_bytes
        s["workspace"] = torch.empty(bytes_of(rows, heads, requests), dtype=torch.uint8, device=device)
    return s


def prepare(case, seed):
    device = torch.device("cuda")
    return {"append": _append_state, "rotate": _rotate_state, "pages": _pages_state,
            "attend": _attend_state}[case["op"]](case, seed, device)


# --------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"append": _own_append, "rotate": _own_rotate, "pages": _own_pages, "attend": _own_attend}[op](s)
    return {"append": _plain_append, "rotate": _plain_rotate, "pages": _plain_pages, "attend": _plain_attend}[op](s)


def _own_append(s):
    import paged_mqa_logits_indexer_amd as lib
    interleaved = s["case"]["interleaved"]
    if s["case"]["axes"] == 1:
        lib.latent_append_mxfp4(s["rows"], s["positions"][0], s["slots"], s["rope"], s["pages"], interleaved)
    else:
        lib.axis_rotations(s["positions"], s["axis_map"], s["rope"], s["table"])
        lib.latent_append_mxfp4(s["rows"], s["tokens"], s["slots"], s["table"], s["pages"], interleaved)
    return _appended(s)


def _appended(s):
    """The appended tokens as the values that their bytes stand for."""
    return _parts(s["pages"].view(-1, ROW4)[s["where"]], s["case"]["dtype"], s["pair"])


def _own_rotate(s):
    import paged_mqa_logits_indexer_amd as lib
    if s["case"]["what"] == "index":
        lib.rotate_index_queries(s["q"], s["positions"], s["rope"], s["out"], s["axis_map"], s["case"]["interleaved"])
        return s["out"].view(torch.float8_e4m3fn)
    lib.rotate_queries(s["q"], s["positions"], s["rope"], s["out"], s["axis_map"], s["case"]["interleaved"])
    return s["out"]


def _own_pages(s):
    import paged_mqa_logits_indexer_amd as lib
    if s["case"]["step"] == "turnover":
        lib.release_pages(s["block_table"], s["lens"], s["ended"], s["refs"], s["lens_between"], s["refs_between"])
        lib.fork_pages(s["block_table"], s["lens_between"], s["parents"], s["refs_between"], s["new_lens"],
                       s["new_refs"], s["src"], s["dst"], s["tokens"], s["counts"], workspace=s["workspace"])
        lib.copy_pages(s["handle"], s["src"], s["dst"], tokens=s["tokens"])
        return s["block_table"], s["new_lens"], s["new_refs"], s["src"], s["dst"], s["tokens"], s["caches"]
    lib.compact_pages(s["block_table"], s["lens"], s["refs"], s["new_table"], s["new_refs"], s["src"], s["dst"],
                      s["counts"], workspace=s["workspace"])
    lib.copy_pages(s["handle"], s["src"], s["dst"], count=s["counts"][1:])
    return s["new_table"], s["new_refs"], s["src"], s["dst"], s["counts"], s["caches"]


def _own_attend(s):
    import paged_mqa_logits_indexer_amd as lib
    case = s["case"]
    options = dict(softcap=case["softcap"], slopes=s["slopes"], row_positions=s["positions"],
                   workspace=s["workspace"])
    if case["over"] == "pages":
        lib.paged_attention_mxfp4(s["q"], s["cache"], s["table"], s["ends"], s["next_n"], SCALE, s["out"], s["lse"],
                                  cu_q=s["cu_q"], row_starts=s["starts"], **options)
    elif case["over"] == "prefix":
        lib.shared_prefix_attention_mxfp4(s["q"], s["cache"], s["table"], s["ends"], s["next_n"], s["prefix"], SCALE,
                                          s["out"], s["lse"], **options)
    else:
        lib.sparse_attention_mxfp4(s["q"], s["cache"], s["table"], s["indices"], s["next_n"], SCALE, s["out"],
                                   s["lse"], cu_q=s["cu_q"], **options)
    return s["out"], s["lse"]


# --------------------------------------------------------------------------- the plain forms

def _turn(x, table, interleaved):
    """x [..., 64] by cosines and sines [..., 64], in 64 bits."""
    x, cos, sin = x.double(), table[..., :32].double(), table[..., 32:].double()
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    a, b = a * cos - b * sin, b * cos + a * sin
    return torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)


def _table_rows(s):
    """[tokens, 64]: each angle's cosine and sine at the position on its axis."""
    at = s["positions"].long()[s["axis_of"]].T                         # [tokens, 32]
    angle = torch.arange(32, device=at.device)
    return torch.cat([s["rope"][at, angle], s["rope"][at, angle + 32]], 1)


def _plain_append(s):
    case = s["case"]
    live = len(s["where"])
    codes, power = _mxfp4(s["rows"][:live, :LATENT].float())
    rotated = _turn(s["rows"][:live, LATENT:], _table_rows(s)[:live], case["interleaved"])
    rotated = rotated.to(TYPES[case["dtype"]]).contiguous().view(torch.uint8)
    s["pages"].view(-1, ROW4)[s["where"]] = torch.cat([codes, power, rotated], 1)
    return _appended(s)


def _plain_rotate(s):
    q, table = s["q"], _table_rows(s)[:, None]
    if s["case"]["what"] == "queries":
        s["out"].copy_(_turn(q, table, s["case"]["interleaved"]))
        return s["out"]
    y = torch.cat([_turn(q[..., :ROPE], table, s["case"]["interleaved"]).float(), q[..., ROPE:].float()], -1)
    s["out"].copy_(y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    return s["out"].view(torch.float8_e4m3fn)


def _plain_pages(s):
    return _plain_turnover(s) if s["case"]["step"] == "turnover" else _plain_compact(s)


def _held(table, lens):
    """Which entries of the block table are pages of a request."""
    return torch.arange(table.shape[1], device=table.device) < ((lens + PAGE - 1) // PAGE)[:, None]


def _plain_turnover(s):
    table, n, pages = s["block_table"].long(), s["case"]["requests"], len(s["refs"])
    held = _held(table, s["lens"])
    gone = held & (s["ended"] != 0)[:, None]
    refs = s["refs"].long() - torch.bincount(table[gone], minlength=pages)
    lens = torch.where(s["ended"] != 0, 0, s["lens"])
    parent = s["parents"].long()
    of = parent.clamp(min=0)
    wanted = (parent >= 0) & (lens == 0)
    part = torch.where(wanted, lens[of] % PAGE, 0)
    free = torch.nonzero(refs == 0)[:, 0]
    rank = torch.cumsum((part > 0).long(), 0)
    forked = wanted & ((part == 0) | (rank <= len(free)))
    takes = forked & (part > 0)
    column = lens[of].long() // PAGE
    dst = torch.full((n,), -1, device=table.device)
    dst[takes] = free[rank[takes] - 1]
    src = torch.where(takes, table[of, column.clamp(max=table.shape[1] - 1)], -1)
    full = torch.arange(table.shape[1], device=table.device) < column[:, None]
    inherited = full & forked[:, None]
    new_table = torch.where(inherited, table[of], table)
    new_table[takes, column[takes]] = dst[takes]
    refs = refs + torch.bincount(new_table[inherited], minlength=pages)
    refs[dst[takes]] = 1
    lens = torch.where(forked, lens[of], lens)
    tokens = torch.where(takes, part, 0)
    s["block_table"].copy_(new_table)
    # rows of a page that the parent's last page holds
    slot = torch.arange(PAGE, device=table.device)
    rows = slot < tokens[takes][:, None]
    to, at = (dst[takes][:, None] * PAGE + slot)[rows], (src[takes][:, None] * PAGE + slot)[rows]
    for cache in s["caches"]:
        flat = cache.view(pages * PAGE, -1)
        flat[to] = flat[at]
    i32 = torch.int32
    return s["block_table"], lens.to(i32), refs.to(i32), src.to(i32), dst.to(i32), tokens.to(i32), s["caches"]


def _plain_compact(s):
    refs, table = s["refs"].long(), s["block_table"].long()
    live = refs > 0
    pages, n = len(refs), int(live.sum())
    at = torch.arange(pages, device=refs.device)
    src, dst = at[live & (at >= n)], at[~live & (at < n)]
    to = at.clone()
    to[src] = dst
    new_refs = refs.clone()
    new_refs[dst] = refs[src]
    new_refs[src] = 0
    new_table = torch.where(_held(table, s["lens"]), to[table], table)
    for cache in s["caches"]:
        cache[dst] = cache[src]
    pad = torch.full((pages - len(src),), -1, device=refs.device)
    counts = torch.tensor([n, len(src)], device=refs.device)
    return tuple(x.int() for x in (new_table, new_refs, torch.cat([src, pad]), torch.cat([dst, pad]), counts)) + (
        s["caches"],)


def _softmax_sum(scores, parts):
    """Softmax over the last axis of the scores times each part's values, summed over the parts."""
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out, at = 0.0, 0
    for v in parts:
        n = v.shape[-2]
        out = out + p[..., at:at + n] @ v
        at += n
    return torch.where(total > 0, out / total, 0.0), (top + torch.log(total))[..., 0]


def _modify(scores, case, slopes, distance):
    """scores [..., rows, heads, keys], distance [..., rows, keys]"""
    scores = scores * SCALE
    if case["softcap"]:
        scores = case["softcap"] * torch.tanh(scores / case["softcap"])
    if slopes is not None:
        scores = scores - slopes[:, None] * distance.abs().unsqueeze(-2)
    return scores


def _plain_attend(s):
    case, q, heads = s["case"], s["q"], s["case"]["heads"]
    rows, requests, ends = q.shape[0], case["requests"], s["ends"].long()
    packed = s["cache"].view(-1, ROW4)
    position = s["positions"].long() if s["positions"] is not None else ends - 1
    if case["over"] == "selection":
        at = s["indices"].long()
        live = at >= 0
        at = at.clamp(min=0)
        slot = s["table"][s["row_request"][:, None], at // PAGE].long() * PAGE + at % PAGE
        keys = _values(packed[slot.flatten()], case["dtype"], s["pair"]).view(rows, -1, ROW)
        scores = (q.float() @ keys.mT).view(rows, heads, -1)
        scores = _modify(scores, case, s["slopes"], position[:, None] - at)
        scores = scores.masked_fill(~live[:, None, :], -math.inf)
        out, lse = _softmax_sum(scores, [keys[..., :LATENT]])
        return out.to(q.dtype), lse
    # every request's rows as one block of the same height
    pages = _values(packed, case["dtype"], s["pair"])
    n = s["widest"]
    at = s["firsts"][:-1, None] + torch.arange(n, device=q.device)
    at = torch.minimum(at, s["firsts"][1:, None] - 1)
    starts = s["starts"].long() if s["starts"] is not None else torch.zeros_like(ends)
    prefix = s["prefix"] * PAGE
    key = torch.arange(s["longest"], device=q.device)
    slot = s["table"][:, key // PAGE].long() * PAGE + key % PAGE           # [requests, longest]
    blocks = q.float()[at].view(requests, n * heads, ROW)
    own_keys = pages[slot[:, prefix:]]
    scores = (blocks @ own_keys.mT).view(requests, n, heads, -1)
    if prefix:
        shared = pages[slot[0, :prefix]]
        first = (blocks.view(-1, ROW) @ shared.T).view(requests, n, heads, prefix)
        scores = torch.cat([first, scores], -1)
    scores = _modify(scores, case, s["slopes"], position[at][:, :, None] - key)
    hidden = (key < starts[at][:, :, None]) | (key >= ends[at][:, :, None])
    scores = scores.masked_fill(hidden[:, :, None, :], -math.inf).view(requests, n * heads, -1)
    values = [own_keys[..., :LATENT]]
    out, lse = _softmax_sum(scores, ([shared[:, :LATENT]] if prefix else []) + values)
    b = s["row_request"]
    j = torch.arange(rows, device=q.device) - s["firsts"][b]
    return out.view(requests, n, heads, LATENT)[b, j].to(q.dtype), lse.view(requests, n, heads)[b, j]


# --------------------------------------------------------------------------- the definition

def exact(case, seed):
    """Each operator from its definition in 64 bits, request by request."""
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s, case)
    if case["op"] == "rotate":
        return _exact_rotate(s, case)
    if case["op"] == "pages":
        return _exact_turnover(s) if case["step"] == "turnover" else _exact_compact(s)
    heads, requests = case["heads"], s["row_request"].tolist()
    out = torch.zeros(s["q"].shape[0], heads, LATENT, dtype=torch.float64, device="cuda")
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    ends = s["ends"].tolist()
    starts = s["starts"].tolist() if s["starts"] is not None else [0] * len(ends)
    held, keys = -1, None
    for r, b in enumerate(requests):
        if case["over"] == "selection":
            at = s["indices"][r][s["indices"][r] >= 0].long()
            if len(at):
                page = s["table"][b].long()[torch.div(at, PAGE, rounding_mode="floor")]
                out[r], lse[r] = _exact_row(s, case, r, _exact_values(s["cache"][page, at % PAGE], case), at)
            continue
        if b != held:
            most = max(e for e, x in zip(ends, requests) if x == b)
            pages = s["cache"][s["table"][b, :-(-most // PAGE)].long()].reshape(-1, ROW4)[:most]
            held, keys = b, _exact_values(pages, case)
        if starts[r] < ends[r]:
            at = torch.arange(starts[r], ends[r], device="cuda")
            out[r], lse[r] = _exact_row(s, case, r, keys[starts[r]:ends[r]], at)
    return out, lse


def _exact_values(rows, case):
    """[n, 400] bytes -> [n, 576] in 64 bits, from the formats' bits."""
    code = torch.stack([rows[:, :CODES] & 15, rows[:, :CODES] >> 4], 2).reshape(-1, BLOCKS, 32).long()
    e, m = (code >> 1) & 3, (code & 1).double()
    size = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * 2.0 ** (e - 1).double())
    x = torch.where(code >= 8, -size, size) * 2.0 ** (rows[:, CODES:CODES + BLOCKS].double() - 127)[:, :, None]
    return torch.cat([x.view(-1, LATENT), rows[:, CODES + BLOCKS:].contiguous().view(TYPES[case["dtype"]]).double()], 1)


def _exact_row(s, case, r, keys, at):
    z = torch.einsum("hd,sd->hs", s["q"][r].double(), keys) * SCALE
    if case["softcap"]:
        z = case["softcap"] * torch.tanh(z / case["softcap"])
    if s["slopes"] is not None:
        z = z - s["slopes"].double()[:, None] * (int(s["positions"][r]) - at).abs()
    return torch.softmax(z, 1) @ keys[:, :LATENT], torch.logsumexp(z, 1)


def _exact_turned(s, case, part):
    """part [tokens, ..., 64] as complex numbers, angle by angle."""
    wave = torch.stack([torch.complex(s["rope"][s["positions"][a].long(), i].double(),
                                      s["rope"][s["positions"][a].long(), i + 32].double())
                        for i, a in enumerate(_axis_of(case["axes"]))], 1)
    wave = wave.view(len(wave), *[1] * (part.dim() - 2), 32)
    x = part.double()
    if case["interleaved"]:
        z = torch.view_as_complex(x.reshape(*x.shape[:-1], 32, 2).contiguous()) * wave
        return torch.view_as_real(z).flatten(-2)
    z = torch.complex(x[..., :32].contiguous(), x[..., 32:].contiguous()) * wave
    return torch.cat([z.real, z.imag], -1)


def _exact_append(s, case):
    live = len(s["where"])
    turned = _exact_turned(s, case, s["rows"][:, LATENT:])[:live]
    blocks = s["rows"][:live, :LATENT].double().reshape(live, BLOCKS, 32)
    power = torch.exp2(torch.floor(torch.log2(blocks.abs().max(2).values)) - 2)[:, :, None]
    grid = torch.tensor(E2M1[:8], dtype=torch.float64, device="cuda")
    edge = (grid[1:] + grid[:-1]) / 2
    m = blocks / power
    low = torch.bucketize(m.abs(), edge)                 # a tie falls to the lower code ...
    odd = (low % 2 == 1) & (low < 7) & (m.abs() == edge[low.clamp(max=6)])
    value = grid[low + odd] * torch.sign(m) * power      # ... and goes up from an odd one
    return value.view(live, LATENT), turned


def _exact_rotate(s, case):
    if case["what"] == "queries":
        return _exact_turned(s, case, s["q"])
    y = torch.cat([_exact_turned(s, case, s["q"][..., :ROPE]).float().double(), s["q"][..., ROPE:].double()], -1)
    m = y.abs().clamp(max=448.0)
    # three bits behind the leading one, steps of 2^-9 below 2^-6
    step = torch.exp2(torch.floor(torch.log2(m.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(y) * torch.round(m / step) * step


def _exact_turnover(s):
    table, lens, refs = s["block_table"].tolist(), s["lens"].tolist(), s["refs"].tolist()
    ended, parents = s["ended"].tolist(), s["parents"].tolist()
    n = len(lens)
    for b in range(n):
        if ended[b]:
            for j in range(-(-lens[b] // PAGE)):
                refs[table[b][j]] -= 1
            lens[b] = 0
    free = [p for p, held in enumerate(refs) if held == 0]
    src, dst, tokens, after = [-1] * n, [-1] * n, [0] * n, list(lens)
    for b, p in enumerate(parents):
        if p < 0 or lens[b]:
            continue
        full, rest = lens[p] // PAGE, lens[p] % PAGE
        if rest and not free:
            continue
        for j in range(full):
            table[b][j] = table[p][j]
            refs[table[p][j]] += 1
        if rest:
            src[b], dst[b], tokens[b] = table[p][full], free.pop(0), rest
            table[b][full] = dst[b]
            refs[dst[b]] = 1
        after[b] = lens[p]
    for cache in s["caches"]:
        for a, b, rest in zip(src, dst, tokens):
            if rest:
                cache[b, :rest] = cache[a, :rest]
    return tuple(torch.tensor(x, device="cuda") for x in (table, after, refs, src, dst, tokens)) + (s["caches"],)


def _exact_compact(s):
    table, lens, refs = s["block_table"].tolist(), s["lens"].tolist(), s["refs"].tolist()
    n = sum(r > 0 for r in refs)
    src = [p for p in range(n, len(refs)) if refs[p] > 0]
    dst = [p for p in range(n) if refs[p] == 0]
    moved = dict(zip(src, dst))
    for a, b in moved.items():
        refs[b], refs[a] = refs[a], 0
        for cache in s["caches"]:
            cache[b] = cache[a]
    for b, row in enumerate(table):
        for j in range(-(-lens[b] // PAGE)):
            row[j] = moved.get(row[j], row[j])
    pad = [-1] * (len(refs) - len(src))
    return tuple(torch.tensor(x, device="cuda") for x in (table, refs, src + pad, dst + pad, [n, len(src)])) + (
        s["caches"],)


# --------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "append":
        live = case["tokens"] - case["padding"]
        table = 4 * ROPE * live
        return {"bytes": live * (2 * ROW + ROW4 + 4 + 4 * case["axes"]) + table + 4 * case["padding"],
                "flops": live * (6 * 32 + 4 * LATENT)}
    if case["op"] == "rotate":
        elements = case["tokens"] * case["heads"] * (INDEX_DIM if case["what"] == "index" else ROPE)
        size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
        written = 1 if case["what"] == "index" else size
        return {"bytes": elements * (size + written) + case["tokens"] * (4 * ROPE + 4 * case["axes"]),
                "flops": case["tokens"] * case["heads"] * 6 * 32}
    if case["op"] == "pages":
        return _pages_work(case)
    start, end, _, counts = _row_ranges(case)
    heads, rows = case["heads"], len(end)
    bytes_ = rows * heads * (ROW * 2 + LATENT * 2 + 4) + 4 * rows
    firsts = np.concatenate([[0], np.cumsum(counts)])
    if case["over"] == "selection":
        seen = np.minimum(end, case["selected"])
        read = sum(min(int(seen[a:b].sum()), int(end[a:b].max())) for a, b in zip(firsts[:-1], firsts[1:]))
        bytes_ += rows * case["selected"] * 4
    else:
        seen = end - start
        prefix = case.get("prefix_pages", 0) * PAGE
        read = prefix + sum(max(0, int(end[a:b].max() - max(prefix, start[a:b].min())))
                            for a, b in zip(firsts[:-1], firsts[1:]))
    return {"bytes": int(bytes_ + read * ROW4), "flops": int(seen.sum()) * heads * 2 * (ROW + LATENT)}


def _pages_work(case):
    """Which requests end, fork and share pages is drawn with the inputs: the mean over that."""
    lens, layers = _page_lengths(case), case["layers"]
    need = -(-lens // PAGE)
    pages, row = int(need.sum()) + case["spare"], ROW4 + INDEX_DIM + 4
    book = 4 * (2 * case["requests"] * (-(-case["longest"] // PAGE) + 1) + 4 * case["requests"] + 2 * pages)
    if case["step"] == "turnover":
        return {"bytes": int(book + 2 * layers * row * (lens % PAGE).mean() * case["forked"]), "flops": 0}
    live = (len(lens) - min(case["released"], len(lens))) * need.mean()
    return {"bytes": int(book + 2 * layers * row * PAGE * live * (1 - live / pages)), "flops": 0}
