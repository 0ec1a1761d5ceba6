"""Timed cases of the paged cache appends and of the attention over the latent cache.

Four operators: the appends that rotate keys and write them into the paged caches
(index keys in FP8 or MXFP4 codes, latent rows in 16 bits), attention over a request's
pages with capped, biased or masked scores, the same for a batch that shares a long
prefix, and attention over the keys that the top-k selected.

``run`` computes a case in its plain form (elementary torch operations in 32 bits) or,
with ``own`` set, through the library's entry points; ``exact`` holds each operator's
definition in 64 bits.
"""

import math

import numpy as np
import torch

own = False

PAGE = 64          # tokens per cache page
INDEX_DIM = 128    # index key
LATENT = 512       # latent part of a cache row: the values
ROPE = 64          # rotated part
ROW = LATENT + ROPE
SCALE = 192 ** -0.5   # 128 unrotated + 64 rotated query dimensions per head
ROTATED_POSITIONS = 1 << 17
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of the headline batch: 8 new index keys
        dict(name="index append fp8, 8", op="index_append", codes="fp8", tokens=8, padding=0, dtype="bf16",
             interleaved=False, run_of=1),
        # an extend chunk's index keys, cut out of a wider projection, one token short of full pages
        dict(name="index append mxfp4, 8191", op="index_append", codes="mxfp4", tokens=8191, padding=0, dtype="fp16",
             interleaved=True, run_of=2048),
        # a verify step of 16 requests with 4 tokens each, the batch padded to 72
        dict(name="latent append, 72", op="latent_append", tokens=72, padding=8, dtype="bf16", interleaved=True,
             run_of=4),
        # four requests that extend by 2048 tokens each
        dict(name="latent append, 8192", op="latent_append", tokens=8192, padding=0, dtype="bf16", interleaved=False,
             run_of=2048),
        # the shortest useful decode: one request just past its first page
        dict(name="paged, 1 of 65", op="paged", heads=16, requests=1, rows=1, shortest=65, longest=65, dtype="bf16",
             softcap=0.0, bias=False, mask="causal", span=0),
        # a decode batch of very different lengths, capped scores with a distance bias, one padded request
        dict(name="paged, 64 varied", op="paged", heads=16, requests=64, rows=1, shortest=0, longest=32768,
             dtype="fp16", softcap=50.0, bias=True, mask="causal", span=0),
        # extend chunks of packed documents on cached prefixes
        dict(name="paged, extend documents", op="paged", heads=16, requests=4, rows=301, shortest=1000, longest=6500,
             dtype="bf16", softcap=0.0, bias=False, mask="document", span=1999),
        # a batch that continues one 32K prompt, all heads on this GPU
        dict(name="shared, 8 on 32K", op="shared", heads=128, requests=8, rows=1, prefix_pages=512, shortest=100,
             longest=2000, dtype="bf16", softcap=0.0, bias=False),
        # many samples of one short prompt, two tokens each to verify
        dict(name="shared, 32 on 2K", op="shared", heads=16, requests=32, rows=2, prefix_pages=33, shortest=1,
             longest=300, dtype="fp16", softcap=30.0, bias=False),
        # one decode row over a small selection
        dict(name="sparse, 1 of 4K", op="sparse", heads=16, requests=1, rows=1, selected=512, shortest=4096,
             longest=4096, dtype="bf16", softcap=0.0, bias=False),
        # the headline decode step: 8 requests of 128K keys, 2048 selected each
        dict(name="sparse, 8 of 128K", op="sparse", heads=128, requests=8, rows=1, selected=2048, shortest=131072,
             longest=131072, dtype="bf16", softcap=0.0, bias=False),
        # extend rows of four requests; the short request's rows see fewer keys than are asked for
        dict(name="sparse, extend 1024", op="sparse", heads=128, requests=4, rows=256, selected=2048, shortest=256,
             longest=30976, dtype="bf16", softcap=0.0, bias=False),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["index_append", "latent_append", "paged", "paged", "shared", "sparse", "sparse"])
    dtype = rng.choice(["bf16", "fp16"])
    if op.endswith("append"):
        tokens = log(1, 16384)
        case = dict(op=op, tokens=tokens, padding=min(tokens - 1, rng.choice([0, 0, 1, 7])), dtype=dtype,
                    interleaved=rng.random() < 0.5, run_of=rng.choice([1, 4, 512]))
        if op == "index_append":
            case.update(codes=rng.choice(["fp8", "mxfp4"]), dtype=rng.choice(["bf16", "fp16", "fp32"]))
        return case
    heads = rng.choice([1, 8, 16, 16, 24, 32, 64, 128, 128])
    case = dict(op=op, heads=heads, dtype=dtype, softcap=rng.choice([0.0, 0.0, 30.0]), bias=rng.random() < 0.3)
    if op == "paged":
        mask = rng.choice(["causal", "document", "prefix", "window"])
        requests, rows = log(1, 64), rng.choice([1, 1, 2, 4, log(5, 400)])
        most = max(64, min(32768, int(2e9 / (requests * rows * heads * 8))))
        longest = log(min(64, most), most)
        case.update(requests=requests, rows=rows, mask=mask, span=log(30, 3000),
                    shortest=rng.choice([0, 1, log(1, longest), longest]), longest=longest)
    elif op == "shared":
        requests, rows = log(2, 64), rng.choice([1, 1, 2, 4])
        most = max(1, min(1024, int(1e6 / (requests * rows * heads))))
        longest = log(1, 3000)
        case.update(requests=requests, rows=rows, prefix_pages=log(1, most), shortest=rng.choice([1, log(1, longest)]),
                    longest=longest)
    else:
        requests, rows = log(1, 16), rng.choice([1, 1, 4, log(5, 100)])
        case.update(requests=requests, rows=rows, selected=rng.choice([2048, 512, log(1, 2048)]),
                    shortest=rows + rng.choice([0, 0, 500]), longest=rows + log(501, 32768))
    return case


# --------------------------------------------------------------------------- inputs

def _lengths(case):
    """Keys of each request, spread evenly over the logarithm of the case's range."""
    n, lo, hi = case["requests"], case["shortest"], case["longest"]
    if n == 1:
        return [hi]
    spread = [math.exp(math.log(max(lo, 1)) + (math.log(max(hi, 1)) - math.log(max(lo, 1))) * i / (n - 1))
              for i in range(n)]
    return [lo] + [int(round(x)) for x in spread[1:-1]] + [hi]


def _ragged_rows(case):
    """Rows of each request: decode and verify batches have the same for all, extend chunks differ."""
    n, rows = case["requests"], case["rows"]
    return [rows] * n if not _ragged(case) else [max(1, rows - (i * 37) % rows) for i in range(n)]


def _ragged(case):
    return case["op"] == "paged" and case["rows"] > 4


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


def _rotation(device):
    """[positions, 64]: the cosines of 32 angles, then their sines."""
    at = torch.arange(ROTATED_POSITIONS, dtype=torch.float64, device=device)
    angle = at[:, None] * 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device=device) / ROPE)
    return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()


def _append_state(case, seed, device):
    g = torch.Generator(device).manual_seed(seed)
    tokens, live, run_of = case["tokens"], case["tokens"] - case["padding"], case["run_of"]
    dim = INDEX_DIM if case["op"] == "index_append" else ROW
    # the rows are cut out of a wider projection's output
    wide = torch.randn(tokens, 1536 + dim, device=device, generator=g).to(TYPES[case["dtype"]])
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
    positions = torch.zeros(tokens, dtype=torch.int32, device=device)
    positions[:live] = (history[r] + first[r] + j).clamp(max=ROTATED_POSITIONS - 1).int()
    s = dict(case=case, rows=wide[:, 1536:], slots=slots, positions=positions, rope=_rotation(device),
             live=torch.arange(live, device=device))
    if case["op"] == "latent_append":
        s["pages"] = torch.zeros(pages, PAGE, ROW, dtype=TYPES[case["dtype"]], device=device)
    elif case["codes"] == "fp8":
        s["pages"] = torch.zeros(pages, PAGE, INDEX_DIM, dtype=torch.uint8, device=device)
        s["scales"] = torch.zeros(pages, PAGE, device=device)
    else:
        s["pages"] = torch.zeros(pages, PAGE, 68, dtype=torch.uint8, device=device)
        codes = torch.arange(256, device=device)
        value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=device)
        s["pair"] = torch.stack([value[codes % 16], value[codes // 16]], 1)
        s["power"] = torch.exp2(codes.float() - 127)
    return s


def prepare(case, seed):
    device = torch.device("cuda")
    if case["op"].endswith("append"):
        return _append_state(case, seed, device)
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
    cache = torch.empty(pages, PAGE, ROW, dtype=dtype, device=device)
    for a in range(0, pages, 2048):
        cache[a:a + 2048] = torch.randn(cache[a:a + 2048].shape, device=device, generator=g).to(dtype)
    # queries lean towards a few of their request's keys, so that some rows are sharp and others flat
    q = torch.randn(rows, heads, ROW, device=device, generator=g)
    q *= 0.3 + 1.2 * torch.rand(rows, heads, 1, device=device, generator=g)
    i32 = dict(dtype=torch.int32, device=device)
    s = dict(case=case, q=q.to(dtype), cache=cache, table=table, ends=torch.tensor(end, **i32), starts=None,
             cu_q=torch.tensor(firsts, **i32) if _ragged(case) else None, positions=None, slopes=None,
             longest=longest, widest=max(counts), firsts=torch.tensor(firsts, device=device), indices=None,
             next_n=0 if _ragged(case) else case["rows"], prefix=prefix,
             row_request=torch.repeat_interleave(torch.arange(requests), torch.tensor(counts)).to(device))
    if case.get("mask") in ("document", "window"):
        s["starts"] = torch.tensor(start, **i32)
    if case["bias"]:
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, heads + 1, device=device) / heads)
        s["positions"] = torch.tensor(position, **i32)
    if case["op"] == "sparse":
        k = case["selected"]
        scores = torch.rand(rows, max(longest, k), device=device, generator=g)
        scores.masked_fill_(torch.arange(scores.shape[1], device=device) >= s["ends"][:, None], -1.0)
        best = scores.topk(k, dim=1)
        s["indices"] = torch.where(best.values < 0, -1, best.indices).int()
    s["out"] = torch.empty(rows, heads, LATENT, dtype=dtype, device=device)
    s["lse"] = torch.empty(rows, heads, device=device)
    if own:
        import paged_mqa_logits_indexer_amd as lib
        size = lib.shared_prefix_workspace_bytes if case["op"] == "shared" else lib.attention_workspace_bytes
        n = size(rows, heads, requests)
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=device)
    return s


# --------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    if op.endswith("append"):
        return _plain_append(s, op)
    return _plain_attention(s, op)


def _own(s, op):
    import paged_mqa_logits_indexer_amd as lib
    case = s["case"]
    if op == "latent_append":
        lib.latent_append(s["rows"], s["positions"], s["slots"], s["rope"], s["pages"], case["interleaved"])
        return s["pages"]
    if op == "index_append" and case["codes"] == "fp8":
        lib.index_k_append(s["rows"], s["positions"], s["slots"], s["rope"], s["pages"], s["scales"],
                           case["interleaved"])
        return s["pages"].view(torch.float8_e4m3fn), s["scales"]
    if op == "index_append":
        lib.index_k_append_mxfp4(s["rows"], s["positions"], s["slots"], s["rope"], s["pages"], case["interleaved"])
        return _mxfp4_values(s)
    options = dict(softcap=case["softcap"], slopes=s["slopes"], row_positions=s["positions"],
                   workspace=s["workspace"])
    if op == "paged":
        lib.paged_attention(s["q"], s["cache"], s["table"], s["ends"], s["next_n"], SCALE, s["out"], s["lse"],
                            cu_q=s["cu_q"], row_starts=s["starts"], **options)
    elif op == "shared":
        lib.shared_prefix_attention(s["q"], s["cache"], s["table"], s["ends"], s["next_n"], s["prefix"], SCALE,
                                    s["out"], s["lse"], **options)
    else:
        lib.sparse_attention(s["q"], s["cache"], s["table"], s["indices"], s["next_n"], SCALE, s["out"], s["lse"],
                             cu_q=s["cu_q"], **options)
    return s["out"], s["lse"]


def _mxfp4_values(s):
    """The appended tokens as the values that their codes and block scales stand for."""
    packed = s["pages"].view(-1, 68)[s["slots"][:len(s["live"])].long()].long()
    return (s["pair"][packed[:, :64]].view(-1, 4, 32) * s["power"][packed[:, 64:]][:, :, None]).view(-1, INDEX_DIM)


def _rotate(x, cos, sin, interleaved):
    a, b = (x[:, 0::2], x[:, 1::2]) if interleaved else (x[:, :32], x[:, 32:])
    a, b = a * cos - b * sin, b * cos + a * sin
    return torch.stack([a, b], 2).reshape(-1, ROPE) if interleaved else torch.cat([a, b], 1)


def _plain_append(s, op):
    case, live = s["case"], s["live"]
    x = s["rows"][live].double()
    table = s["rope"][s["positions"][live].long()].double()
    cos, sin = table[:, :32], table[:, 32:]
    slots = s["slots"][live].long()
    if op == "latent_append":
        y = torch.cat([x[:, :LATENT], _rotate(x[:, LATENT:], cos, sin, case["interleaved"])], 1)
        s["pages"].view(-1, ROW)[slots] = y.to(s["pages"].dtype)
        return s["pages"]
    # next to a code's border 32 bits decide otherwise than the definition: the rotation is rounded once
    y = torch.cat([_rotate(x[:, :ROPE], cos, sin, case["interleaved"]), x[:, ROPE:]], 1).float()
    if case["codes"] == "fp8":
        scale = y.abs().amax(1) / 448.0
        codes = (y / torch.where(scale > 0, scale, 1.0)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        s["pages"].view(-1, INDEX_DIM)[slots] = codes.view(torch.uint8)
        s["scales"].view(-1)[slots] = scale
        return s["pages"].view(torch.float8_e4m3fn), s["scales"]
    blocks = y.view(-1, 4, 32)
    power = (torch.frexp(blocks.abs().amax(2)).exponent - 3).clamp(-127, 127)
    z = torch.ldexp(blocks, -power[:, :, None]).view(-1, INDEX_DIM)
    # steps of 1/2 below 2, of 1 below 4, of 2 above; ties go to the even code
    m = z.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    m = (torch.round(m / step) * step).clamp(max=6.0)
    code = torch.where(m <= 2, 2 * m, torch.where(m <= 4, m + 2, m / 2 + 4)).to(torch.uint8)
    code = code + 8 * (z < 0).to(torch.uint8)
    packed = torch.cat([code[:, 0::2] + 16 * code[:, 1::2], (power + 127).to(torch.uint8)], 1)
    s["pages"].view(-1, 68)[slots] = packed
    return _mxfp4_values(s)


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


def _plain_attention(s, op):
    case, q, heads = s["case"], s["q"], s["case"]["heads"]
    rows, requests, ends = q.shape[0], case["requests"], s["ends"].long()
    pages = s["cache"].view(-1, ROW)
    position = s["positions"].long() if s["positions"] is not None else ends - 1
    out_dtype = q.dtype
    if op == "sparse":
        at = s["indices"].long()
        live = at >= 0
        at = at.clamp(min=0)
        slot = s["table"][s["row_request"][:, None], at // PAGE].long() * PAGE + at % PAGE
        keys = pages[slot].float()                                        # [rows, k, 576]
        scores = (q.float() @ keys.mT).view(rows, heads, -1)
        scores = _modify(scores, case, s["slopes"], position[:, None] - at)
        scores = scores.masked_fill(~live[:, None, :], -math.inf)
        out, lse = _softmax_sum(scores, [keys[..., :LATENT]])
        return out.to(out_dtype), lse
    # every request's rows as one block of the same height
    n = s["widest"]
    at = s["firsts"][:-1, None] + torch.arange(n, device=q.device)
    at = torch.minimum(at, s["firsts"][1:, None] - 1)
    starts = s["starts"].long() if s["starts"] is not None else torch.zeros_like(ends)
    prefix = s["prefix"] * PAGE
    key = torch.arange(s["longest"], device=q.device)
    slot = s["table"][:, key // PAGE].long() * PAGE + key % PAGE           # [requests, longest]
    blocks = q.float()[at].view(requests, n * heads, ROW)
    own_keys = pages[slot[:, prefix:]].float()
    scores = (blocks @ own_keys.mT).view(requests, n, heads, -1)
    if prefix:
        shared = pages[slot[0, :prefix]].float()
        first = (blocks.view(-1, ROW) @ shared.T).view(requests, n, heads, prefix)
        scores = torch.cat([first, scores], -1)
    scores = _modify(scores, case, s["slopes"], position[at][:, :, None] - key)
    hidden = (key < starts[at][:, :, None]) | (key >= ends[at][:, :, None])
    scores = scores.masked_fill(hidden[:, :, None, :], -math.inf).view(requests, n * heads, -1)
    values = [own_keys[..., :LATENT]]
    out, lse = _softmax_sum(scores, ([shared[:, :LATENT]] if prefix else []) + values)
    t = torch.arange(rows, device=q.device)
    b = s["row_request"]
    j = t - s["firsts"][b]
    return out.view(requests, n, heads, LATENT)[b, j].to(out_dtype), lse.view(requests, n, heads)[b, j]


# --------------------------------------------------------------------------- the definition

def exact(case, seed):
    """Each operator from its definition in 64 bits, request by request."""
    s = prepare(case, seed)
    if case["op"].endswith("append"):
        return _exact_append(s, case)
    if case["op"] == "sparse":
        return _exact_sparse(s, case)
    heads = case["heads"]
    out = torch.zeros(s["q"].shape[0], heads, LATENT, dtype=torch.float64, device="cuda")
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    first = s["firsts"].tolist()
    ends = s["ends"].tolist()
    starts = s["starts"].tolist() if s["starts"] is not None else [0] * len(ends)
    for b in range(case["requests"]):
        most = max(ends[first[b]:first[b + 1]])
        if not most:
            continue
        cache = s["cache"][s["table"][b, :-(-most // PAGE)].long()].reshape(-1, ROW)[:most].double()
        for r in range(first[b], first[b + 1]):
            keys = cache[starts[r]:ends[r]]
            if len(keys):
                at = torch.arange(starts[r], ends[r], device="cuda")
                out[r], lse[r] = _exact_row(s, case, r, keys, at, ends[r] - 1)
    return out, lse


def _exact_row(s, case, r, keys, at, position):
    z = torch.einsum("hd,sd->hs", s["q"][r].double(), keys) * SCALE
    if case["softcap"]:
        z = case["softcap"] * torch.tanh(z / case["softcap"])
    if s["slopes"] is not None:
        here = int(s["positions"][r]) if s["positions"] is not None else position
        z = z - s["slopes"].double()[:, None] * (here - at).abs()
    return torch.softmax(z, 1) @ keys[:, :LATENT], torch.logsumexp(z, 1)


def _exact_sparse(s, case):
    rows, heads = s["q"].shape[:2]
    out = torch.zeros(rows, heads, LATENT, dtype=torch.float64, device="cuda")
    lse = torch.full((rows, heads), -math.inf, dtype=torch.float64, device="cuda")
    pick, request = s["indices"].cpu(), s["row_request"].tolist()
    for r in range(rows):
        at = pick[r][pick[r] >= 0].long().cuda()
        if len(at):
            page = s["table"][request[r]].long()[torch.div(at, PAGE, rounding_mode="floor")]
            out[r], lse[r] = _exact_row(s, case, r, s["cache"][page, at % PAGE].double(), at, 0)
    return out, lse


def _exact_append(s, case):
    live = len(s["live"])
    x, where = s["rows"][:live].double(), s["slots"][:live].long()
    page, slot = where // PAGE, where % PAGE
    turn = s["rope"][s["positions"][:live].long()].double()
    wave = torch.complex(turn[:, :32], turn[:, 32:])
    part = x[:, LATENT:] if case["op"] == "latent_append" else x[:, :ROPE]
    if case["interleaved"]:
        turned = torch.view_as_real(torch.view_as_complex(part.reshape(live, 32, 2).contiguous()) * wave)
        turned = turned.reshape(live, ROPE)
    else:
        z = torch.complex(part[:, :32].contiguous(), part[:, 32:].contiguous()) * wave
        turned = torch.cat([z.real, z.imag], 1)
    if case["op"] == "latent_append":
        pages = torch.zeros(s["pages"].shape, dtype=torch.float64, device="cuda")
        pages[page, slot] = torch.cat([x[:, :LATENT], turned], 1)
        return pages
    y = torch.cat([turned, x[:, ROPE:]], 1)
    if case["codes"] == "fp8":
        pages = torch.zeros(s["pages"].shape, dtype=torch.float64, device="cuda")
        scales = torch.zeros(s["scales"].shape, dtype=torch.float64, device="cuda")
        scale = y.abs().max(1).values / 448
        scales[page, slot] = scale
        pages[page, slot] = (y / scale[:, None]).float().to(torch.float8_e4m3fn).double()
        return pages, scales
    blocks = y.view(live, 4, 32)
    power = torch.exp2(torch.floor(torch.log2(blocks.abs().max(2).values.float().double())) - 2)[:, :, None]
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    edge = (grid[1:] + grid[:-1]) / 2
    m = (blocks / power).float().double()
    low = torch.bucketize(m.abs(), edge)                 # a tie falls to the lower code ...
    odd = (low % 2 == 1) & (low < 7) & (m.abs() == edge[low.clamp(max=6)])
    value = grid[low + odd] * torch.sign(m) * power      # ... and goes up from an odd one
    return value.view(live, INDEX_DIM)


# --------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"].endswith("append"):
        live = case["tokens"] - case["padding"]
        size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
        if case["op"] == "latent_append":
            moved, flops = 2 * ROW * size, 6 * 32
        else:
            moved, flops = INDEX_DIM * size + (132 if case["codes"] == "fp8" else 68), 6 * 32 + 4 * INDEX_DIM
        return {"bytes": live * (moved + 8 + 4 * ROPE) + 8 * case["padding"], "flops": live * flops}
    start, end, _, counts = _row_ranges(case)
    heads, rows = case["heads"], len(end)
    bytes_ = rows * heads * (ROW * 2 + LATENT * 2 + 4) + 4 * rows
    if case["op"] == "sparse":
        seen = np.minimum(end, case["selected"])
        firsts = np.concatenate([[0], np.cumsum(counts)])
        read = sum(min(int(seen[a:b].sum()), int(end[a:b].max())) for a, b in zip(firsts[:-1], firsts[1:]))
        bytes_ += rows * case["selected"] * 4
    else:
        seen = end - start
        firsts = np.concatenate([[0], np.cumsum(counts)])
        prefix = case.get("prefix_pages", 0) * PAGE
        read = prefix + sum(max(0, int(end[a:b].max() - max(prefix, start[a:b].min())))
                            for a, b in zip(firsts[:-1], firsts[1:]))
    return {"bytes": int(bytes_ + read * ROW * 2), "flops": int(seen.sum()) * heads * 2 * (ROW + LATENT)}
