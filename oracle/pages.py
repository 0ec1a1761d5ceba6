"""Plain CPU oracle of the care of cache pages: release, fork and compaction, one
request and one page after another, on Python lists.

TEST INFRASTRUCTURE ONLY, like indexer_oracle.
"""

from __future__ import annotations

PAGE = 64


def held(length, max_pages):
    return -(-max(0, min(length, PAGE * max_pages)) // PAGE)


def release(table, lens, ended, refs):
    """-> (lens, refs) after the requests with ended[b] have given up their pages."""
    lens, refs = list(lens), list(refs)
    for b, row in enumerate(table):
        if ended[b]:
            for page in row[:held(lens[b], len(row))]:
                if 0 <= page < len(refs):
                    refs[page] -= 1
            lens[b] = 0
    return lens, refs


def fork(table, lens, parents, refs):
    """-> (table, lens, refs, src, dst, tokens, [taken, without]).  Pages are taken
    before the shared ones are counted (which matters only where refs and table
    contradict each other: a page of the table without a holder)."""
    table, refs, after = [list(row) for row in table], list(refs), list(lens)
    n = len(lens)
    free = [p for p, r in enumerate(refs) if r <= 0]
    src, dst, tokens, without = [-1] * n, [-1] * n, [0] * n, 0
    taken = 0
    before = [list(row) for row in table]
    shared = []
    for b, p in enumerate(parents):
        if not 0 <= p < n or lens[b] > 0:
            continue
        length = max(0, min(lens[p], PAGE * len(table[p])))
        full, rest = divmod(length, PAGE)
        if rest and taken == len(free):
            without += 1
            continue
        for j in range(full):
            shared.append(before[p][j])
            table[b][j] = before[p][j]
        if rest:
            src[b], dst[b], tokens[b] = before[p][full], free[taken], rest
            taken += 1
            table[b][full] = dst[b]
            refs[dst[b]] = 1
        after[b] = length
    for page in shared:
        if 0 <= page < len(refs):
            refs[page] += 1
    return table, after, refs, src, dst, tokens, [taken, without]


def compact(table, lens, refs):
    """-> (table, refs, src, dst, [held pages, moves])."""
    live = sum(r > 0 for r in refs)
    src = [p for p in range(live, len(refs)) if refs[p] > 0]
    dst = [p for p in range(live) if refs[p] <= 0]
    assert len(src) == len(dst)
    to = dict(zip(src, dst))
    after = list(refs)
    for a, b in to.items():
        after[b], after[a] = refs[a], 0
    out = [[to.get(page, page) if j < held(lens[b], len(row)) else page for j, page in enumerate(row)]
           for b, row in enumerate(table)]
    pad = [-1] * (len(refs) - len(src))
    return out, after, src + pad, dst + pad, [live, len(src)]
