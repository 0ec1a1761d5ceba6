"""Rotated queries bit for bit: each value is the exact a c - b s or b c + a s, rounded
once to nearest even -- next to rounding borders against fractions, and elsewhere
against the rotated part that latent_append writes for the same rows."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from tests.gpu_harness import DEV, announce
from tests.test_gpu_append import rope_table
from tests.test_gpu_append_rounding import BITS, DTYPES, border_pairs, nearest
from tests.test_gpu_rotary import AXES, dev, positions_of

pytestmark = pytest.mark.gpu


def border_rows(kind):
    """a, b, c, s [rows, 32]: results that rounding by way of float32 gets wrong, and
    half-way values a hair up, down and neither, by less than float64 holds."""
    a, b, c, s = border_pairs(kind, 7)
    half, hair = 1 + 2.0 ** -BITS[kind], 2.0 ** (-100 if kind == "bf16" else -24)
    more = [(sign * 1.0, side * hair, c1, s1) for sign in (1, -1) for side in (1, -1)
            for c1, s1 in ((half, 2.0 ** -60), (half + 2.0 ** (1 - BITS[kind]), 2.0 ** -60), (half, 0.0))]
    a, b, c, s = [np.concatenate([x, y]) for x, y in zip((a, b, c, s), zip(*more))]
    rows = -(-len(a) // 32)
    pad = lambda x, v: np.pad(x, (0, rows * 32 - len(x)), constant_values=v).reshape(rows, 32)
    return pad(a, 0.75), pad(b, 0.75), pad(c, 0.5).astype(np.float32), pad(s, 0.5).astype(np.float32)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_queries_next_to_borders(gpu, kind, interleaved, in_place):
    announce(f"rotate_queries rounding borders {kind} interleaved={interleaved} in_place={in_place}")
    a, b, c, s = border_rows(kind)
    rows, heads = len(a), 3
    x = np.zeros((rows, 64))
    if interleaved:
        x[:, 0::2], x[:, 1::2] = a, b
    else:
        x[:, :32], x[:, 32:] = a, b
    q = torch.from_numpy(x).to(DTYPES[kind]).to(DEV)[:, None].repeat(1, heads, 1)
    assert (q.double().cpu().numpy() == x[:, None]).all()
    out = q if in_place else torch.empty_like(q)
    gpu.rotate_queries(q, torch.arange(rows, dtype=torch.int32, device=DEV), dev(np.concatenate([c, s], 1)), out,
                       0, interleaved)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    first, second = (got[..., 0::2], got[..., 1::2]) if interleaved else (got[..., :32], got[..., 32:])
    for r in range(rows):
        for i in range(32):
            fa, fb, fc, fs = (Fraction(float(v)) for v in (a[r, i], b[r, i], c[r, i], s[r, i]))
            assert (first[r, :, i] == nearest(fa * fc - fb * fs, kind)).all(), (r, i)
            assert (second[r, :, i] == nearest(fb * fc + fa * fs, kind)).all(), (r, i)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes", [1, 3])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("tokens,heads", [(1, 128), (65, 16), (257, 33)])
def test_queries_are_what_the_append_writes(gpu, tokens, heads, kind, axes, interleaved):
    """Every head's row as a latent row of its own, at the same position."""
    announce(f"rotate_queries against latent_append {tokens} x {heads} {kind} axes={axes} interleaved={interleaved}")
    g = torch.Generator().manual_seed(tokens + heads)
    q = torch.randn(tokens, heads, 64, generator=g).to(DTYPES[kind]).to(DEV)
    table, positions = dev(rope_table()), positions_of(axes, tokens, 5)
    at, amap = dev(positions[0] if axes == 1 else positions), gpu.axis_map(AXES[axes])
    out = torch.empty_like(q)
    gpu.rotate_queries(q, at, table, out, amap, interleaved)
    turned = torch.empty(tokens, 64, device=DEV)
    gpu.axis_rotations(dev(positions), amap, table, turned)
    n = tokens * heads
    rows = torch.zeros(n, 576, dtype=DTYPES[kind], device=DEV)
    rows[:, 512:] = q.view(n, 64)
    cache = torch.zeros(-(-n // 64), 64, 576, dtype=DTYPES[kind], device=DEV)
    slots = torch.arange(n, dtype=torch.int32, device=DEV)
    gpu.latent_append(rows, slots // heads, slots, turned, cache, interleaved)
    torch.cuda.synchronize()
    assert torch.equal(out.view(n, 64).view(torch.int16), cache.view(-1, 576)[:n, 512:].contiguous().view(torch.int16))
