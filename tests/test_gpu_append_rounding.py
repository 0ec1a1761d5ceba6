"""Rotated values of the cache appends next to rounding borders, bit for bit:
what is rounded is the exact value of a c - b s and b c + a s (fractions here),
once, to nearest even."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from tests.gpu_harness import DEV, announce

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
BITS = {"bf16": 8, "fp16": 11, "fp32": 24}           # of the significand
LOWEST = {"bf16": -126, "fp16": -14, "fp32": -126}   # exponent of the smallest normal value


def nearest(x, kind):
    """The value of the type nearest to the fraction x, ties to even (no overflow)."""
    if x == 0:
        return 0.0
    a = abs(x)
    e = a.numerator.bit_length() - a.denominator.bit_length()
    if Fraction(2) ** e > a:
        e -= 1
    step = Fraction(2) ** (max(e, LOWEST[kind]) - BITS[kind] + 1)
    n = round(a / step)  # (Python rounds ties to even)
    return float(n * step) * (1 if x > 0 else -1)


def narrowed(y, kind):
    """float64 values rounded once to the type's bits (normal values)."""
    m, e = np.frexp(y)
    return np.ldexp(np.rint(m * 2.0 ** BITS[kind]), e - BITS[kind])


def border_pairs(kind, seed):
    """(a, b, c, s) whose a c - b s rounds otherwise by way of float32."""
    rng = np.random.default_rng(seed)
    n = 1 << 22
    t = DTYPES[kind]
    a, b = [torch.from_numpy(rng.standard_normal(n)).to(t).double().numpy() for _ in range(2)]
    angle = rng.uniform(-np.pi, np.pi, n)
    c, s = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    y = a * c.astype(np.float64) - b * s.astype(np.float64)
    off = np.nonzero((narrowed(y, kind) != narrowed(y.astype(np.float32).astype(np.float64), kind)) &
                     (np.abs(y) > 2.0 ** -10))[0]
    return a[off], b[off], c[off], s[off]


def test_nearest():
    """The rounding that the other tests go by, against the types' own."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal(500) * 2.0 ** rng.integers(-30, 10, 500)
    for kind, t in (("fp16", np.float16), ("fp32", np.float32)):
        assert [nearest(Fraction(float(v)), kind) for v in x] == x.astype(t).astype(np.float64).tolist()
    y = x[np.abs(x) > 2.0 ** -9].astype(np.float32)
    want = torch.from_numpy(y).bfloat16().double().tolist()
    assert [nearest(Fraction(float(v)), "bf16") for v in y] == want


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_latent_rows_are_rounded_once(gpu, kind, interleaved):
    announce(f"latent_append rounding borders {kind} interleaved={interleaved}")
    a, b, c, s = border_pairs(kind, 5)
    assert len(a) >= 10
    # next to a border by less than float64 holds: half-way values, a hair up and down
    half = 1 + 2.0 ** -BITS[kind]
    hair = 2.0 ** (-100 if kind == "bf16" else -24)
    for sign in (1, -1):
        for c1, s1 in ((half, 2.0 ** -60), (half + 2 * 2.0 ** (1 - BITS[kind]) / 2, 2.0 ** -60), (half, 0.0)):
            a, b = np.append(a, sign * 1.0), np.append(b, hair)
            c, s = np.append(c, np.float32(c1)), np.append(s, np.float32(s1))
            a, b = np.append(a, sign * 1.0), np.append(b, -hair)
            c, s = np.append(c, np.float32(c1)), np.append(s, np.float32(s1))
    rows = -(-len(a) // 32)
    fill = rows * 32 - len(a)
    a, b = [np.pad(x, (0, fill), constant_values=0.75).reshape(rows, 32) for x in (a, b)]
    c, s = [np.pad(x, (0, fill), constant_values=0.5).reshape(rows, 32) for x in (c, s)]
    x = np.zeros((rows, 576))
    if interleaved:
        x[:, 512::2], x[:, 513::2] = a, b
    else:
        x[:, 512:544], x[:, 544:] = a, b
    kv = torch.from_numpy(x).to(DTYPES[kind]).to(DEV)
    assert (kv.double().cpu().numpy() == x).all()
    table = torch.from_numpy(np.concatenate([c, s], 1).astype(np.float32)).to(DEV)
    at = torch.arange(rows, dtype=torch.int32, device=DEV)
    pages = -(-rows // 64)
    cache = torch.zeros(pages, 64, 576, dtype=DTYPES[kind], device=DEV)
    gpu.latent_append(kv, at, at, table, cache, interleaved)
    torch.cuda.synchronize()
    got = cache.view(-1, 576)[:rows, 512:].double().cpu().numpy()
    first, second = (got[:, 0::2], got[:, 1::2]) if interleaved else (got[:, :32], got[:, 32:])
    for r in range(rows):
        for i in range(32):
            fa, fb, fc, fs = (Fraction(float(v)) for v in (a[r, i], b[r, i], c[r, i], s[r, i]))
            assert first[r, i] == nearest(fa * fc - fb * fs, kind), (r, i)
            assert second[r, i] == nearest(fb * fc + fa * fs, kind), (r, i)


@pytest.mark.gpu
def test_index_keys_are_rounded_once(gpu):
    """A rotated float32 key half-way between two values but for a hair that
    float64 does not hold beside it: seen in the scale, max|y| / 448."""
    announce("index_k_append rounding borders")
    half = np.float32(1 + 2.0 ** -12)  # its square is 1 + 2^-11 + 2^-24: half-way
    cases = [(sign * half, hair, half, np.float32(2.0 ** -60)) for sign in (1, -1)
             for hair in (2.0 ** -40, -2.0 ** -40, 0.0)]
    k = np.zeros((len(cases), 128), np.float32)
    table = np.zeros((len(cases), 64), np.float32)
    for r, (a, b, c, s) in enumerate(cases):
        k[r, 3], k[r, 35], table[r, 3], table[r, 35] = a, b, c, s
    at = torch.arange(len(cases), dtype=torch.int32, device=DEV)
    kv = torch.zeros(1, 64, 128, dtype=torch.uint8, device=DEV)
    sc = torch.zeros(1, 64, device=DEV)
    gpu.index_k_append(torch.from_numpy(k).to(DEV), at, at, torch.from_numpy(table).to(DEV), kv, sc)
    torch.cuda.synchronize()
    for r, (a, b, c, s) in enumerate(cases):
        y = nearest(Fraction(float(a)) * Fraction(float(c)) - Fraction(float(b)) * Fraction(float(s)), "fp32")
        assert sc[0, r].item() == np.float32(abs(np.float32(y)) / np.float32(448)), (r, y)
    assert len(set(sc[0, :len(cases)].tolist())) == 2
