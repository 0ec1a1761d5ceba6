"""Attention over the latent cache where float32 comes near its ends: large and
small values under scores that rise along a request, one key that outweighs the
rest, and scores next to the lowest float32.  Scores are set through one rotated
dimension, values through the latent ones."""
import numpy as np
import pytest
import torch

import oracle as O
from tests.gpu_harness import DEV, announce
from tests.test_gpu_attention import DTYPES, SCALE, WIDE, Batch

pytestmark = pytest.mark.gpu
L = O.latent
# heads and table width: between them all four sizes of pair tiles
TILES = pytest.mark.parametrize("heads,width", [(16, 0), (32, WIDE), (64, WIDE), (128, WIDE)])
FORMS = pytest.mark.parametrize("form", ["paged", "shared", "sparse"])


def scored(seed, heads, lens, score, value, dtype="bf16", width=0, shared=0):
    """A batch of one-row requests whose key s of request r has the score
    (1 + h / 1024) * score(r, s) under head h, up to the rounding of the key, and
    whose values are value(r, s) times numbers in +-[1, 2)."""
    b = Batch(seed, heads, [1] * len(lens), lens, dtype=dtype, width=width, shared=shared)
    t = DTYPES[dtype]
    flat = b.cache.view(-1, 576)
    rng = np.random.default_rng(seed)
    for r, n in enumerate(lens):
        at = np.arange(shared * 64 if r else 0, n)
        rows = np.zeros((len(at), 576))
        rows[:, :512] = (rng.choice([-1.0, 1.0], (len(at), 512)) * rng.uniform(1, 2, (len(at), 512)) *
                         np.array([value(r, s) for s in at])[:, None])
        rows[:, 512] = [score(r, s) for s in at]
        flat[torch.from_numpy(b.slots(r, at))] = torch.from_numpy(rows).to(t)
    b.q = torch.zeros(len(lens), heads, 576, dtype=t)
    b.q[:, :, 512] = torch.tensor([(1 + h / 1024) / SCALE for h in range(heads)]).to(t)
    return b


def call(gpu, b, form, prefix=0, **kw):
    """One call of the given form on all keys of the batch's rows."""
    out, lse = b.out()
    head = (b.q.to(DEV), b.cache.to(DEV), b.dev(b.table))
    ends = b.dev(b.ends.astype(np.int32))
    if form == "paged":
        gpu.paged_attention(*head, ends, 1, SCALE, out, lse, **kw)
    elif form == "shared":
        gpu.shared_prefix_attention(*head, ends, 1, prefix, SCALE, out, lse, **kw)
    else:
        k = -(-int(b.ends.max()) // 64) * 64
        lists = np.full((len(b.ends), k), -1, np.int32)
        for r, n in enumerate(b.ends):
            lists[r, :n] = np.arange(n)
        gpu.sparse_attention(*head, b.dev(lists), 1, SCALE, out, lse, **kw)
    torch.cuda.synchronize()
    return out, lse


@FORMS
@TILES
@pytest.mark.parametrize("size", [1e-30, 1.0, 1e22, 1e30, 1e35])
def test_values_of_any_size(gpu, heads, width, size, form):
    """Values times keys that end well inside float32 come out, however far a
    later score rises over the first ones."""
    announce(f"{form} attention heads={heads} width={width} values of {size}")
    rises = [0.0, 3.3, 14.6, 17.1, 31.7, 58.9, 70.2, 120.4]  # powers of two
    lens = [200 + 3 * r for r in range(len(rises))]
    b = scored(201, heads, lens, lambda r, s: rises[r] * np.log(2) if s >= 150 else 0.0, lambda r, s: size,
               width=width, shared=1)
    out, lse = call(gpu, b, form, 1)
    assert torch.isfinite(out).all()
    b.check(out, lse)


@FORMS
@TILES
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_outweighing_key(gpu, dtype, heads, width, form):
    """One key outweighs the others by a fraction of a power of two more than a
    whole number, so that its softmax weight is not representable in 16 bits:
    the weight's rounding has to cancel in the quotient.

    Bound: with weights p_s (1 + d_s), |d_s| <= u = half a step of the type, in
    numerator and normaliser, the quotient is off by at most the sum of
    p_s |d_s| |v_s - out| / (1 - u); scores and exponentials are off by dz each;
    64 float32 roundings of the sums; then the output's own rounding.  The log
    of the sum does not see the weights' rounding."""
    announce(f"{form} attention heads={heads} width={width} {dtype} outweighing key")
    rises = [0.4, 1.3, 2.7, 5.5, 9.3, 12.4, 14.2, 15.7]  # powers of two
    lens = [140 + 9 * r for r in range(len(rises))]
    # (a key behind each live one lies in the same 16 keys of a step)
    live = {5: lambda r: 0.0, 69: lambda r: 0.0, 133: lambda r: rises[r] * np.log(2)}
    b = scored(211, heads, lens, lambda r, s: live[s](r) if s in live else -300.0, lambda r, s: 1.0, dtype, width, 1)
    out, lse = call(gpu, b, form, 1)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    e, u = L.HALF_STEP["fp32"], L.HALF_STEP[dtype]
    flat = b.cache.view(-1, 576)
    at = np.array(sorted(live))
    for r in range(len(lens)):
        keys = flat[torch.from_numpy(b.slots(r, at))].double().numpy()
        want, wl, _, _ = L.attend_row(b.q[r].double().numpy(), keys, at, SCALE, dtype=dtype)
        z = SCALE * (b.q[r].double().numpy() @ keys.T)
        p = np.exp(z - wl[:, None])
        dz = 8 * e * np.abs(z).max(1) + 8 * e
        off = (p[:, :, None] * np.abs(keys[None, :, :512] - want[:, None])).sum(1)
        inner = (1.01 * u + 2 * dz[:, None]) * off + 64 * e * (p @ np.abs(keys[:, :512]))
        bad = ~(np.abs(out[r] - want) <= inner + u * (np.abs(want) + inner))
        assert not bad.any(), f"row {r}: {bad.sum()} of {bad.size} outputs off"
        assert (np.abs(lse[r] - wl) <= 16 * e * (np.abs(z).max(1) + 16)).all()


@FORMS
@TILES
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_scores_next_to_the_lowest(gpu, dtype, heads, width, form):
    """Rows whose scores are all finite but lie in the last octave above the
    lowest float32: the nearest key under the steepest bias outweighs the rest."""
    announce(f"{form} attention heads={heads} width={width} {dtype} lowest scores")
    lens = [70, 1, 140, 65]
    b = scored(221, heads, lens, lambda r, s: 0.0, lambda r, s: 1.0, dtype, width, 1 if form == "shared" else 0)
    far = 1 << 20
    slopes = np.linspace(1.14e32, 2.2e32, heads).astype(np.float32)  # times the distance, in powers of two: 1.7e38 .. 3.3e38
    out, lse = call(gpu, b, form, 1, slopes=b.dev(slopes), row_positions=b.dev(np.full(len(lens), far, np.int32)))
    flat = b.cache.view(-1, 576)
    for r, n in enumerate(lens):
        key = flat[torch.from_numpy(b.slots(r, np.array([n - 1])))][0, :512]
        assert torch.equal(out[r].cpu(), key.expand(heads, 512)), f"row {r}"
        # float32 roundings of slope, distance, score, maximum and the way back
        want = -slopes.astype(np.float64) * (far - n + 1)
        assert (np.abs(lse[r].double().cpu().numpy() - want) <= 8 * L.HALF_STEP["fp32"] * np.abs(want)).all(), f"row {r}"


@FORMS
@TILES
@pytest.mark.parametrize("power", [20, 33, 66, 123])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_size(gpu, heads, width, sign, power, form):
    """Scores so large that float32's steps there are many powers of two: the
    keys of a row's largest score share all its weight, wherever they stand."""
    announce(f"{form} attention heads={heads} width={width} scores of {sign} * 2^{power}")
    lens = [333, 1, 70, 140, 200]
    score = lambda r, s: sign * 2.0 ** power * (1 + (37 * s % 128) / 128)  # a BF16 value, every 128 keys again
    b = scored(231, heads, lens, score, lambda r, s: 1.0, width=width, shared=1 if form == "shared" else 0)
    out, lse = call(gpu, b, form, 1)
    e, u = L.HALF_STEP["fp32"], L.HALF_STEP["bf16"]
    flat = b.cache.view(-1, 576)
    for r, n in enumerate(lens):
        at = np.arange(n)
        z = np.array([score(r, s) for s in at])
        top = flat[torch.from_numpy(b.slots(r, at[z == z.max()]))][:, :512].double().numpy()
        want = np.broadcast_to(top.mean(0), (heads, 512))
        bad = ~(np.abs(out[r].double().cpu().numpy() - want) <= u * np.abs(want) + 16 * e * np.abs(top).max(0))
        assert not bad.any(), f"row {r}: {bad.sum()} of {bad.size} outputs off"
        zh = SCALE * b.q[r, :, 512].double().numpy() * z.max()
        assert (np.abs(lse[r].double().cpu().numpy() - zh) <= 8 * e * np.abs(zh) + 2).all(), f"row {r}"
