"""Rows into the 4-bit latent cache and the rotation of queries on the GPU, at ragged
token counts, strided inputs, positions of one and several axes, both pairings and
all types: codes byte by byte against the CPU oracle, rotated values within the one
rounding that they take."""
import numpy as np
import pytest
import torch

import oracle as O
from tests.gpu_harness import DEV, announce
from tests.test_gpu_append import DTYPES, MAX_POS, live_of, make, rope_table

pytestmark = pytest.mark.gpu
L = O.latent
ROW4 = 400
AXES = {1: [0] * 32, 2: [i % 2 for i in range(32)], 3: [0] * 8 + [1] * 12 + [2] * 12, 4: [3, 0, 2, 1] * 8}


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def positions_of(axes, tokens, seed):
    """Among them negative ones and ones past the table, which are clamped."""
    rng = np.random.default_rng(seed)
    p = rng.integers(0, MAX_POS, (axes, tokens)).astype(np.int32)
    p[:, 0], p[-1, -1] = 0, MAX_POS - 1
    if tokens > 3:
        p[0, 1], p[-1, 2] = -7, MAX_POS + 100
    return p


def rounded_once(got, x, rows, interleaved, dtype):
    """got against the rotation of x: half a step of the type (fp16: of its
    subnormals too), and what float64 loses of the definition itself, 2^-52 of the
    two products."""
    want = L.rotate(x, rows, interleaved)
    room = L.HALF_STEP[dtype] * np.abs(want) + 2.0 ** -50 * np.abs(x).max() + (2.0 ** -25 if dtype == "fp16" else 0.0)
    assert (np.abs(got - want) <= room).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tokens,wide,skip", [(1, 0, 0), (7, 8, 2), (64, 0, 0), (1003, 24, 4)])
def test_latent_rows_in_4_bits(gpu, tokens, wide, skip, dtype, interleaved):
    announce(f"latent_append_mxfp4 {tokens} {dtype} interleaved={interleaved}")
    kv, pos, slots, pages = make(tokens, 576, dtype, 61 + tokens, wide, skip=skip)
    kv[:, 100:400] *= 37.0  # blocks of very different sizes
    kv[:, 40:50] *= 0.001
    table = rope_table()
    cache = torch.full((pages, 64, ROW4), 0x5A, dtype=torch.uint8, device=DEV)
    gpu.latent_append_mxfp4(kv, pos, slots, dev(table), cache, interleaved)
    other = torch.zeros(pages, 64, 576, dtype=DTYPES[dtype], device=DEV)
    gpu.latent_append(kv, pos, slots, dev(table), other, interleaved)
    torch.cuda.synchronize()
    at, where = live_of(slots, pages)
    want = np.full((pages * 64, ROW4), 0x5A, np.uint8)
    want[where, :272] = L.mxfp4_key(kv[:, :512].float().cpu().numpy()[at])
    # the rotated part is that of the 16-bit row, bit by bit
    want[where, 272:] = other.view(torch.uint8).cpu().numpy().reshape(-1, 1152)[where, 1024:]
    assert np.array_equal(cache.cpu().numpy().reshape(-1, ROW4), want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_special_latent_rows(gpu, dtype):
    """Zeros, subnormal and largest values, ties of the codes, infinities and NaN in a
    block and in the rotated part; a bad block leaves its neighbours alone."""
    announce(f"latent_append_mxfp4 special rows {dtype}")
    t, info = DTYPES[dtype], torch.finfo(DTYPES[dtype])
    kv = torch.randn(10, 576, generator=torch.Generator().manual_seed(5)).to(t)
    kv[0] = 0
    kv[1, :512] = info.max
    kv[2, :512] = info.smallest_normal * 2.0 ** -4 * torch.arange(512).remainder(16)
    kv[3, :32] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 7.75] * 2)
    kv[4, 70] = float("nan")
    kv[5, 511] = float("-inf")
    kv[6, 0] = float("inf")
    kv[7, 530] = float("nan")
    kv[8, 575] = float("inf")
    kv[9, :512] = -kv[9, :512].abs()
    kv[9, ::7] = -0.0
    table = rope_table()
    cache = torch.zeros(1, 64, ROW4, dtype=torch.uint8, device=DEV)
    pos, slots = torch.arange(10, dtype=torch.int32, device=DEV), torch.arange(10, dtype=torch.int32, device=DEV)
    gpu.latent_append_mxfp4(kv.to(DEV), pos, slots, dev(table), cache)
    torch.cuda.synchronize()
    got = cache.cpu().numpy()[0, :10]
    assert np.array_equal(got[:, :272], L.mxfp4_key(kv[:, :512].float().numpy()))
    values = L.latent_mxfp4_values(got, dtype)
    assert np.isnan(values[4, 64:96]).all() and np.isfinite(values[4, :64]).all() and np.isfinite(values[4, 96:]).all()
    assert np.isnan(values[7, 512:]).any() and np.isfinite(values[7, :512]).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("tokens", [1, 5, 16, 259])
def test_axis_rotations(gpu, tokens, axes, interleaved):
    """The composed table row by row, and the three appends that take it against the
    definition."""
    announce(f"axis_rotations {tokens} tokens {axes} axes")
    table, positions = rope_table(), positions_of(axes, tokens, tokens + axes)
    out = torch.full((tokens + 1, 64), 9.0, device=DEV)
    gpu.axis_rotations(dev(positions), gpu.axis_map(AXES[axes]), dev(table), out[:tokens])
    torch.cuda.synchronize()
    rows = L.axis_rows(table, positions, AXES[axes])
    assert np.array_equal(out[:tokens].cpu().numpy(), rows) and (out[tokens] == 9).all()
    kv, _, slots, pages = make(tokens, 576, "bf16", 3 + tokens)
    at = torch.arange(tokens, dtype=torch.int32, device=DEV)
    cache = torch.zeros(pages, 64, ROW4, dtype=torch.uint8, device=DEV)
    gpu.latent_append_mxfp4(kv, at, slots, out[:tokens], cache, interleaved)
    k, _, _, _ = make(tokens, 128, "fp16", 4 + tokens)
    codes = torch.zeros(pages, 64, 128, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(pages, 64, device=DEV)
    gpu.index_k_append(k, at, slots, out[:tokens], codes, scales, interleaved)
    torch.cuda.synchronize()
    where = slots.cpu().numpy()
    got = L.latent_mxfp4_values(cache.cpu().numpy().reshape(-1, ROW4)[where], "bf16")
    rounded_once(got[:, 512:], kv[:, 512:].double().cpu().numpy(), rows, interleaved, "bf16")
    want, want_scale = L.fp8_key(L.index_key(k.float().cpu().numpy(), rows, interleaved))
    assert np.array_equal(codes.cpu().numpy().reshape(-1, 128)[where], want)
    assert np.array_equal(scales.cpu().numpy().reshape(-1)[where], want_scale)


def query_places(layout, tokens, heads, dtype, g):
    """(x, out, in place): rows of 64 in tensors laid out in different ways."""
    wide = lambda *shape: (torch.randn(*shape, generator=g) * 3).to(DTYPES[dtype]).to(DEV)
    if layout == "packed":
        return wide(tokens, heads, 64), torch.full((tokens, heads, 64), 7.0, dtype=DTYPES[dtype], device=DEV)
    if layout == "slices":
        return (wide(tokens, heads, 192)[:, :, 128:],
                torch.full((tokens, heads, 576), 7.0, dtype=DTYPES[dtype], device=DEV)[:, :, 512:])
    if layout == "heads first":
        return (wide(heads, tokens, 64).transpose(0, 1),
                torch.full((heads, tokens, 72), 7.0, dtype=DTYPES[dtype], device=DEV)[:, :, 8:].transpose(0, 1))
    if layout == "broadcast":
        return wide(1, 1, 64).expand(tokens, heads, 64), torch.zeros(tokens, heads, 64, dtype=DTYPES[dtype], device=DEV)
    x = wide(tokens, heads, 576)[:, :, 512:]
    return x, x


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("layout", ["packed", "slices", "heads first", "broadcast", "in place"])
@pytest.mark.parametrize("tokens,heads,axes", [(1, 1, 1), (1, 128, 3), (3, 7, 2), (65, 16, 1), (33, 33, 4)])
def test_rotate_queries(gpu, tokens, heads, axes, layout, dtype, interleaved):
    announce(f"rotate_queries {tokens} x {heads} axes={axes} {layout} {dtype}")
    g = torch.Generator().manual_seed(tokens + heads)
    x, out = query_places(layout, tokens, heads, dtype, g)
    before = x.double().cpu().numpy()
    whole = None if layout != "slices" else out._base if out._base is not None else None
    table, positions = rope_table(), positions_of(axes, tokens, 8)
    at = dev(positions[0] if axes == 1 else positions)
    gpu.rotate_queries(x, at, dev(table), out, gpu.axis_map(AXES[axes]), interleaved)
    torch.cuda.synchronize()
    rows = L.axis_rows(table, positions, AXES[axes])[:, None]
    rounded_once(out.double().cpu().numpy(), before, rows, interleaved, dtype)
    if layout != "in place":
        assert np.array_equal(x.double().cpu().numpy(), before)
    if whole is not None:
        assert (whole[:, :, :512] == 7).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("tokens,axes,sliced", [(1, 1, False), (3, 3, True), (130, 4, True), (64, 1, False)])
def test_rotate_index_queries(gpu, tokens, axes, sliced, dtype, interleaved):
    announce(f"rotate_index_queries {tokens} axes={axes} {dtype}")
    g = torch.Generator().manual_seed(tokens)
    q = (torch.randn(tokens, 32, 160 if sliced else 128, generator=g) * 4).to(DTYPES[dtype]).to(DEV)[:, :, -128:]
    q[0, 0, 70], q[0, 1, 90], q[0, 2, 100] = 5000.0, -460.0, 0.001
    codes = torch.zeros(tokens, 32, 128, dtype=torch.uint8, device=DEV)
    table, positions = rope_table(), positions_of(axes, tokens, 9)
    at = dev(positions[0] if axes == 1 else positions)
    gpu.rotate_index_queries(q, at, dev(table), codes, gpu.axis_map(AXES[axes]), interleaved)
    torch.cuda.synchronize()
    rows = L.axis_rows(table, positions, AXES[axes])[:, None]
    want = L.e4m3_codes(L.index_key(q.float().cpu().numpy(), rows, interleaved))
    assert np.array_equal(codes.cpu().numpy(), want)


def test_index_queries_that_are_not_finite(gpu):
    announce("rotate_index_queries infinities and NaN")
    q = torch.ones(1, 32, 128, dtype=torch.bfloat16, device=DEV)
    q[0, 0, 80], q[0, 1, 80], q[0, 2, 80], q[0, 3, 5] = float("inf"), float("-inf"), float("nan"), float("nan")
    codes = torch.zeros(1, 32, 128, dtype=torch.uint8, device=DEV)
    at = torch.zeros(1, dtype=torch.int32, device=DEV)
    gpu.rotate_index_queries(q, at, dev(rope_table()), codes)
    torch.cuda.synchronize()
    v = codes.view(torch.float8_e4m3fn).float()[0]
    assert v[0, 80] == 448 and v[1, 80] == -448 and torch.isnan(v[2, 80])
    assert torch.isnan(v[3, [5, 37]]).all() and torch.isfinite(v[3, 64:]).all() and torch.isnan(v).sum() == 3


def test_a_captured_step_replays(gpu):
    """Positions composed, rows appended and queries rotated in one graph, its inputs
    changed between the replays, with eager work of the same calls in between."""
    announce("axis_rotations, latent_append_mxfp4, rotate_queries captured")
    tokens, heads, amap = 40, 16, gpu.axis_map(AXES[3])
    table = dev(rope_table())
    kv, _, slots, pages = make(tokens, 576, "bf16", 17)
    kv = kv.contiguous()
    at = torch.arange(tokens, dtype=torch.int32, device=DEV)
    positions = dev(positions_of(3, tokens, 1))
    q = torch.randn(tokens, heads, 576, device=DEV).to(torch.bfloat16)

    def step(rows, cache, out):
        gpu.axis_rotations(positions, amap, table, rows)
        gpu.latent_append_mxfp4(kv, at, slots, rows, cache)
        gpu.rotate_queries(q[:, :, 512:], positions, table, out, amap)

    def buffers():
        return (torch.zeros(tokens, 64, device=DEV), torch.zeros(pages, 64, ROW4, dtype=torch.uint8, device=DEV),
                torch.zeros(tokens, heads, 64, dtype=torch.bfloat16, device=DEV))

    mine, eager = buffers(), buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*mine)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*mine)
    for i in range(3):
        positions.copy_(dev(positions_of(3, tokens, 20 + i)))
        kv.mul_(-1.5)
        graph.replay()
        step(*eager)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(mine, eager))
