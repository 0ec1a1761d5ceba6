"""Appends to the paged caches on the GPU: FP8 index keys, packed MXFP4 index
keys and latent rows, code by code against the CPU oracle, at ragged token
counts, strided inputs, far positions, both pairings and all types; slots that
no token names keep what they held."""
import numpy as np
import pytest
import torch

import oracle as O
from tests.gpu_harness import DEV, announce

pytestmark = pytest.mark.gpu
L = O.latent

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
MAX_POS = 5000


def rope_table(n=MAX_POS, seed=3):
    rng = np.random.default_rng(seed)
    angle = rng.uniform(-np.pi, np.pi, (n, 32))
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def make(tokens, dim, dtype, seed, wide=0, pages=None, skip=0):
    """Rows cut out of a wider tensor, positions and distinct slots; the last
    ``skip`` tokens are padding with slots of no page."""
    g = torch.Generator().manual_seed(seed)
    full = (torch.randn(tokens, wide + dim + 16, generator=g) * 2).to(DTYPES[dtype])
    rows = full.to(DEV)[:, wide:wide + dim]
    pages = pages or -(-tokens // 64) + 2
    slots = torch.randperm(pages * 64, generator=g)[:tokens].int()
    if skip:
        slots[-skip:] = torch.tensor([-1, pages * 64, -(2 ** 31), 2 ** 31 - 1] * skip, dtype=torch.int64)[:skip].int()
    positions = torch.randint(0, MAX_POS, (tokens,), generator=g).int()
    positions[0], positions[-1] = 0, MAX_POS - 1
    return rows, positions.to(DEV), slots.to(DEV), pages


def live_of(slots, pages):
    s = slots.cpu().numpy().astype(np.int64)
    ok = (s >= 0) & (s < pages * 64)
    return np.nonzero(ok)[0], s[ok]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("tokens,wide,skip", [(1, 0, 0), (7, 8, 2), (16, 0, 0), (65, 1536, 1), (1003, 24, 4)])
def test_fp8_keys(gpu, tokens, wide, skip, dtype, interleaved):
    announce(f"index_k_append {tokens} {dtype} interleaved={interleaved}")
    k, pos, slots, pages = make(tokens, 128, dtype, 11 + tokens, wide, skip=skip)
    table = rope_table()
    kv = torch.full((pages, 64, 128), 0x5A, dtype=torch.uint8, device=DEV)
    sc = torch.full((pages, 64), -3.0, device=DEV)
    gpu.index_k_append(k, pos, slots, torch.from_numpy(table).to(DEV), kv, sc, interleaved)
    torch.cuda.synchronize()
    at, where = live_of(slots, pages)
    y = L.index_key(k.float().cpu().numpy()[at], table[pos.cpu().numpy()[at]], interleaved)
    codes, scale = L.fp8_key(y)
    want = np.full((pages * 64, 128), 0x5A, np.uint8)
    want_sc = np.full(pages * 64, -3.0, np.float32)
    want[where], want_sc[where] = codes, scale
    assert np.array_equal(kv.cpu().numpy().reshape(-1, 128), want)
    assert np.array_equal(sc.cpu().numpy().reshape(-1), want_sc)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("tokens,wide,skip", [(1, 0, 0), (7, 8, 2), (65, 1536, 1), (1003, 24, 4)])
def test_mxfp4_keys(gpu, tokens, wide, skip, dtype, interleaved):
    announce(f"index_k_append_mxfp4 {tokens} {dtype} interleaved={interleaved}")
    k, pos, slots, pages = make(tokens, 128, dtype, 21 + tokens, wide, skip=skip)
    table = rope_table()
    kv = torch.full((pages, 64, 68), 0x5A, dtype=torch.uint8, device=DEV)
    gpu.index_k_append_mxfp4(k, pos, slots, torch.from_numpy(table).to(DEV), kv, interleaved)
    torch.cuda.synchronize()
    at, where = live_of(slots, pages)
    want = np.full((pages * 64, 68), 0x5A, np.uint8)
    want[where] = L.mxfp4_key(L.index_key(k.float().cpu().numpy()[at], table[pos.cpu().numpy()[at]], interleaved))
    assert np.array_equal(kv.cpu().numpy().reshape(-1, 68), want)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tokens,wide,skip", [(1, 0, 0), (7, 8, 2), (64, 0, 0), (1003, 24, 4)])
def test_latent_rows(gpu, tokens, wide, skip, dtype, interleaved):
    announce(f"latent_append {tokens} {dtype} interleaved={interleaved}")
    kv, pos, slots, pages = make(tokens, 576, dtype, 31 + tokens, wide, skip=skip)
    table = rope_table()
    cache = torch.full((pages, 64, 576), 7.0, dtype=DTYPES[dtype], device=DEV)
    gpu.latent_append(kv, pos, slots, torch.from_numpy(table).to(DEV), cache, interleaved)
    torch.cuda.synchronize()
    at, where = live_of(slots, pages)
    x = kv.double().cpu().numpy()[at]
    want = np.full((pages * 64, 576), 7.0)
    want[where] = np.concatenate([x[:, :512], L.rotate(x[:, 512:], table[pos.cpu().numpy()[at]], interleaved)], 1)
    got = cache.double().cpu().numpy().reshape(-1, 576)
    assert np.array_equal(got[:, :512], want[:, :512])
    # rounded to float32 and from there to the type: half a step of each
    u = L.HALF_STEP[dtype] * (1 + 2.0 ** -11)
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0  # half a subnormal step
    assert (np.abs(got - want) <= u * np.abs(want) + tiny).all()
    untouched = np.setdiff1d(np.arange(pages * 64), where)
    assert (got[untouched] == 7.0).all()


def test_special_keys(gpu):
    """Zeros, values whose scale is subnormal or zero, the largest values, ties
    of both code types, infinities and NaN (in and out of the rotated half)."""
    announce("index appends of special keys")
    f = np.finfo(np.float32)
    k = np.zeros((16, 128), np.float32)
    k[1] = 1e-44
    k[2] = f.tiny * np.linspace(0.01, 3, 128)
    k[3, 64:] = f.max
    k[4, 100] = np.inf
    k[5, 3] = np.nan
    k[6, 40] = -np.inf
    k[7, 64:] = np.tile([448, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5], 8)
    k[8, 64:] = np.tile([-6, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5], 8)
    k[9, 64:96] = 7.0          # above the largest E2M1 value at this scale
    k[9, 96:] = 5.999
    k[10, 64:] = 2.0 ** -130
    k[11, 64:96] = 1.0         # three blocks of zeros beside one of ones
    k[12] = np.random.default_rng(0).standard_normal(128) * 1e38
    k[13, 64:] = np.float32(448) * (1 + np.arange(64) % 16 / 16 + 1 / 32) / 2  # E4M3 midpoints
    k[14, 64] = -0.0
    k[15, 64:] = 2.0 ** np.linspace(-20, 8, 64)
    table = rope_table()
    pos = np.arange(16, dtype=np.int32) * 3
    dev = [torch.from_numpy(x).to(DEV) for x in (k, pos, np.arange(16, dtype=np.int32), table)]
    kv = torch.zeros((1, 64, 128), dtype=torch.uint8, device=DEV)
    sc = torch.zeros((1, 64), device=DEV)
    mx = torch.zeros((1, 64, 68), dtype=torch.uint8, device=DEV)
    gpu.index_k_append(dev[0], dev[1], dev[2], dev[3], kv, sc)
    gpu.index_k_append_mxfp4(dev[0], dev[1], dev[2], dev[3], mx)
    torch.cuda.synchronize()
    y = L.index_key(k, table[pos], False)
    codes, scale = L.fp8_key(y)
    assert np.isnan(scale[4:7]).all()
    assert np.array_equal(sc.cpu().numpy()[0, :16], scale, equal_nan=True)
    assert np.array_equal(kv.cpu().numpy()[0, :16], codes)
    assert np.array_equal(mx.cpu().numpy()[0, :16], L.mxfp4_key(y))


def test_positions_are_clamped_and_far_slots(gpu):
    """Positions outside the table use its ends; slots past 2^31 bytes of cache."""
    announce("latent_append far slots")
    pages = 30000  # 2.2 GB
    cache = torch.zeros((pages, 64, 576), dtype=torch.bfloat16, device=DEV)
    kv = torch.randn(3, 576, device=DEV).bfloat16()
    table = rope_table()
    pos = torch.tensor([-5, MAX_POS + 9, 17], dtype=torch.int32, device=DEV)
    slots = torch.tensor([0, pages * 64 - 1, pages * 64 - 64], dtype=torch.int32, device=DEV)
    gpu.latent_append(kv, pos, slots, torch.from_numpy(table).to(DEV), cache)
    torch.cuda.synchronize()
    got = cache.view(-1, 576)[slots.long()].double().cpu().numpy()
    x = kv.double().cpu().numpy()
    want = np.concatenate([x[:, :512], L.rotate(x[:, 512:], table[[0, MAX_POS - 1, 17]], False)], 1)
    assert (np.abs(got - want) <= 2.0 ** -8 * (1 + 2.0 ** -11) * np.abs(want)).all()
    assert int((cache.view(-1, 576)[:, 0] != 0).sum()) == 3


def test_appended_keys_are_scored(gpu):
    """The caches that the appends write are the ones the logits read: FP8 and
    MXFP4 keys appended token by token, scored against the oracle on the same
    codes; an FP8 key with a NaN (scale NaN) is never selected.  The scale NaN
    of an MXFP4 block stands inside the product, whose ReLU max(0, NaN) is 0:
    that key's logit says nothing."""
    announce("append -> logits -> top-k")
    n = 200
    k, pos, _, _ = make(n, 128, "bf16", 77)
    k = k.clone()
    k[50, 100] = float("nan")
    table = rope_table()
    perm = torch.randperm(6, generator=torch.Generator().manual_seed(1))
    bt = perm[:4].int().view(1, 4).to(DEV)
    s = torch.arange(n)
    slots = (perm[s // 64] * 64 + s % 64).int().to(DEV)
    kv = torch.zeros((6, 64, 128), dtype=torch.uint8, device=DEV)
    sc = torch.zeros((6, 64), device=DEV)
    mx = torch.zeros((6, 64, 68), dtype=torch.uint8, device=DEV)
    rope = torch.from_numpy(table).to(DEV)
    for a, b in ((0, 1), (1, 150), (150, n)):
        gpu.index_k_append(k[a:b], pos[a:b], slots[a:b], rope, kv, sc)
        gpu.index_k_append_mxfp4(k[a:b], pos[a:b], slots[a:b], rope, mx)
    g = torch.Generator().manual_seed(5)
    q = torch.randn(1, 32, 128, generator=g).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    w = torch.rand(1, 32, generator=g).to(DEV)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    for pages, scales in ((kv, sc), (mx, None)):
        logits = torch.full((1, 256), 9.0, device=DEV)
        if scales is None:
            gpu.indexer_logits_mxfp4(q, pages, w, bt, lens, 1, logits)
        else:
            gpu.indexer_logits(q, pages, scales, w, bt, lens, 1, logits)
        idx = torch.full((1, 256), -7, dtype=torch.int32, device=DEV)
        gpu.topk_rows(logits, None, lens, 256, gpu.KEY_FP32, idx)
        torch.cuda.synchronize()
        args = (q.cpu().numpy(), pages.cpu().numpy(), None if scales is None else scales.cpu().numpy(),
                w.cpu().numpy(), bt.cpu().numpy(), 1, 0, np.arange(n))
        live = np.arange(n) != 50
        assert O.check_logits(logits.cpu().numpy()[0, :n][live], O.indexer_logits_at(*args)[live],
                              O.logits_error_bound_at(*args)[live]).all()
        chosen = idx.cpu().numpy()[0]
        if scales is not None:
            assert np.isnan(logits.cpu().numpy()[0, 50])
            assert set(chosen[chosen >= 0]) == set(range(n)) - {50}
        assert set(range(n)) - set(chosen) <= {50}
