"""The attention's workspace: as large as its pieces need and no larger, also for
selections over 4-bit rows whose tiles are counted into it, up to the most rows."""
import numpy as np
import pytest
import torch

import oracle as O
import paged_mqa_logits_indexer_amd as pmqa
from tests.gpu_harness import DEV, announce
from tests.mxfp4_cache import pack

L = O.latent
SCALE = 192 ** -0.5


@pytest.mark.parametrize("rows,heads,requests,pairs", [(1, 1, 1, 16), (64, 16, 64, 16), (64, 17, 64, 32),
                                                       (16, 16, 4, 64), (8, 128, 8, 128), (65535, 16, 4096, 128),
                                                       (65535, 128, 1, 128), (4096, 16, 4096, 16)])
def test_size_is_that_of_the_pieces(rows, heads, requests, pairs):
    """256 join records of 32 bytes, and two pieces of 514 floats a pair for each of 256 workgroups."""
    need = pmqa.attention_workspace_bytes(rows, heads, requests)
    assert need == 256 * 32 + 2 * 256 * pairs * 514 * 4 and need <= 135_000_000


@pytest.mark.gpu
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("rows,heads", [(65535, 9), (32900, 16), (65535, 32), (20001, 64), (9001, 128)])
def test_counted_selections_stay_in_their_workspace(gpu, rows, heads, ragged):
    """Rows of every count of keys in a workspace of just the size, which held NaN before."""
    announce(f"sparse_attention_mxfp4 workspace rows={rows} heads={heads} ragged={ragged}")
    g = torch.Generator().manual_seed(rows)
    plain = torch.randn(4, 64, 576, generator=g).bfloat16()
    cache = pack(plain)
    keys = L.latent_mxfp4_values(cache.view(-1, 400).numpy(), "bf16")
    k = 192
    live = (torch.arange(rows) * 7) % (k + 1)
    lists = (torch.arange(rows)[:, None] * 5 + torch.arange(k) * 3) % 256
    lists = torch.where(torch.arange(k) < live[:, None], lists, -1).int()
    q = torch.randn(256, heads, 576, generator=g).bfloat16().to(DEV)[torch.arange(rows, device=DEV) % 256].contiguous()
    out = torch.empty(rows, heads, 512, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(rows, heads, device=DEV)
    need = gpu.attention_workspace_bytes(rows, heads, 1)
    whole = torch.full((need + (1 << 20),), 0xFF, dtype=torch.uint8, device=DEV)
    table = torch.arange(4, dtype=torch.int32, device=DEV).view(1, 4)
    gpu.sparse_attention_mxfp4(q, cache.to(DEV), table, lists.to(DEV), 0 if ragged else rows, SCALE, out, lse,
                               cu_q=torch.tensor([0, rows], dtype=torch.int32, device=DEV) if ragged else None,
                               workspace=whole[:need])
    torch.cuda.synchronize()
    assert (whole[need:] == 0xFF).all()
    assert torch.equal(torch.isneginf(lse).all(1).cpu(), live == 0) and not torch.isnan(out).any()
    edges = [r for r in (0, 1, 2, 4096, 8191, 16447, 16448, 32895, 32896, 32899, rows - 2, rows - 1) if r < rows]
    for r in edges + np.random.default_rng(rows).integers(0, rows, 12).tolist():
        n = int(live[r])
        at = lists[r, :n].numpy().astype(np.int64)
        got, got_lse = out[r].double().cpu().numpy(), lse[r].double().cpu().numpy()
        if n == 0:
            assert (got == 0).all()
            continue
        want, wl, ob, lb = L.attend_row(q[r].double().cpu().numpy(), keys[at], at, SCALE)
        assert (np.abs(got - want) <= ob).all() and (np.abs(got_lse - wl) <= lb).all(), r
