"""The rotations of queries at their most tokens: the launch grid on the host, and calls
that reach beyond its first slab of tokens on the GPU."""
import pytest
import torch

from tests.gpu_harness import DEV, announce
from tests.test_host_logic import _build_and_run


def test_grids_stay_within_the_launch_limits(tmp_path):
    res = _build_and_run("rotate_grid_check.hip", tmp_path)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "mismatches 0" in res.stdout


POSITIONS = 1024


def table():
    angle = torch.arange(POSITIONS).double()[:, None] * 10000.0 ** (-torch.arange(32).double() / 32)
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(DEV)


def same_rows(out, want):
    """out[t] is want[t % POSITIONS], in pieces."""
    for at in range(0, len(out), 64 * POSITIONS):
        piece = out[at:at + 64 * POSITIONS]
        whole = len(piece) // POSITIONS * POSITIONS
        assert (piece[:whole].view(-1, *want.shape) == want).all(), at
        assert (piece[whole:] == want[:len(piece) - whole]).all(), at


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,heads", [(1 << 24, 1), ((1 << 24) - 1, 3), ((1 << 21) + 3, 33)])
def test_most_query_rows(gpu, tokens, heads):
    """One row of queries for all tokens (a token stride of 0), each turned by its own position."""
    announce(f"rotate_queries {tokens} x {heads}")
    x = torch.randn(1, heads, 64, generator=torch.Generator().manual_seed(heads)).bfloat16().to(DEV)
    rope, at = table(), torch.arange(tokens, dtype=torch.int32, device=DEV) % POSITIONS
    want = torch.empty(POSITIONS, heads, 64, dtype=torch.bfloat16, device=DEV)
    gpu.rotate_queries(x.expand(POSITIONS, heads, 64), at[:POSITIONS], rope, want)
    out = torch.full((tokens, heads, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    gpu.rotate_queries(x.expand(tokens, heads, 64), at, rope, out)
    torch.cuda.synchronize()
    same_rows(out, want)


@pytest.mark.gpu
def test_slabs_on_several_axes(gpu):
    """Tokens of a second launch: their positions on every axis, their rows, in and out."""
    tokens, heads, axis_of = (1 << 21) + 5, 2, [0] * 8 + [1] * 12 + [2] * 12
    announce(f"rotate_queries {tokens} x {heads} on three axes")
    g = torch.Generator().manual_seed(4)
    x = torch.randn(tokens, heads, 64, dtype=torch.bfloat16, device=DEV)
    rope, amap = table(), gpu.axis_map(axis_of)
    at = torch.randint(0, POSITIONS, (3, tokens), generator=g).int().to(DEV)
    out = torch.empty(tokens, heads, 64, dtype=torch.bfloat16, device=DEV)
    gpu.rotate_queries(x, at, rope, out, amap)
    want = torch.empty(40, heads, 64, dtype=torch.bfloat16, device=DEV)
    gpu.rotate_queries(x[-40:], at[:, -40:].contiguous(), rope, want, amap)
    torch.cuda.synchronize()
    assert torch.equal(out[-40:], want)


@pytest.mark.gpu
def test_most_index_rows(gpu):
    tokens = (1 << 21) + 3
    announce(f"rotate_index_queries {tokens}")
    q = torch.randn(1, 32, 128, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    rope, at = table(), torch.arange(tokens, dtype=torch.int32, device=DEV) % POSITIONS
    want = torch.empty(POSITIONS, 32, 128, dtype=torch.uint8, device=DEV)
    gpu.rotate_index_queries(q.expand(POSITIONS, 32, 128), at[:POSITIONS], rope, want)
    codes = torch.full((tokens, 32, 128), 9, dtype=torch.uint8, device=DEV)
    gpu.rotate_index_queries(q.expand(tokens, 32, 128), at, rope, codes)
    torch.cuda.synchronize()
    same_rows(codes, want)
