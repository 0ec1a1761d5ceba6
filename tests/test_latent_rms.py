"""The root-mean-square allowance of oracle/latent.py on the host: a plain
emulation of the attention (float32, running maximum, weights in 16 bits) stays
within it, and the same with weights of too few bits, a rescale left out or keys
left out does not."""
import numpy as np
import pytest
import torch

import oracle as O

L = O.latent
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
SCALE = 192 ** -0.5


def rounded(x, dtype):
    return torch.from_numpy(x).to(DTYPES[dtype]).float().numpy()


def emulate(q, keys, dtype, weights=None, skip=None, drop=None, raises=None):
    """One row in float32, 64 keys at a time.  raises [heads]: receives the last
    step at which each head's maximum was raised; skip [heads]: the step whose
    rescale is left out."""
    q, keys = q.astype(np.float32), keys.astype(np.float32)
    shift, room = (-16.0, 16.0) if dtype == "bf16" else (8.0, 6.0)
    heads = len(q)
    m, l = np.full(heads, -3e38, np.float32), np.zeros(heads, np.float32)
    acc = np.zeros((heads, 512), np.float32)
    for i in range(0, len(keys), 64):
        k = keys[i:i + 64]
        z = (q @ k.T) * np.float32(SCALE * np.log2(np.e))
        if drop is not None and i <= drop < i + 64:
            z[:, drop - i] = -np.inf
        top = z.max(1) - np.float32(shift)
        raised = np.where(top > m + np.float32(room), top, m)
        by = np.exp2(m - raised)
        if raises is not None and i:
            raises[by < 1] = i
        if skip is not None:
            by = np.where(skip == i, np.float32(1), by)
        m = raised
        p = rounded(np.exp2(z - m[:, None]), weights or dtype)
        acc = acc * by[:, None] + p @ k[:, :512]
        l = l * by + p.sum(1)
    return rounded(acc / l[:, None], dtype)


def data(dtype, seed, n, q_scale=1.0, growing=False):
    g = torch.Generator().manual_seed(seed)
    keys = torch.randn(n, 576, generator=g).to(DTYPES[dtype]).float()
    if growing:
        keys = (keys * (0.05 + 8.0 * torch.arange(n) / n)[:, None]).to(DTYPES[dtype]).float()
    q = (torch.randn(8, 576, generator=g) * q_scale).to(DTYPES[dtype]).float()
    return q.numpy(), keys.numpy()


def rms(out, want):
    return np.sqrt(((out.astype(np.float64) - want) ** 2).mean(1))


CASES = pytest.mark.parametrize("n,q_scale,growing", [(1, 1.0, False), (2, 1.0, False), (65, 1.0, False),
                                                      (333, 1.0, False), (4097, 2.0, False), (3000, 4.0, True),
                                                      (400, 4.0, True)])


@CASES
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_emulation_stays_within(dtype, n, q_scale, growing):
    q, keys = data(dtype, 3 + n, n, q_scale, growing)
    want, _, allowed, _ = L.attend_row_rms(q, keys, np.arange(n), SCALE, dtype=dtype)
    assert (rms(emulate(q, keys, dtype), want) <= allowed).all()


@pytest.mark.parametrize("n", [65, 333, 4097])
def test_weights_of_too_few_bits_show(n):
    q, keys = data("fp16", 3 + n, n, 0.5)
    want, _, allowed, _ = L.attend_row_rms(q, keys, np.arange(n), SCALE, dtype="fp16")
    assert (rms(emulate(q, keys, "fp16"), want) <= allowed).all()
    assert (rms(emulate(q, keys, "fp16", weights="bf16"), want) > 1.2 * allowed).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_a_rescale_left_out_shows(dtype):
    q, keys = data(dtype, 9, 640, 4.0, growing=True)
    want, _, allowed, _ = L.attend_row_rms(q, keys, np.arange(640), SCALE, dtype=dtype)
    last = np.zeros(8, int)
    assert (rms(emulate(q, keys, dtype, raises=last), want) <= allowed).all()
    assert (last > 0).all()
    # (some heads' sums before their last rescale are nothing beside those after it)
    assert (rms(emulate(q, keys, dtype, skip=last), want) > 3 * allowed).sum() >= 2


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_a_key_left_out_shows(dtype):
    q, keys = data(dtype, 11, 333)
    want, _, allowed, _ = L.attend_row_rms(q, keys, np.arange(333), SCALE, dtype=dtype)
    p = np.exp(SCALE * q.astype(np.float64) @ keys.T.astype(np.float64))
    heavy = int((p / p.sum(1, keepdims=True)).min(0).argmax())
    assert (rms(emulate(q, keys, dtype, drop=heavy), want) > allowed).any()
