"""The tests of the attention over the 16-bit latent cache on 4-bit rows: batches whose
caches hold nothing but values that 4-bit rows hold, and a stand-in for the library
whose attention calls pack the cache and call the _mxfp4 entry points."""
import numpy as np
import torch

import oracle as O
from tests.test_gpu_attention import SCALE, Batch

E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def pack(cache):
    """uint8 [..., 400] of 16-bit rows [..., 576]; a block with a NaN or an infinity
    gets the byte 255."""
    x = cache[..., :512].float().reshape(*cache.shape[:-1], 16, 32)
    good = torch.isfinite(x).all(-1)
    x = torch.where(good[..., None], x, 0.0)
    power = (torch.frexp(x.abs().amax(-1)).exponent - 3).clamp(min=-127)
    m = torch.ldexp(x, -power[..., None]).abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))  # between the codes' values; ties to the even code
    m = (torch.round(m / step) * step).clamp(max=6.0)
    code = torch.where(m <= 2, 2 * m, torch.where(m <= 4, m + 2, m / 2 + 4)).to(torch.uint8)
    code = (code + 8 * torch.signbit(x).to(torch.uint8)).flatten(-2)
    byte = torch.where(good, power + 127, 255).to(torch.uint8)
    return torch.cat([code[..., 0::2] + 16 * code[..., 1::2], byte, cache[..., 512:].contiguous().view(torch.uint8)], -1)


def unpack(rows, dtype):
    """16-bit rows [..., 576] of uint8 [..., 400]."""
    table = E2M1.to(rows.device)
    codes = torch.stack([rows[..., :256] & 15, rows[..., :256] >> 4], -1).flatten(-2)
    power = rows[..., 256:272].float()
    scale = torch.where(power == 255, torch.nan, torch.exp2(power - 127))
    latent = table[codes.int()].view(*rows.shape[:-1], 16, 32) * scale[..., None]
    return torch.cat([latent.flatten(-2).to(dtype), rows[..., 272:].contiguous().view(dtype)], -1)


class Batch4(Batch):
    """A Batch whose cache is rounded to 4-bit rows whenever it is looked at."""

    @property
    def cache(self):
        if self._seen != self._cache._version:
            self._cache.copy_(unpack(pack(self._cache), self._cache.dtype))
            self._seen = self._cache._version
        return self._cache

    @cache.setter
    def cache(self, t):
        self._cache, self._seen = t, None


    def check(self, out, lse, softcap=0.0, slopes=None, positions=None, picked=None, rows=None):
        """Batch.check, with room for the weights that float32 ends below: 4-bit values
        are often exactly zero, and where those of all heavy keys are, nothing but
        such weights is left of an output.  A weight is taken under a maximum that
        stands at most 16 powers of two (FP16: 14, and a first one 8 below) over the
        row's largest score, and is zero below 2^-126: what is lost is below 2^-110 of
        the largest weight, which is at most 1 of the sum, times the value, for each
        key.  (FP16's own allowance for its smallest weights is far above that.)  For
        the same reason outputs come out below FP16's normal range, where half a step
        is 2^-25 whatever the value."""
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        cache = self.cache.view(-1, 576)
        for r in range(len(self.ends)) if rows is None else rows:
            at = self.visible(r) if picked is None else picked[r]
            if len(at) == 0:
                assert (out[r] == 0).all() and (lse[r] == -np.inf).all(), f"row {r} without keys"
                continue
            keys = cache[torch.from_numpy(self.slots(r, at))].double().numpy()
            pos = int(positions[r]) if positions is not None else int(self.ends[r]) - 1
            want, wl, ob, lb = O.latent.attend_row(self.q[r].double().numpy(), keys, at, SCALE, softcap, slopes, pos,
                                                   self.dtype)
            ob = ob + len(at) * 2.0 ** -110 * np.abs(keys[:, :512]).max() + (2.0 ** -25 if self.dtype == "fp16" else 0)
            bad = ~(np.abs(out[r] - want) <= ob)
            assert not bad.any(), (f"row {r} ({len(at)} keys): {bad.sum()} of {bad.size} outputs off, worst "
                                   f"{np.nanmax(np.abs(out[r] - want) / np.maximum(ob, 1e-300)):.2f} bounds, "
                                   f"{np.isnan(out[r]).sum()} NaN")
            assert (np.abs(lse[r] - wl) <= lb).all(), f"row {r} lse: {np.abs(lse[r] - wl).max()} over {lb.min()}"


class Packing:
    """The library, its attention calls over 4-bit rows of the cache they are given."""

    def __init__(self, lib):
        self.lib = lib

    def __getattr__(self, name):
        if name not in ("paged_attention", "shared_prefix_attention", "sparse_attention"):
            return getattr(self.lib, name)
        call = getattr(self.lib, name + "_mxfp4")
        return lambda q, cache, *args, **kw: call(q, pack(cache), *args, **kw)
