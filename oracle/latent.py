"""Plain CPU oracle (numpy, float64) of the cache appends and of the attention
over the latent cache.

TEST INFRASTRUCTURE ONLY, like indexer_oracle.

* ``rotate``            -- the position rotation of 64 dimensions;
* ``fp8_key``, ``mxfp4_key`` -- codes and scales of one rotated index key;
* ``attend_row``        -- one row's attention over given keys, with the error
                           that float32 sums and 16-bit softmax weights allow.
"""

from __future__ import annotations

import numpy as np

from .indexer_oracle import decode_e4m3fn, e2m1_decode_table

LATENT_DIM = 512
ROPE_DIM = 64
LATENT_ROW = 576

# Half a step of each type relative to the value: finfo(t).eps / 2.
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


def rotate(x, table, interleaved):
    """x [..., 64] and table [..., 64] (32 cosines, 32 sines) -> float64."""
    x = np.asarray(x, np.float64)
    c, s = np.asarray(table, np.float64)[..., :32], np.asarray(table, np.float64)[..., 32:]
    y = np.empty_like(x)
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        y[..., 0::2] = a * c - b * s
        y[..., 1::2] = b * c + a * s
    else:
        a, b = x[..., :32], x[..., 32:]
        y[..., :32] = a * c - b * s
        y[..., 32:] = b * c + a * s
    return y


def index_key(k, table, interleaved):
    """The rotated index key, rounded once to float32."""
    k = np.asarray(k, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        return np.concatenate([rotate(k[..., :64], table, interleaved), k[..., 64:]], -1).astype(np.float32)


def _nearest_even(z, values):
    """Index of the nearest of the ascending ``values`` (magnitudes of codes
    0, 1, 2, ...) to each z >= 0; a tie goes to the even code, magnitudes above
    the last value to it."""
    z = np.asarray(z, np.float64)
    hi = np.clip(np.searchsorted(values, z, side="left"), 1, len(values) - 1)
    lo = hi - 1
    d_lo, d_hi = z - values[lo], values[hi] - z
    return np.where(d_lo < d_hi, lo, np.where(d_hi < d_lo, hi, np.where(lo % 2 == 0, lo, hi)))


_E4M3 = decode_e4m3fn(np.arange(127, dtype=np.uint8)).astype(np.float64)  # codes 0..126: 0 .. 448


def fp8_key(y):
    """(codes uint8 [..., 128], scale float32 [...]) of a rotated float32 key."""
    y = np.asarray(y, np.float32)
    bad = ~np.isfinite(y).all(-1)
    y = np.where(bad[..., None], np.float32(0), y)
    scale = (np.abs(y).max(-1) / np.float32(448)).astype(np.float32)
    by = np.where(scale > 0, scale, np.float32(1))
    z = (y / by[..., None]).astype(np.float32)
    codes = _nearest_even(np.abs(z), _E4M3).astype(np.uint8) | (np.signbit(z).astype(np.uint8) << 7)
    codes = np.where(bad[..., None], np.uint8(0), codes)
    return codes, np.where(bad, np.float32(np.nan), scale)


def mxfp4_key(y):
    """Packed [..., 68] uint8 token of a rotated float32 key."""
    y = np.asarray(y, np.float32)
    blocks = y.reshape(y.shape[:-1] + (4, 32)).astype(np.float64)
    bad = ~np.isfinite(blocks).all(-1)
    blocks = np.where(bad[..., None], 0.0, blocks)
    amax = np.abs(blocks).max(-1)
    power = np.where(amax > 0, np.frexp(np.where(amax > 0, amax, 1.0))[1] - 1 - 2, -127)
    power = np.maximum(power, -127)
    z = blocks * 2.0 ** -power[..., None].astype(np.float64)
    values = np.abs(np.asarray(e2m1_decode_table(), np.float64)[:8])
    codes = _nearest_even(np.abs(z), values).astype(np.uint8) | (np.signbit(z).astype(np.uint8) << 3)
    codes = np.where(bad[..., None], np.uint8(0), codes).reshape(y.shape)
    scale = np.where(bad, 255, power + 127).astype(np.uint8)
    return np.concatenate([codes[..., 0::2] | (codes[..., 1::2] << 4), scale], -1)


def attend_row(q, keys, at, scale, softcap=0.0, slopes=None, position=0, dtype="bf16"):
    """One row over its visible keys.

    q [heads, 576], keys [n, 576], at [n] logical positions.  Returns
    (out [heads, 512], lse [heads], out_bound, lse_bound) in float64.

    The bounds count what a float32 kernel with softmax weights in the cache's
    type may lose, u being half a step of that type and e one of float32:

      score     576 products summed in float32 (exact products: 16-bit
                factors): 576 e scale sum|q k|, plus 8 e |z| for the factor
                log2(e), the exponential's argument and the bias, plus 16 e
                softcap for tanh  =: dz
      weight    exp: 2 dz relative with its own 4 e; rounded: u relative
                (fp16: 2^-33 absolute for the smallest ones, which are kept
                2^8 above the value's own scale)
      sum       n e of sum p |v|, and n e of the normaliser
      output    u |out|
      lse       dz + (n + 8) e + 4 e |lse|
    """
    q, keys = np.asarray(q, np.float64), np.asarray(keys, np.float64)
    heads, n = q.shape[0], keys.shape[0]
    if n == 0:
        return (np.zeros((heads, LATENT_DIM)), np.full(heads, -np.inf), np.zeros((heads, LATENT_DIM)),
                np.zeros(heads))
    e, u = HALF_STEP["fp32"], HALF_STEP[dtype]
    z = scale * (q @ keys.T)
    dz = 576 * e * abs(scale) * (np.abs(q) @ np.abs(keys).T)
    if softcap:
        z = softcap * np.tanh(z / softcap)
        dz = dz + 16 * e * softcap
    if slopes is not None:
        far = np.asarray(slopes, np.float64)[:, None] * np.abs(position - np.asarray(at, np.float64))[None, :]
        z = z - far
        dz = dz + 4 * e * far
    dz = (dz + 8 * e * np.abs(z)).max(1)
    top = z.max(1, keepdims=True)
    w = np.exp(z - top)
    total = w.sum(1, keepdims=True)
    p = w / total
    out = p @ keys[:, :LATENT_DIM]
    spread = p @ np.abs(keys[:, :LATENT_DIM])
    lse = (top + np.log(total))[:, 0]
    tiny = n * 2.0 ** -33 * np.abs(keys[:, :LATENT_DIM]).max(0)[None, :] if dtype == "fp16" else 0.0
    rel = u + 4 * dz + (2 * n + 16) * e
    bound = u * np.abs(out) + rel[:, None] * spread + tiny + u * rel[:, None] * spread
    return out, lse, bound, dz + (n + 8) * e + 4 * e * np.abs(lse)


def attend_row_rms(q, keys, at, scale, softcap=0.0, slopes=None, position=0, dtype="bf16"):
    """attend_row's values with what their errors should amount to, instead of
    what they can at worst: (out, lse, rms allowance [heads], lse allowance
    [heads]).  The first allowance is of the root mean square over the 512
    dimensions of a head's error; u and e as in attend_row:

      output    rounded by up to u |out| in each dimension, evenly in between:
                u |out| / sqrt(3) over the dimensions
      weights   rounded by d_s, |d_s| <= u, in sum and divisor: the error vector
                is sum p_s d_s (v_s - out), and where the values of different
                keys are as good as orthogonal its square is at most
                u^2 sum p_s^2 |v_s - out|^2  (these two: root of the sum of squares)
      scores    a float32 sum of 576 terms t_i walks at random: its steps are
                rounded by e times partial sums of about sqrt(i) |t| / sqrt(576),
                together 24 e |t| / sqrt(2); twice that, 8 e |z| for the factors
                and the exponential, 16 e softcap for tanh =: dz_s, moving the
                output by sum p_s dz_s |v_s - out|
      sums      of n terms that walk at random too: (4 sqrt(n) + 16) e of
                |out| + sqrt(sum p_s^2 |v_s|^2); FP16's smallest weights are
                rounded by 2^-33 of the largest
      all       10 % more, for values that are not quite orthogonal
    """
    q, keys = np.asarray(q, np.float64), np.asarray(keys, np.float64)
    out, lse, _, _ = attend_row(q, keys, at, scale, softcap, slopes, position, dtype)
    heads, n = q.shape[0], keys.shape[0]
    if n == 0:
        return out, lse, np.zeros(heads), np.zeros(heads)
    e, u = HALF_STEP["fp32"], HALF_STEP[dtype]
    z = scale * (q @ keys.T)
    dz = 2 * 24 / 2 ** 0.5 * e * abs(scale) * np.sqrt(q ** 2 @ (keys ** 2).T)
    if softcap:
        z = softcap * np.tanh(z / softcap)
        dz = dz + 16 * e * softcap
    if slopes is not None:
        far = np.asarray(slopes, np.float64)[:, None] * np.abs(position - np.asarray(at, np.float64))[None, :]
        z = z - far
        dz = dz + 4 * e * far
    dz = dz + 8 * e * np.abs(z)
    p = np.exp(z - lse[:, None])
    v = keys[:, :LATENT_DIM]
    # |v_s - out_h|^2 of every key and head
    apart = np.maximum((v ** 2).sum(1)[None, :] - 2 * out @ v.T + (out ** 2).sum(1)[:, None], 0.0)
    size = np.sqrt((v ** 2).sum(1))
    walk = np.sqrt((out ** 2).sum(1)) + np.sqrt(p ** 2 @ size ** 2)
    tiny = n ** 0.5 * 2.0 ** -33 * p.max(1) * size.max() if dtype == "fp16" else 0.0
    rounding = u * np.sqrt((out ** 2).sum(1) / 3 + (p ** 2 * apart).sum(1))
    rest = (p * dz * np.sqrt(apart)).sum(1) + (4 * n ** 0.5 + 16) * e * walk + tiny
    allowed = 1.1 * (rounding + rest) / LATENT_DIM ** 0.5
    return out, lse, allowed, (p * dz).sum(1) + (4 * n ** 0.5 + 16) * e + 4 * e * np.abs(lse)
