"""The 4-bit K/V cache, float64.  Test infrastructure only (see package doc).

A row of D values is cut into groups of 16.  With k the global scale (a power
of two) and a = max |x| / k over a group, the group's scale is the e4m3 value
nearest to a / 6 and each value is stored as the e2m1 value nearest to
x / k / s (both: halfway cases to the even code, values past the largest code
to the largest).  The cache stands for code * s * k.  A group with an infinity
or NaN has the NaN scale.  Searches among the codes' values, no rounding
arithmetic: independent of how a kernel converts.

A (block, kv head) tile: block_size rows of D/2 code bytes (element 2i in the
low nibble), block_size rows of D/16 scale bytes, zero padding to 16 bytes.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# e4m3 byte -> value for the finite non-negative bytes 0 .. 126; 127 is NaN
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)]
                + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:119])
NAN_SCALE = 127


def nearest(x: np.ndarray, levels: np.ndarray) -> np.ndarray:
    """Index of the level nearest to x >= 0 (halfway: the even index)."""
    mid = (levels[1:] + levels[:-1]) / 2
    lo = np.searchsorted(mid, x, side="left")
    hi = np.searchsorted(mid, x, side="right")
    return np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))


def quantise(x: np.ndarray, gscale: float):
    """[..., D] -> (code bytes [..., D/2], scale bytes [..., D/16]) uint8."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(*x.shape[:-1], -1, 16) / gscale
    bad = ~np.isfinite(g).all(axis=-1)
    g = np.where(bad[..., None], 0.0, g)
    si = nearest(np.abs(g).max(axis=-1) / 6.0, E4M3)
    s = E4M3[si][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        mag = np.where(s > 0, np.abs(g) / s, 0.0)
    code = nearest(mag, E2M1) + 8 * (g < 0)  # a zero, of either sign, is code 0
    code = np.where(bad[..., None], 0, code).reshape(x.shape).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), np.where(bad, NAN_SCALE, si).astype(np.uint8)


def dequantise(codes: np.ndarray, scales: np.ndarray, gscale: float) -> np.ndarray:
    """The float64 values that code and scale bytes stand for."""
    c = np.stack((codes & 15, codes >> 4), axis=-1).reshape(*codes.shape[:-1], -1)
    v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.concatenate((E4M3, [np.nan], -E4M3, [np.nan]))[scales] * gscale  # any byte (sign bit: never written)
    return (v.reshape(*v.shape[:-1], -1, 16) * s[..., None]).reshape(v.shape)


def tile_bytes(bs: int, d: int) -> int:
    return -(-bs * (d // 2 + d // 16) // 16) * 16


def rows(cache: np.ndarray, bs: int, d: int):
    """Views of a pool [NB, Hkv, tile]: codes [NB, Hkv, bs, D/2], scales [NB, Hkv, bs, D/16]."""
    n = bs * d // 2
    shape = cache.shape[:-1]
    return (cache[..., :n].reshape(*shape, bs, d // 2),
            cache[..., n:n + bs * d // 16].reshape(*shape, bs, d // 16))


def values(cache: np.ndarray, bs: int, d: int, gscale: float) -> np.ndarray:
    """The pool as float64 [NB, Hkv, bs, D]."""
    return dequantise(*rows(cache, bs, d), gscale)


def reshape_and_cache(x, cache: np.ndarray, slot_mapping, bs: int, gscale: float) -> None:
    """Quantise token t's rows ([T, Hkv, D]) into slot ``slot_mapping[t]``, in place."""
    d = x.shape[-1]
    n = bs * d // 2
    codes, scales = quantise(x, gscale)
    for t, s in enumerate(np.asarray(slot_mapping)):
        if s < 0:
            continue
        blk, off = divmod(int(s), bs)
        cache[blk, :, off * (d // 2):(off + 1) * (d // 2)] = codes[t]
        cache[blk, :, n + off * (d // 16):n + (off + 1) * (d // 16)] = scales[t]


def compact(token_rows: dict, start: int, keep) -> dict:
    """{position: row} of one sequence after its kept positions moved to
    ``start``, ``start + 1``, ...; other positions stay as they are."""
    out = dict(token_rows)
    for j, p in enumerate(keep):
        out[start + j] = token_rows[int(p)]
    return out
