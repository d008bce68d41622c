"""A plain 64-bit model of the 8-bit cache, for the tests: e4m3 codes from the format's
definition (1 sign, 4 exponent bits with bias 7, 3 mantissa bits, no infinities, 0x7f and 0xff
NaN), the store's scale rule, and pools as numpy arrays."""
from __future__ import annotations

import numpy as np

GROUP, D = 64, 128


def _decode(c: int) -> float:
    sign = -1.0 if c & 0x80 else 1.0
    e, m = (c >> 3) & 15, c & 7
    if e == 15 and m == 7:
        return float("nan")
    return sign * (m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))


VALUES = np.array([_decode(c) for c in range(256)])
_POS = VALUES[:127]                 # codes 0 .. 126: increasing, 0 .. 448


def encode(x: np.ndarray) -> np.ndarray:
    """Codes of float64 values: nearest, ties to the even code, saturated; NaN -> 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0, x)), 448.0)
    hi = np.searchsorted(_POS, a, side="left")           # first code with value >= a
    hi = np.minimum(hi, 126)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - _POS[lo], _POS[hi] - a
    up = (dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0))
    code = np.where(up, hi, lo).astype(np.uint8)
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def scale_of(x: np.ndarray) -> float:
    """Scale of one group and head: its rows x [n, D] in float64."""
    a = np.abs(x[np.isfinite(x)])
    top = float(a.max()) if a.size else 0.0
    e = -90
    while top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def same_codes(a: np.ndarray, b: np.ndarray) -> np.ndarray:
    """Equal codes, every NaN code being equal to every other."""
    nan = ((a & 0x7F) == 0x7F) & ((b & 0x7F) == 0x7F)
    return (a == b) | nan


def append(x, codes, scale, table, start: int) -> None:
    """Rows x [n, Hkv, D] (float64) stored at positions start .. of one sequence, in place:
    codes uint8 [NB, bs, Hkv, D], scale float64 [NB, Hkv, bs / 64]."""
    bs, hkv = codes.shape[1], codes.shape[2]
    pos, end = start, start + len(x)
    while pos < end:
        stop = min(end, (pos // GROUP + 1) * GROUP)
        blk, off = int(table[pos // bs]), pos % bs
        g, base = off // GROUP, off // GROUP * GROUP
        part = x[pos - start:stop - start]
        for h in range(hkv):
            s = scale_of(part[:, h])
            if off > base:
                old = scale[blk, h, g]
                if s > old:
                    codes[blk, base:off, h] = encode(VALUES[codes[blk, base:off, h]] * (old / s))
                s = max(s, old)
            codes[blk, off:off + stop - pos, h] = encode(part[:, h] / s)
            scale[blk, h, g] = s
        pos = stop


def rows(codes, scale, table, n: int) -> np.ndarray:
    """Values [n, Hkv, D] (float64) of a sequence's first n positions."""
    bs = codes.shape[1]
    out = np.empty((n, codes.shape[2], D))
    for p in range(0, n, GROUP):
        m = min(GROUP, n - p)
        blk, off = int(table[p // bs]), p % bs
        out[p:p + m] = VALUES[codes[blk, off:off + m]] * scale[blk, :, off // GROUP][None, :, None]
    return out


def tables_for(lens, bs: int, g, spare: int = 2, width: int | None = None):
    """Random disjoint blocks for sequences of these lengths: (tables [B, W] padded with -1,
    number of blocks)."""
    need = [-(-int(n) // bs) for n in lens]
    nb = sum(need) + spare
    ids = g.permutation(nb)
    w = max(need + [1]) if width is None else width
    t = np.full((len(need), w), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = ids[at:at + n]
        at += n
    return t, nb


def random_cache(nb, bs, hkv, g, spread=2.0):
    """A cache of random codes and scales (what a store may have left anywhere)."""
    x = g.standard_normal((nb, bs, hkv, D))
    x *= np.exp(spread * 0.5 * g.standard_normal((1, 1, hkv, D)))
    e = g.integers(-8, -2, (nb, hkv, bs // GROUP)).astype(np.float64)
    return encode(32.0 * x), 2.0 ** e


def device_cache(codes, scale):
    import torch
    c = torch.from_numpy(np.ascontiguousarray(codes)).cuda().view(torch.float8_e4m3fn)
    return c, torch.from_numpy(scale.astype(np.float32)).cuda()


def host_codes(c):
    import torch
    return c.view(torch.uint8).cpu().numpy()
