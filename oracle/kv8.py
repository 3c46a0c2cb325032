"""The paged cache in e4m3 with a power-of-two scale per (block, kv head), in float64 (TEST
INFRASTRUCTURE ONLY, see the package docstring).

e4m3: sign, 4 exponent bits (bias 7), 3 fraction bits; 448 the largest, no infinities, codes 0x7f and
0xff NaN.  A block's scale is 2^e with the smallest e >= -64 that brings its rows to at most 448;
a block that goes on keeps the larger of its former and the new rows' scale, its rows moving
along.
"""
from __future__ import annotations

import numpy as np

E_MIN = -64


def decode_table():
    """Value of each of the 256 codes."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


DECODE = decode_table()


def decode(codes):
    return DECODE[np.asarray(codes, np.int64)]


def encode(x):
    """Nearest code (ties to even) of float64 x; beyond the range +-448, NaN 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    mags = DECODE[:127]  # rising: codes 0 .. 126
    hi = np.clip(np.searchsorted(mags, np.nan_to_num(a), side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = np.nan_to_num(a) - mags[lo], mags[hi] - np.nan_to_num(a)
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 0x7F, code)
    return (code | np.where(np.signbit(x) & ~np.isnan(x), 0x80, 0)).astype(np.uint8)


def exponent(amax):
    """Smallest e >= E_MIN with amax <= 448 * 2^e."""
    e = E_MIN
    while e < 127 and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def append(codes, scales, rows, block_table, ctx_len, counts, block_size):
    """Adds rows[b] [counts[b], h, D] (float64) at positions ctx_len[b] ..; codes [nb, h, bs, D] and
    scales [nb, h] are updated in place."""
    for b, n in enumerate(counts):
        p, end = int(ctx_len[b]), int(ctx_len[b]) + int(n)
        j = 0
        while p < end:
            blk, off = int(block_table[b, p // block_size]), p % block_size
            k = min(block_size - off, end - p)
            for g in range(codes.shape[1]):
                x = rows[b][j:j + k, g]
                a = np.abs(x[np.isfinite(x)])
                s = 2.0 ** exponent(a.max() if a.size else 0.0)
                if off > 0:
                    old = float(scales[blk, g])
                    if old >= s:
                        s = old
                    else:
                        codes[blk, g, :off] = encode(decode(codes[blk, g, :off]) * (old / s))
                scales[blk, g] = s
                codes[blk, g, off:off + k] = encode(x / s)
            p += k
            j += k
