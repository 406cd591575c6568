"""Plain forms of the 4-bit store: what is held of a value, and records taken apart, in NumPy."""
from __future__ import annotations

import numpy as np

# every e4m3 value that a scale can be, by its bits (0 .. 126; 127 is NaN)
E4M3 = np.array([(b & 7) * 2.0 ** -9 if b < 8 else (8 + (b & 7)) * 2.0 ** ((b >> 3) - 10) for b in range(127)])


def scale_bits(top):
    """e4m3 bits of top / 7 (top >= 0 in 64 bits, NaN among them): the nearest, of two as near the even, at most 448."""
    x = np.minimum(top / 7, 448.0)
    nan = np.isnan(x)
    # compare 2 x 7 with neighbours' sums x 7, all exact: 14 top / 7 against 7 (a + b)
    hi = np.searchsorted(E4M3, np.where(nan, 0, x), side="left").clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    t = np.where(nan, 0, np.minimum(top, 3136.0))
    gap = 2 * t - 7 * (E4M3[lo] + E4M3[hi])
    b = np.where(gap > 0, hi, np.where(gap < 0, lo, np.where(hi % 2 == 0, hi, lo)))
    return np.where(nan, 127, b)


def codes(x):
    """(codes [..., D] 1 .. 15, scale bits [..., D / 32]) of values x [..., D] of a 16-bit type, in 64 bits."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    with np.errstate(invalid="ignore", divide="ignore"):
        b = scale_bits(np.abs(g).max(-1))
        s = np.append(E4M3, np.nan)[b][..., None]
        r = np.clip(np.nan_to_num(g, nan=0.0, posinf=1e30, neginf=-1e30), -7 * s, 7 * s)
        n = np.where(s > 0, np.rint(r / np.where(s > 0, s, 1.0)), 0.0)     # (at most 16 + 4 bits: a tie's quotient is exact)
    n = np.nan_to_num(n, nan=0.0)
    return (n + 8).astype(np.int64).reshape(x.shape), b


def value(code, bits):
    """Held values [..., D] from codes and scale bits."""
    s = np.append(E4M3, np.nan)[bits]
    return ((code - 8).reshape(*bits.shape, 32) * s[..., None]).reshape(code.shape)


def held(x):
    return value(*codes(x))


def unpack(records, page, dim):
    """(K codes, K scale bits, V codes, V scale bits) of records [n, Hkv, bytes], slot by slot: [n, page, Hkv, ...]."""
    n, hkv, size = records.shape
    assert size == page * (dim + dim // 16)
    r = records.astype(np.int64)
    kc, vc = (np.zeros((n, page, hkv, dim), np.int64) for _ in range(2))
    ks, vs = (np.zeros((n, page, hkv, dim // 32), np.int64) for _ in range(2))
    for p in range(page):
        for d in range(dim):
            bit = 4 * (d % 8 // 2) + 16 * (d % 2)
            byte = d // 8 * 4 + bit // 8
            kc[:, p, :, d] = r[:, :, p * dim // 2 + byte] >> (bit % 8) & 15
            byte = (byte // 16 ^ (p // 4 % (dim // 32))) * 16 + byte % 16
            vc[:, p, :, d] = r[:, :, (page + p) * dim // 2 + byte] >> (bit % 8) & 15
        for x in range(dim // 32):
            ks[:, p, :, x] = r[:, :, page * dim + p * (dim // 32) + x]
            vs[:, p, :, x] = r[:, :, page * dim + page * (dim // 32) + x * page + p]
    return kc, ks, vc, vs
