"""Plain 64-bit forms of the paged cache's operators, and the bounds that the tests hold kernels to.

NumPy only; rows and pages are walked one by one.
"""
from __future__ import annotations

import numpy as np
import torch

from tests.helpers import EPS_EXP2, to64


def gather(pages: np.ndarray, table_row, start: int, n: int):
    """Slots [start, n) of a row: [n - start, Hkv, D]."""
    ps = pages.shape[1]
    return np.stack([pages[table_row[p // ps], p % ps] for p in range(start, n)]) if n > start else \
        np.zeros((0,) + pages.shape[2:])


def attend_rows(q, k, v, visible, scale, dtype):
    """Softmax attention of q [n, H, D] over k, v [S, Hkv, D], query i seeing visible[i] [S] (bool).

    Returns (out [n, H, D], lse [n, H], out_bound, lse_bound).  The bounds are on a kernel that forms scores
    and sums in fp32, exponentials with relative error EPS_EXP2, weights rounded to `dtype` before the product with v
    (none for fp32), and rounds the result once:
     * a score: an fp32 sum of D products, any order, errs by at most 2 D 2^-24 * 2 * scale * sum |q_d k_d|; scaling and
       subtracting the maximum add 2^-22 (|s| + |max|).  All scores off by at most e change each weight by a factor
       within exp(+-2 e).
     * a weight: its exponential, at most T = S / 16 + 400 rescales of the sums, S + 64 fp32 additions (2^-24
       each), and its own rounding, finfo(dtype).eps / 2 relative, or half the type's least step where that is more.
     * the result: one rounding, finfo(dtype).eps / 2 relative (or half a least step).
    """
    n, H, D = q.shape
    S, Hkv = k.shape[:2]
    G = H // Hkv
    eps = float(torch.finfo(dtype).eps) / 2
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}[dtype]
    out, bound = np.zeros((n, H, D)), np.full((n, H, D), 2 * tiny)
    lse, lse_bound = np.full((n, H), -np.inf), np.zeros((n, H))
    T = S / 16 + 400
    rel = (T + 4) * EPS_EXP2 + (S + 64) * 2.0 ** -24
    p_eps = 0.0 if dtype == torch.float32 else eps
    for h in range(H):
        kk, vv = k[:, h // G], v[:, h // G]
        s = scale * (q[:, h] @ kk.T) if S else np.zeros((n, 0))
        mag = scale * (np.abs(q[:, h]) @ np.abs(kk).T) if S else s
        for i in range(n):
            see = visible[i]
            if not see.any():
                continue
            si, vi = s[i, see], vv[see]
            m = si.max()
            w = np.exp(si - m)
            L = w.sum()
            w = w / L
            out[i, h] = w @ vi
            lse[i, h] = m + np.log(L)
            e = (4 * D * 2.0 ** -24 * mag[i, see]).max() + 2.0 ** -22 * 2 * np.abs(si).max()
            off = np.expm1(2 * e) + rel + p_eps
            av = w @ np.abs(vi)
            bound[i, h] = 2 * off * av + eps * np.abs(out[i, h]) + 2 * tiny
            if p_eps:      # weights below the type's normal range: against a maximum of 1 (or more), half a least step
                bound[i, h] += tiny * np.abs(vi).sum(0) / L
            lse_bound[i, h] = e + rel / (1 - rel) + 2.0 ** -21 * (abs(lse[i, h]) + 1)
    return out, lse, bound, lse_bound


def visible_mask(n_slots_end, start, n, length, causal):
    """[n, S]: query i of n (the row's last tokens) sees slots start.. up to its own, or up to length."""
    slots = np.arange(start, n_slots_end)
    if causal:
        return np.stack([slots <= length - n + i for i in range(n)]) if n else np.zeros((0, len(slots)), bool)
    return np.broadcast_to(slots < length, (n, len(slots)))


def check(got, lse_got, want, what):
    out, lse, bound, lse_bound = want
    g = to64(got)
    assert np.isfinite(g).all(), f"{what}: not finite"
    err = np.abs(g - out)
    assert (err <= bound).all(), f"{what}: {np.max(err - bound):.3e} over its bound, error {err.max():.3e}"
    if lse_got is not None:
        L = to64(lse_got)
        none = np.isneginf(lse)
        assert np.array_equal(np.isneginf(L), none), f"{what}: lse of tokens that see nothing"
        d = np.abs(L[~none] - lse[~none])
        assert (d <= lse_bound[~none]).all(), f"{what}: lse off by {d.max():.3e}"


def page_bounds(k_pages, page, filled):
    """[2, Hkv, D] maximum and minimum of a page's first `filled` keys."""
    x = k_pages[page, :filled]
    return np.stack([x.max(0), x.min(0)])


def select(q, bounds, table_row, n_pages_row, n_select, first, recent):
    """Columns taken for one row, per kv head: q [H, D], bounds [pages, Hkv, 2, D] in 64 bits."""
    H, Hkv = q.shape[0], bounds.shape[1]
    G = H // Hkv
    taken = []
    for e in range(Hkv):
        if n_pages_row <= n_select:
            taken.append(list(range(n_pages_row)))
            continue
        score = {}
        for j in range(n_pages_row):
            hi, lo = bounds[table_row[j], e]
            score[j] = max(np.maximum(q[e * G + g] * hi, q[e * G + g] * lo).sum() for g in range(G))
        kept = set(range(first)) | set(range(n_pages_row - recent, n_pages_row))
        rest = sorted((j for j in score if j not in kept), key=lambda j: (-score[j], j))
        taken.append(sorted(kept | set(rest[:n_select - len(kept)])))
    return taken
