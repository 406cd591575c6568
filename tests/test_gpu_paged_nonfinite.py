"""GPU tests of the paged cache's key bounds and page selection where keys are infinite or not numbers.

A page with a NaN among its keys has NaN bounds in that channel wherever in the page it stands; a score is
max over the group's heads of sum_d max(q hi, q lo), where a query element of 0 adds 0, and a page whose score is NaN
ranks before all others (attending it gives NaN, as attending every page would).
"""
import numpy as np
import pytest
import torch

from tests.helpers import to64
from tests.test_gpu_paged import BF16, F16, F32, make, randn

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def same(got, want):
    got, want = to64(got), np.asarray(want)
    return np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("page,dim", [(16, 128), (128, 64)])
def test_a_nan_key_shows_in_its_bounds_wherever_it_stands(dtype, page, dim):
    """First, last or in between of a run; of one token, or many; and in a page that is continued later."""
    places = sorted({0, 1, 3, 4, 7, 8, page // 2, page - 2, page - 1})
    n, hkv = page, 2
    B = len(places)
    c, table, g = make(B, 4, hkv, dim, dtype, page, [n] * B, seed=101, bounds=True, fill=False)
    c.bounds.fill_(99.0)
    k = randn(g, B, n, hkv, dim, dtype=dtype)
    for b, p in enumerate(places):
        k[b, p, 0, 5] = NAN
        k[b, p, 1, dim - 1] = INF if b % 2 else -INF
    k = k.cuda()
    c.append(k, k)
    for b in range(B):
        x = to64(k[b])
        assert same(c.bounds[table[b, 0]], np.stack([x.max(0), x.min(0)], 1)), places[b]
    # the same tokens, one by one and by two runs
    d, table, _ = make(B, 4, hkv, dim, dtype, page, [n] * B, seed=101, bounds=True, fill=False)
    for cuts in (list(range(n + 1)), [0, 5, n]):
        d.bounds.fill_(99.0)
        for lo, hi in zip(cuts, cuts[1:]):
            d.kv_len.fill_(hi)
            d.append(k[:, lo:hi].contiguous(), k[:, lo:hi].contiguous())
        for b in range(B):
            assert same(d.bounds[table[b, 0]], to64(c.bounds[table[b, 0]])), places[b]
    assert c.get_error() == 0 and d.get_error() == 0


def chosen(q, bounds, table_row, cols, n_select, first, recent):
    """Columns taken per kv head, by the definition in 64 bits: q [H, D], bounds [pages, Hkv, 2, D]."""
    H, Hkv = q.shape[0], bounds.shape[1]
    G = H // Hkv
    taken = []
    for e in range(Hkv):
        hi, lo = bounds[table_row[:cols], e, 0], bounds[table_row[:cols], e, 1]
        score = np.full(cols, -INF)
        for x in q[e * G:(e + 1) * G]:
            with np.errstate(invalid="ignore"):
                s = np.where(x == 0, 0.0, np.where(x > 0, x * hi, x * lo)).sum(-1)      # (NaN times anything is NaN)
            score = np.where(np.isnan(score) | np.isnan(s), NAN, np.fmax(score, s))
        kept = set(range(first)) | set(range(cols - recent, cols))
        rest = sorted((j for j in range(cols) if j not in kept), key=lambda j: (not np.isnan(score[j]), -score[j] if score[j] == score[j] else 0, j))
        taken.append(sorted(kept | set(rest[:n_select - len(kept)])))
    return taken


WHAT = ["one page above", "upper bounds", "lower bounds", "both", "all of a channel", "nan", "nan and infinite", "large", "opposite"]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 64), (16, 2, 128), (12, 1, 64)])
@pytest.mark.parametrize("cols", [90, 900])
@pytest.mark.parametrize("what", WHAT)
def test_selection_with_bounds_that_are_not_finite(what, cols, heads, kv_heads, dim, dtype):
    page = 16
    lens = [cols * page - 3, 40 * page]
    c, table, g = make(2, heads, kv_heads, dim, dtype, page, lens, seed=103, bounds=True)
    one = torch.randn(c.cfg.n_pages, kv_heads, 2, dim, generator=g)
    bd = torch.stack([one.amax(2), one.amin(2)], 2)
    some = table[0, 7:cols:11]                                   # (of row 0's pages)
    if what == "one page above":
        bd[table[0, cols // 2], :, 0, 3] = INF
    elif what == "upper bounds":
        bd[some, :, 0, 3] = INF
    elif what == "lower bounds":
        bd[some, :, 1, 3] = -INF
    elif what == "both":
        bd[some, :, 0, 3], bd[some, :, 1, 3] = INF, -INF
    elif what == "all of a channel":
        bd[:, :, 0, 3], bd[:, :, 1, 3] = INF, -INF
    elif what == "nan":
        bd[some[:5], :, :, 9] = NAN
    elif what == "nan and infinite":
        bd[some, :, 0, 3] = INF
        bd[some[1::2], 0, :, 9] = NAN
        bd[some[::3], :, :, 4] = -INF
    elif what == "large":
        bd *= {F16: 6e3, BF16: 3e37, F32: 3e37}[dtype]
    else:                                                        # keys of one sign of infinity only
        bd[some, :, :, 3] = INF
        bd[some[1::2], :, :, 3] = -INF
    c.bounds.copy_(bd.to(dtype))
    bounds = to64(c.bounds)
    q = torch.randn(2, heads, dim, generator=g)
    q[0, ::2, 3] = 0.0                                           # half the heads do not look at the channel
    q[1, :, 3] = 0.0
    q[1, 0] = 0.0
    q = (q * (20 if what == "large" and dtype != F16 else 1)).to(dtype)
    for n_select, first, recent in ((9, 1, 1), (30, 0, 2), (1, 0, 0)):
        for row in range(2):                                     # (row 1 in the place of row 0, too)
            out, sel = c.attend_sparse((q if row == 0 else q.flip(0)).cuda().contiguous(), n_select, first=first, recent=recent)
            for b, n in enumerate((cols, 40)):
                want = chosen(to64(q[b ^ row]), bounds, table[b], n, n_select, first, recent)
                assert sel[b].tolist() == want, (what, n_select, b, row)
    assert c.get_error() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_query_that_is_not_a_number_leaves_the_lowest_columns(dtype):
    """Every page's score is NaN for that kv head; the others choose as ever, and so does the next call."""
    c, table, g = make(1, 16, 2, 64, dtype, 16, [700], seed=104, bounds=True)
    one = torch.randn(c.cfg.n_pages, 2, 2, 64, generator=g)
    c.bounds.copy_(torch.stack([one.amax(2), one.amin(2)], 2).to(dtype))
    bounds = to64(c.bounds)
    q = randn(g, 1, 16, 64, dtype=dtype)
    bad = q.clone()
    bad[0, 2, 7] = NAN
    for x in (bad, q, bad, q):
        out, sel = c.attend_sparse(x.cuda(), 6)
        assert sel[0].tolist() == chosen(to64(x[0]), bounds, table[0], 44, 6, 1, 1)
        assert torch.isfinite(out[0, 8:]).all()
    assert c.get_error() == 0
