"""GPU tests of the paged cache's key bounds and page selection where keys are infinite or not numbers.

A page with a NaN among its keys has NaN bounds in that channel wherever in the page it stands; a score is
max over the group's heads of sum_d max(q hi, q lo), where a query element of 0 adds 0, and a page whose score is NaN
ranks before all others (attending it gives NaN, as attending every page would).
"""
import numpy as np
import pytest
import torch

from tests import paged_ref as ref
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
