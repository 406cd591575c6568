"""GPU tests of the paged cache with tables sized for far longer rows than they hold, prefix lists longer than the prefix, and
query buffers whose tokens behind the last row are not numbers.

Which kernel runs goes by capacities (columns, list length, max_q), since lengths are on the device: the results are the same.
"""
import pytest
import torch

from diffusion_serving_gb300 import workloads as wl
from tests.test_gpu_paged import BF16, F16, F32, check, expect, ints, make, randn
from tests.test_gpu_paged_runs import big

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from diffusion_serving_gb300 import paged


def widened(c, cols, max_tokens=0):
    """The same pools and rows under a table of `cols` columns whose rest is out of range."""
    table = torch.full((c.batch, cols), 2 ** 30, dtype=torch.int32, device="cuda")
    table[:, :c.cfg.max_pages] = c.block_table
    d = paged.PagedKVCache(c.batch, c.heads, c.kv_heads, c.head_dim, c.dtype, page_size=c.cfg.page_size, n_pages=c.cfg.n_pages,
                           max_pages=cols, max_tokens=max_tokens, bounds=c.bounds, k_pages=c.k_pages, v_pages=c.v_pages,
                           block_table=table, kv_len=c.kv_len)
    return d


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("heads,kv_heads,dim,page,lens,new", [
    (8, 2, 128, 16, [300, 0, 41, 16], [1, 1, 1, 1]),
    (32, 8, 128, 16, [600, 33], [5, 3]),                          # 20 query rows a group
    (12, 4, 64, 64, [200, 131, 7], [60, 131, 2]),
])
def test_wide_tables_and_padded_queries(dtype, heads, kv_heads, dim, page, lens, new):
    c, table, g = make(len(lens), heads, kv_heads, dim, dtype, page, lens, seed=120)
    d = widened(c, 40000 // page * 16)
    cu = wl.seqlens_to_cu(new)
    q = randn(g, cu[-1] + 5, heads, dim, dtype=dtype).cuda()
    q[cu[-1]:] = float("nan")
    want = expect(c, table, q[:cu[-1]], lens, cu, True)
    for x in (c, d):
        for most in (max(new), 1 << 20):
            out, lse = torch.full_like(q, 7.0), torch.full((len(q), heads), 7.0, device="cuda")
            x.attend(q, cu_q=ints(cu), max_q=most, out=out, lse=lse, flags=paged.CAUSAL)
            assert x.get_error() == 0
            check(out, lse, want, f"{x.cfg.max_pages} columns, max_q {most}", cu[-1])
            assert torch.all(out[cu[-1]:] == 7.0) and torch.all(lse[cu[-1]:] == 7.0)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("prefix", [64, 4096])
def test_prefix_lists_longer_than_the_prefix(dtype, prefix):
    heads, kv_heads, dim, page = 8, 2, 128, 16
    lens, new = [prefix + n for n in (1, 30, 17, 2)], [1, 4, 2, 2]
    c, table, g = make(4, heads, kv_heads, dim, dtype, page, lens, seed=121, shared=prefix // page, max_tokens=16)
    d = widened(c, 9000, max_tokens=16)
    d.block_table[:, :prefix // page] = -1
    pages = torch.full((8000,), -9, dtype=torch.int32, device="cuda")      # (what is past the prefix is not read)
    pages[:prefix // page] = ints(c.perm[:prefix // page])
    cu = wl.seqlens_to_cu(new)
    q = randn(g, cu[-1] + 5, heads, dim, dtype=dtype).cuda()
    q[cu[-1]:] = float("nan")
    want = expect(c, table, q[:cu[-1]], lens, cu, True)
    for x, p in ((c, pages[:prefix // page].clone()), (d, pages)):
        out, lse = torch.full_like(q, 7.0), torch.full((len(q), heads), 7.0, device="cuda")
        x.attend_shared(q, p, ints([prefix]), cu_q=ints(cu), max_q=max(new), out=out, lse=lse, flags=paged.CAUSAL)
        assert x.get_error() == 0
        check(out, lse, want, f"list of {len(p)}", cu[-1])
        assert torch.all(out[cu[-1]:] == 7.0) and torch.all(lse[cu[-1]:] == 7.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_selection_from_wide_tables(dtype):
    """Bit for bit what a table cut to the rows gives."""
    c, g = big([3000, 40, 1700, 1], 16, 4, 64, dtype, 16, seed=122, bounds=True)
    q = torch.randn(4, 16, 64, device="cuda", generator=g).to(dtype)
    want = c.attend_sparse(q, 12, lse=True)
    for cols in (1000, 32768):
        d = widened(c, cols)
        got = d.attend_sparse(q, 12, lse=True)
        assert d.get_error() == 0
        assert torch.equal(got[2], want[2]) and torch.equal(got[1], want[1])
        assert torch.equal(got[0], want[0])
