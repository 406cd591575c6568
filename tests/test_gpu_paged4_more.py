"""GPU tests of the 4-bit paged cache's attention: items cut and joined behind whole ones where there are several rows, and queries
scaled down."""
import numpy as np
import pytest
import torch

from diffusion_serving_gb300 import workloads as wl
from tests import paged_ref as ref
from tests.helpers import to64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from diffusion_serving_gb300 import paged, paged4
    from tests.test_gpu_paged import bits, ints, randn
    from tests.test_gpu_paged4 import make
    from tests.test_gpu_paged4_runs import big

BF16, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype,heads,dim,page,lens,new", [
    (F16, 78, 64, 32, [6400, 6100], [120, 120]),                     # 156 items of two rows: a wave of whole ones, four cut
    (BF16, 77, 64, 16, [6400, 3000, 700, 6000], [60, 60, 0, 30]),    # 231 items, of which the call's tokens alone show 154
])
def test_cut_items_of_several_rows_behind_whole_ones(dtype, heads, dim, page, lens, new):
    """A few items left over from a wave, in many parts, joined by a launch of their own (by the rule that the sizes below meet)."""
    items = heads * -(-sum(new) // 128)
    assert 0 < items % 152 < 152 / 6 and items * (max(lens) // 128 + 1) >= 152 * 48
    c, g, k, v = big(lens, heads, heads, dim, dtype, page, seed=9)
    cu = wl.seqlens_to_cu(new)
    q = torch.randn(cu[-1], heads, dim, device="cuda", generator=g).to(dtype)
    args = dict(cu_q=ints(cu), max_q=max(new), lse=True)
    for flags in (paged.CAUSAL, 0):
        out, lse = c.attend(q, flags=flags, **args)
        for _ in range(3):                                # the same bits again
            again, lse2 = c.attend(q, flags=flags, **args)
            assert torch.equal(bits(again), bits(out)) and torch.equal(bits(lse2), bits(lse))
        assert c.get_error() == 0
        for b, n in enumerate(lens):
            kk, vv = to64(k[b]), to64(v[b])
            for i in range(b, new[b], 29):
                t = cu[b] + i
                see = ref.visible_mask(n, 0, new[b], n, flags == paged.CAUSAL)[i:i + 1]
                got = ref.attend_rows(to64(q[t:t + 1]), kk, vv, see, dim ** -0.5, dtype)
                got[2][:] += 2.0 ** -31 * np.abs(vv).sum(0)                # (weights below fp16's normal range: they are 2^6 too large)
                ref.check(out[t:t + 1], lse[t:t + 1], got, f"token {t}, flags {flags}")


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("e", [-6, -2, 3, 12])
def test_fp16_queries_times_a_power_of_two(new, e):
    """2^e times the queries under 2^-e times the scale give the same bits.  (Elements below 2^-8 are 0, so that 2^-6 times the others
    is within fp16's normal range and all products are exact.)"""
    lens = [300, 77]
    c, table, g, k, v = make(2, 8, 2, 128, F16, 16, lens, seed=15, scale=0.09)
    q = randn(g, 2 * new, 8, 128, dtype=F16).cuda()
    q[q.abs() < 2.0 ** -8] = 0
    x = (q.double() * 2.0 ** e).to(F16)
    assert torch.equal(x.double(), q.double() * 2.0 ** e)
    d = paged4.PagedKVCache4(2, 8, 2, 128, F16, page_size=16, n_pages=c.cfg.n_pages, max_pages=c.cfg.max_pages, pages=c.pages,
                             block_table=c.block_table, kv_len=c.kv_len, softmax_scale=0.09 * 2.0 ** -e)
    for a, b in zip(d.attend(x, lse=True), c.attend(q, lse=True)):
        assert torch.equal(bits(a), bits(b))
    assert c.get_error() == 0 and d.get_error() == 0
