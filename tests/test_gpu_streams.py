"""GPU tests of memory across streams: a call on a stream that is not the current one, with outputs it allots itself, and
buffers that are given back while it is pending.

torch's allocator hands a freed block out again at once on the stream it belongs to.  `torch.cuda._sleep` keeps one stream
busy for some 50 ms, so that what follows on it comes late, whatever the other stream does meanwhile.
"""
import pytest
import torch

from tests.test_gpu_paged import BF16, F32, bits, ints, make, randn

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from diffusion_serving_gb300 import kvc, paged

SLEEP = 100_000_000                                      # clocks


def pending(*like):
    """Blocks as large as these tensors, freed while the current stream has yet to write them."""
    held = [torch.empty_like(t) for t in like for _ in range(4)]
    torch.cuda._sleep(SLEEP)
    for t in held:
        t.fill_(7)


@pytest.mark.parametrize("as_int", [False, True])
@pytest.mark.parametrize("dtype,new", [(BF16, 1), (BF16, 40), (F32, 1)])
def test_outputs_are_not_memory_that_the_current_stream_still_writes(dtype, new, as_int):
    lens, P = [900, 400], 64
    c, table, g = make(2, 8, 2, 128, dtype, 32, lens, seed=35, bounds=new == 1, max_tokens=2 * new)
    c.block_table[1, :P // 32] = c.block_table[0, :P // 32]
    q = randn(g, 2, new, 8, 128, dtype=dtype).cuda()
    k = randn(g, 2, new, 2, 128, dtype=dtype).cuda()
    rope = torch.ones(1000, 64, 2, device="cuda")
    pages, plen = c.block_table[0, :P // 32].clone(), ints([P])
    s = torch.cuda.Stream()
    on = s.cuda_stream if as_int else s
    calls = [lambda st: c.attend(q, lse=True, stream=st), lambda st: c.attend_shared(q, pages, plen, lse=True, stream=st),
             lambda st: [c.append(k, k, rope=rope, q=q, stream=st)]]
    if new == 1:
        c.bounds.copy_(torch.stack([c.k_pages.nan_to_num(0).amax(1), c.k_pages.nan_to_num(0).amin(1)], 2))
        calls.insert(2, lambda st: c.attend_sparse(q, 4, lse=True, stream=st))
    for i, call in enumerate(calls):
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        pending(*want)
        got = call(on)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(bits(x), bits(y)), i
    assert c.get_error() == 0


@pytest.mark.parametrize("default", [0, "default_stream"])
def test_the_default_stream_from_another(default):
    """Its handle is 0."""
    c, table, g = make(2, 8, 2, 128, BF16, 32, [300, 40], seed=41)
    q = randn(g, 2, 8, 128, dtype=BF16).cuda()
    want = c.attend(q, lse=True)
    on = default if default == 0 else torch.cuda.default_stream()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        pending(*want)
        got = c.attend(q, lse=True, stream=on)
        d = paged.PagedKVCache(2, 8, 2, 128, BF16, page_size=32, n_pages=c.cfg.n_pages, max_pages=c.cfg.max_pages, k_pages=c.k_pages,
                               v_pages=c.v_pages, block_table=c.block_table, kv_len=c.kv_len, stream=on)
        more = d.attend(q, lse=True, stream=on)
    torch.cuda.synchronize()
    for x, y, z in zip(got, more, want):
        assert torch.equal(bits(x), bits(z)) and torch.equal(bits(y), bits(z))
    assert c.get_error() == 0 and d.get_error() == 0


def test_outputs_are_not_handed_out_again_while_the_current_stream_reads_them():
    c, table, g = make(2, 8, 2, 128, BF16, 32, [300, 40], seed=36)
    q = randn(g, 2, 8, 128, dtype=BF16).cuda()
    want = c.attend(q)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = c.attend(q, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(SLEEP)
    copy = out.clone()                                   # late
    del out
    with torch.cuda.stream(s):
        for t in [torch.empty_like(q) for _ in range(4)]:
            t.fill_(7)
    torch.cuda.synchronize()
    assert torch.equal(bits(copy), bits(want))


@pytest.mark.parametrize("how", ["stream=", "current"])
def test_a_cache_given_back_while_another_stream_has_calls_pending(how):
    c, table, g = make(2, 8, 2, 128, BF16, 32, [3000, 400], seed=37)
    q = randn(g, 2, 8, 128, dtype=BF16).cuda()
    want, out = c.attend(q), torch.empty_like(q)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(SLEEP)
        if how == "current":
            c.attend(q, out=out)
    if how == "stream=":
        c.attend(q, out=out, stream=s)
    shapes = [(t.shape, t.dtype) for t in (c.k_pages, c.v_pages, c.block_table, c.kv_len, c.workspace)]
    del c
    for shape, dtype in shapes:
        torch.empty(shape, dtype=dtype, device="cuda").fill_(1)
    torch.cuda.synchronize()
    assert torch.equal(bits(out), bits(want))


def test_a_cache_made_on_a_stream_that_is_not_the_current_one():
    """The buffers' first values and the workspace's zeros are there for both streams."""
    lens = [3000, 2500]
    c, table, g = make(2, 8, 2, 128, BF16, 32, lens, seed=38)
    q = randn(g, 2, 8, 128, dtype=BF16).cuda()
    want = c.attend(q)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    pending(c.workspace)
    d = paged.PagedKVCache(2, 8, 2, 128, BF16, page_size=32, n_pages=c.cfg.n_pages, max_pages=c.cfg.max_pages, k_pages=c.k_pages,
                           v_pages=c.v_pages, block_table=c.block_table, kv_len=c.kv_len, stream=s)
    first, second = d.attend(q, stream=s), None
    torch.cuda.current_stream().wait_stream(s)
    second = d.attend(q)
    torch.cuda.synchronize()
    assert torch.equal(bits(first), bits(want)) and torch.equal(bits(second), bits(want))
    assert d.get_error() == 0


@pytest.mark.parametrize("dtype,n_q", [(BF16, 1), (BF16, 200), (F32, 1)])
def test_linear_cache_outputs_are_not_memory_that_the_current_stream_still_writes(dtype, n_q):
    c = kvc.KVCache(2, 8, 2, 128, dtype, "linear", capacity=600)
    g = torch.Generator().manual_seed(39)
    k = randn(g, 2, 500, 2, 128, dtype=dtype).cuda()
    c.append(k, k)
    q = randn(g, 2, n_q, 8, 128, dtype=dtype).cuda()
    s = torch.cuda.Stream()
    calls = [lambda st: [c.attend(q, stream=st)], lambda st: c.attend_lse(q, stream=st)]
    if n_q == 1 and dtype != F32:
        new = randn(g, 2, 1, 2, 128, dtype=dtype).cuda()

        def step(st):
            c.reset(stream=st)
            c.append(k, k, stream=st)
            return [c.append_attend(new, new, q, stream=st)]
        calls.append(step)
    for call in calls:
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        pending(*want)
        got = call(s)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            # (the order of sums may differ between calls: outputs below 2 in size, three roundings of half a step each)
            torch.testing.assert_close(x, y, rtol=0, atol=2.0 ** -5)
    assert c.get_error() == 0


def test_a_cache_of_another_stream_given_back_while_the_default_one_has_calls_pending():
    c, table, g = make(2, 8, 2, 128, BF16, 32, [3000, 400], seed=40)
    q = randn(g, 2, 8, 128, dtype=BF16).cuda()
    want, out = c.attend(q), torch.empty_like(q)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        d = paged.PagedKVCache(2, 8, 2, 128, BF16, page_size=32, n_pages=c.cfg.n_pages, max_pages=c.cfg.max_pages)
        for x, y in ((d.k_pages, c.k_pages), (d.v_pages, c.v_pages), (d.block_table, c.block_table), (d.kv_len, c.kv_len)):
            x.copy_(y)
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    d.attend(q, out=out)
    shapes = [(t.shape, t.dtype) for t in (d.k_pages, d.v_pages, d.block_table, d.kv_len, d.workspace)]
    del d, x, y
    with torch.cuda.stream(s):
        for shape, dtype in shapes:
            torch.empty(shape, dtype=dtype, device="cuda").fill_(1)
    torch.cuda.synchronize()
    assert torch.equal(bits(out), bits(want))
