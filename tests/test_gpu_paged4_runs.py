"""GPU tests of the 4-bit paged cache as a server runs it: prompts with images, chunks and captured decode steps together, streams,
graphs on one handle, large batches and groups, wide tables, and waits that run out."""
import numpy as np
import pytest
import torch

from diffusion_serving_gb300 import workloads as wl
from tests import paged4_ref as ref4
from tests import paged_ref as ref
from tests.helpers import to64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from diffusion_serving_gb300 import kvc, paged, paged4
    from tests.test_gpu_paged import bits, ints, randn
    from tests.test_gpu_paged4 import check, expect, make
    from tests.test_gpu_paged_axes import turned

BF16, F16 = torch.bfloat16, torch.float16


def big(lens, heads, kv_heads, dim, dtype, page, *, seed, max_pages=None):
    """Rows of `lens` tokens appended at once, pages in random order, all on the device; and their held values, read back."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    c = paged4.PagedKVCache4(len(lens), heads, kv_heads, dim, dtype, page_size=page, n_pages=sum(need),
                             max_pages=max_pages or max(need))
    perm = torch.randperm(sum(need), generator=g, device="cuda").int()
    at = 0
    for b, p in enumerate(need):
        c.block_table[b, :p] = perm[at:at + p]
        at += p
    c.kv_len.copy_(ints(lens))
    cu = ints(wl.seqlens_to_cu(lens))
    k, v = (torch.randn(sum(lens), kv_heads, dim, device="cuda", generator=g).to(dtype) for _ in range(2))
    c.append(k, v, cu_new=cu)
    k, v = c.read(sum(lens), cu=cu)
    assert c.get_error() == 0
    return c, g, k.split(lens), v.split(lens)


@pytest.mark.parametrize("dtype,heads,kv_heads,dim,page", [(BF16, 8, 2, 128, 16), (F16, 6, 6, 64, 64)])
def test_prompts_with_images_then_captured_steps(dtype, heads, kv_heads, dim, page):
    """Two prompts with an image each at positions of three axes, attended as a causal chunk; then single tokens by one captured
    step, whose lengths, positions and tokens change between replays."""
    n = dim // 2
    pair_axis = [0] * (n // 4) + [1] * (3 * n // 8) + [2] * (3 * n // 8)
    axes, rope = paged.rope_axes(pair_axis), wl.rope_table(300, dim)
    lens, steps = [70, 133], 5
    total = [x + steps for x in lens]
    c, table, g, _, _ = make(2, heads, kv_heads, dim, dtype, page, total, fill=False, seed=21)
    c.kv_len.copy_(ints(lens))
    cu = wl.seqlens_to_cu(lens)
    k, v, q = (randn(g, cu[-1], h, dim, dtype=dtype) for h in (kv_heads, kv_heads, heads))
    pos = []
    for m in lens:                                        # text, an image of 6 x 9, text
        pos += [[i] * 3 for i in range(5)] + [[5, 5 + i // 9, 5 + i % 9] for i in range(54)] + [[14 + i] * 3 for i in range(m - 59)]
    pos = torch.tensor(pos, dtype=torch.int32)
    qr = c.append(k.cuda(), v.cuda(), cu_new=ints(cu), rope=rope.cuda(), q=q.cuda(), positions=pos.cuda(), axes=axes)
    out, lse = c.attend(qr, cu_q=ints(cu), max_q=max(lens), lse=True, flags=paged.CAUSAL)
    assert c.get_error() == 0
    held_k = [ref4.held(to64(turned(k[cu[b]:cu[b + 1]], pos[cu[b]:cu[b + 1]].numpy(), pair_axis, rope.numpy(), False, dtype))) for b in range(2)]
    held_v = [ref4.held(to64(v[cu[b]:cu[b + 1]])) for b in range(2)]
    check(out, lse, expect(c, held_k, held_v, qr, lens, cu, True), "prompts")

    k1, v1, q1 = (torch.zeros(2, h, dim, dtype=dtype, device="cuda") for h in (kv_heads, kv_heads, heads))
    p1, rope = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), rope.cuda()
    qr1, out1, lse1 = torch.zeros_like(q1), torch.zeros_like(q1), torch.zeros(2, heads, device="cuda")

    def step():
        c.kv_len.add_(1)
        c.append(k1, v1, rope=rope, q=q1, q_out=qr1, positions=p1, axes=axes)
        c.attend(qr1, out=out1, lse=lse1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        c.kv_len.sub_(1)                                  # (a run before the capture, over the last prompt token's slot ...)
        keep = c.pages.clone()
        step()
        c.pages.copy_(keep)                               # (... which is then put back)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        step()
    assert c.kv_len.tolist() == lens                      # (capturing runs nothing)
    for s in range(steps):
        kk, vv, qq = (randn(g, 2, h, dim, dtype=dtype) for h in (kv_heads, kv_heads, heads))
        where = torch.tensor([[lens[b] - 45 + s] * 3 for b in range(2)], dtype=torch.int32)
        k1.copy_(kk), v1.copy_(vv), q1.copy_(qq), p1.copy_(where)
        graph.replay()
        assert c.get_error() == 0
        for b in range(2):
            held_k[b] = np.concatenate([held_k[b], ref4.held(to64(turned(kk[b:b + 1], where[b:b + 1].numpy(), pair_axis, rope.cpu().numpy(), False, dtype)))])
            held_v[b] = np.concatenate([held_v[b], ref4.held(to64(vv[b:b + 1]))])
        check(out1, lse1, expect(c, held_k, held_v, qr1, [x + s + 1 for x in lens], None, False), f"step {s}")
    got_k, got_v = c.read(sum(total), cu=ints(wl.seqlens_to_cu(total)))
    assert np.array_equal(to64(got_k), np.concatenate(held_k)) and np.array_equal(to64(got_v), np.concatenate(held_v))


@pytest.mark.parametrize("dtype,heads,kv_heads,dim,page,lens,new", [
    (BF16, 32, 8, 128, 64, [4500, 7000], [700, 1024]),
    (F16, 40, 40, 64, 16, [5200, 3000], [333, 300]),
    (BF16, 64, 64, 128, 128, [300, 9000, 40], [290, 129, 40]),       # one long row among short ones
    (F16, 156, 156, 64, 32, [6400], [120]),                          # a few items left over from a wave, in many parts
    (BF16, 2, 1, 128, 16, [20000], [100]),                           # few items, cut among all blocks
])
def test_long_chunks_of_whole_and_cut_items(dtype, heads, kv_heads, dim, page, lens, new):
    c, g, k, v = big(lens, heads, kv_heads, dim, dtype, page, seed=5)
    cu = wl.seqlens_to_cu(new)
    q = torch.randn(cu[-1], heads, dim, device="cuda", generator=g).to(dtype)
    args = dict(cu_q=ints(cu), max_q=max(new), lse=True, flags=paged.CAUSAL)
    out, lse = c.attend(q, **args)
    for _ in range(3):                                    # the same bits again
        again, lse2 = c.attend(q, **args)
        assert torch.equal(bits(again), bits(out)) and torch.equal(bits(lse2), bits(lse))
    assert c.get_error() == 0
    for b, n in enumerate(lens):
        kk, vv = to64(k[b]), to64(v[b])
        for i in range(b, new[b], 97):
            t = cu[b] + i
            see = ref.visible_mask(n, 0, new[b], n, True)[i:i + 1]
            got = ref.attend_rows(to64(q[t:t + 1]), kk, vv, see, dim ** -0.5, dtype)
            got[2][:] += 2.0 ** -31 * np.repeat(np.abs(vv).sum(0), heads // kv_heads, 0)       # (weights: 2^6 too large here)
            ref.check(out[t:t + 1], lse[t:t + 1], got, f"token {t}")


@pytest.mark.parametrize("dim", [64, 128])
def test_what_shared_memory_held_before_decides_nothing(dim):
    """Slots behind a row's end in a tile are not brought in: query rows that an item does not have (3 of 5 heads' tokens in 16 rows)
    meet there what an earlier block left.  The same call gives the same bits whatever ran before it."""
    lens, new = [1552, 353, 2475, 546, 349], [4, 2, 2, 1, 4]
    c, g, _, _ = big(lens, 40, 8, dim, BF16, 16, seed=31)
    cu = wl.seqlens_to_cu(new)
    q = (3 * torch.randn(cu[-1], 40, dim, device="cuda", generator=g)).to(BF16)
    noise = paged4.PagedKVCache4(64, 8, 8, dim, F16, page_size=16, n_pages=64 * 40, max_pages=40)
    noise.block_table.copy_(torch.arange(64 * 40, dtype=torch.int32).reshape(64, 40))
    noise.kv_len.fill_(640)
    qn = torch.randn(64, 8, dim, device="cuda", generator=g).half()
    args = dict(cu_q=ints(cu), max_q=max(new), lse=True)
    want = c.attend(q, **args)
    for fill in (255, 127, 0, 119, 256):
        noise.pages.copy_(torch.randint(0, 256, noise.pages.shape, device="cuda", generator=g, dtype=torch.uint8) if fill == 256
                          else torch.full_like(noise.pages, fill))
        for _ in range(4):
            noise.attend(qn)
            for x, y in zip(c.attend(q, **args), want):
                assert torch.equal(bits(x), bits(y)), fill
    assert c.get_error() == 0


def test_a_batch_of_1024_rows():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 70, 1024)]
    lens[7] = 2000
    c, g, k, v = big(lens, 4, 2, 64, BF16, 16, seed=6)
    for new in (1, 24):
        q = torch.randn(1024 * new, 4, 64, device="cuda", generator=g).to(BF16)
        out, lse = c.attend(q, lse=True, flags=paged.CAUSAL)
        assert c.get_error() == 0
        for b in [7, 0, 1023] + list(range(11, 1024, 61)):
            n, rows = lens[b], slice(b * new, (b + 1) * new)
            got = ref.attend_rows(to64(q[rows]), to64(k[b]).reshape(-1, 2, 64), to64(v[b]).reshape(-1, 2, 64),
                                  ref.visible_mask(n, 0, new, n, True), 64 ** -0.5, BF16)
            ref.check(out[rows], lse[rows], got, f"row {b}")


@pytest.mark.parametrize("dtype,heads,dim,page", [(BF16, 8, 128, 16), (F16, 32, 128, 64), (F16, 8, 64, 32), (BF16, 32, 64, 128)])
def test_many_short_rows_and_a_few_long_ones(dtype, heads, dim, page):
    """Rows of a few tiles, which sets of warps take by themselves, and among them some of more tiles than are in flight at once."""
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.integers(0, 400, 160)]
    lens[7], lens[90], lens[91] = 3000, 1700, 2500
    c, g, k, v = big(lens, heads, 2, dim, dtype, page, seed=8)
    q = torch.randn(len(lens), heads, dim, device="cuda", generator=g).to(dtype)
    out, lse = c.attend(q, lse=True)
    for _ in range(3):                                    # the same bits again
        again, lse2 = c.attend(q, lse=True)
        assert torch.equal(bits(again), bits(out)) and torch.equal(bits(lse2), bits(lse))
    assert c.get_error() == 0
    for b, n in enumerate(lens):
        kk, vv = to64(k[b]).reshape(-1, 2, dim), to64(v[b]).reshape(-1, 2, dim)
        got = ref.attend_rows(to64(q[b:b + 1]), kk, vv, ref.visible_mask(n, 0, 1, n, False), dim ** -0.5, dtype)
        got[2][:] += 2.0 ** -33 * np.repeat(np.abs(vv).sum(0), heads // 2, 0)               # (weights: 2^8 too large here)
        ref.check(out[b:b + 1], lse[b:b + 1], got, f"row {b}")


def test_a_wait_that_ran_out_among_short_rows():
    c, g, _, _ = big([100] * 200, 8, 2, 128, BF16, 16, seed=42)
    q = torch.randn(200, 8, 128, device="cuda", generator=g).to(BF16)
    want = c.attend(q)
    assert c.get_error() == 0
    paged4.kvc_paged4_debug_stall_waits(c.handle, 200_000)
    c.attend(q)
    paged4.kvc_paged4_debug_stall_waits(c.handle, 0)
    assert c.get_error() & paged.DEV_TIMEOUT
    got = c.attend(q)
    assert c.get_error() == 0 and torch.equal(bits(got), bits(want))


@pytest.mark.parametrize("heads,kv_heads", [(96, 1), (22, 2), (33, 1)])
@pytest.mark.parametrize("new", [1, 9])
def test_large_and_odd_groups(heads, kv_heads, new):
    lens = [400, 33]
    c, table, g, k, v = make(2, heads, kv_heads, 128, F16, 32, lens, seed=13)
    q = randn(g, 2 * new, heads, 128, dtype=F16)
    out, lse = c.attend(q.cuda(), lse=True, flags=paged.CAUSAL)
    assert c.get_error() == 0
    check(out, lse, expect(c, k, v, q, lens, None, True), "groups")


@pytest.mark.parametrize("new", [1, 5, 60])
def test_wide_tables_and_padded_queries(new):
    """A table sized for far longer rows, its rest out of range; queries behind the last row that are not numbers; a large max_q."""
    lens, news = [300, 0, 141, 16], [new, 2, new, 1]
    c, table, g, k, v = make(4, 8, 2, 128, BF16, 16, lens, seed=14)
    wide = torch.full((4, 40000), 2 ** 30, dtype=torch.int32, device="cuda")
    wide[:, :c.cfg.max_pages] = c.block_table
    d = paged4.PagedKVCache4(4, 8, 2, 128, BF16, page_size=16, n_pages=c.cfg.n_pages, max_pages=40000, pages=c.pages, block_table=wide,
                             kv_len=c.kv_len)
    cu = wl.seqlens_to_cu(news)
    q = randn(g, cu[-1] + 5, 8, 128, dtype=BF16).cuda()
    q[cu[-1]:] = float("nan")
    want = expect(c, k, v, q[:cu[-1]], lens, cu, True)
    for x in (c, d):
        for most in (max(news), 1 << 20):
            out, lse = torch.full_like(q, 7.0), torch.full((len(q), 8), 7.0, device="cuda")
            x.attend(q, cu_q=ints(cu), max_q=most, out=out, lse=lse, flags=paged.CAUSAL)
            assert x.get_error() == 0
            check(out, lse, want, f"{x.cfg.max_pages} columns, max_q {most}", cu[-1])
            assert torch.all(out[cu[-1]:] == 7.0) and torch.all(lse[cu[-1]:] == 7.0)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("new", [1, 40])
def test_queries_times_a_power_of_two(dtype, new):
    """Queries are taken as fp16 times a power of 2, row by row: 2^k times the queries under 2^-k times the scale give the same bits."""
    lens = [300, 77]
    c, table, g, k, v = make(2, 8, 2, 128, dtype, 16, lens, seed=15, scale=0.09)
    q = randn(g, 2 * new, 8, 128, dtype=dtype).cuda()
    want = c.attend(q, lse=True)
    for e in (-5, 4, -40, 50, -100, 90) if dtype == BF16 else (-2, 4, 12):
        d = paged4.PagedKVCache4(2, 8, 2, 128, dtype, page_size=16, n_pages=c.cfg.n_pages, max_pages=c.cfg.max_pages, pages=c.pages,
                                 block_table=c.block_table, kv_len=c.kv_len, softmax_scale=0.09 * 2.0 ** -e)
        x = (q.double() * 2.0 ** e).to(dtype)
        if not torch.equal(x.double(), q.double() * 2.0 ** e):
            x = None                                      # (fp16's elements below its normal range lose bits: not the same queries)
        got = d.attend(x if x is not None else q, lse=True)
        if x is not None:
            for a, b in zip(got, want):
                assert torch.equal(bits(a), bits(b)), e
        assert d.get_error() == 0


@pytest.mark.parametrize("new", [1, 40])
def test_queries_of_zero_and_infinity(new):
    """A zero query weighs all slots alike; one with an infinity spoils its own token and head alone."""
    lens = [300]
    c, table, g, k, v = make(1, 4, 2, 128, BF16, 16, lens, seed=16)
    q = randn(g, new, 4, 128, dtype=BF16)
    q[:, 0] = 0
    q[0, 3, 17] = float("inf")
    out, lse = c.attend(q.cuda(), lse=True)
    assert c.get_error() == 0
    want = expect(c, k, v, torch.nan_to_num(q, posinf=0.0), lens, None, False)
    assert torch.isnan(out[0, 3]).any()
    out[0, 3], lse[0, 3] = torch.from_numpy(want[0][0, 3]).to(BF16), float(want[1][0, 3])
    check(out, lse, want, "zero queries")
    assert np.allclose(to64(lse[:, 0]), np.log(300), atol=1e-5)


@pytest.mark.parametrize("new", [1, 40, 300])
def test_queries_of_zero_under_a_tiny_scale(new):
    """A zero row is brought up by 2^120, and the scale 2^-93 times what undoes that is below fp32: masked scores stay masked."""
    lens = [300, 45]
    c, table, g, k, v = make(2, 4, 2, 128, BF16, 16, lens, seed=22, scale=2.0 ** -93)
    q = torch.zeros(2 * new, 4, 128, dtype=BF16)
    out, lse = c.attend(q.cuda(), lse=True, flags=paged.CAUSAL)
    assert c.get_error() == 0
    check(out, lse, expect(c, k, v, q, lens, None, True), "zero queries, tiny scale")


def test_two_rows_may_share_pages():
    lens = [100, 100]
    c, table, g, k, v = make(2, 4, 2, 64, F16, 16, lens, seed=17)
    c.block_table[1] = c.block_table[0]
    q = randn(g, 2, 4, 64, dtype=F16)
    out, lse = c.attend(q.cuda(), lse=True)
    assert c.get_error() == 0
    check(out, lse, expect(c, [k[0], k[0]], [v[0], v[0]], q, lens, None, False), "shared pages")


def test_records_may_be_copied():
    """A row moved to other pages of another pool, by way of host memory."""
    lens = [100]
    c, table, g, k, v = make(1, 4, 2, 128, BF16, 32, lens, seed=18)
    d, other, _, _, _ = make(1, 4, 2, 128, BF16, 32, lens, seed=19, fill=False, extra=9)
    for j in range(4):
        d.pages[other[0, j]] = c.pages[table[0, j]].cpu().cuda()
    q = randn(g, 1, 4, 128, dtype=BF16).cuda()
    assert torch.equal(bits(c.attend(q)), bits(d.attend(q)))
    assert torch.equal(bits(c.read(100)[0]), bits(d.read(100)[0]))


def test_handles_on_two_streams_at_once():
    """A handle and a workspace each over one pool: steps and chunks on two streams, many times, give the same bits."""
    lens = [3000, 700]
    c, g, k, v = big(lens, 8, 2, 128, BF16, 16, seed=22)
    d = paged4.PagedKVCache4(2, 8, 2, 128, BF16, page_size=16, n_pages=c.cfg.n_pages, max_pages=c.cfg.max_pages, pages=c.pages,
                             block_table=c.block_table, kv_len=c.kv_len)
    q1 = torch.randn(2, 8, 128, device="cuda", generator=g).to(BF16)
    q2 = torch.randn(2 * 100, 8, 128, device="cuda", generator=g).to(BF16)
    want1, want2 = c.attend(q1), c.attend(q2, flags=paged.CAUSAL)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append((c.attend(q1, stream=a), d.attend(q2, flags=paged.CAUSAL, stream=b)))
        got.append((d.attend(q1, stream=b), c.attend(q2, flags=paged.CAUSAL, stream=a)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(bits(x), bits(want1)) and torch.equal(bits(y), bits(want2))
    ko, vo = c.read(sum(lens), cu=ints(wl.seqlens_to_cu(lens)), stream=a)
    a.synchronize()
    assert torch.equal(bits(ko), bits(torch.cat(k))) and torch.equal(bits(vo), bits(torch.cat(v)))
    assert c.get_error(stream=a) == 0 and d.get_error(stream=b.cuda_stream) == 0


def test_two_graphs_on_one_handle():
    """A step and a chunk captured on a handle, replayed back to back many times: they share counters and partials."""
    lens = [9000, 300]
    c, g, k, v = big(lens, 8, 2, 128, F16, 64, seed=23)
    q1 = torch.randn(2, 8, 128, device="cuda", generator=g).to(F16)
    q2 = torch.randn(2 * 40, 8, 128, device="cuda", generator=g).to(F16)
    want = c.attend(q1, lse=True) + c.attend(q2, lse=True, flags=paged.CAUSAL)
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        r1 = c.attend(q1, lse=True)
    with torch.cuda.graph(two):
        r2 = c.attend(q2, lse=True, flags=paged.CAUSAL)
    for i in range(30):
        for x in r1 + r2:
            x.fill_(7)
        one.replay(), two.replay(), one.replay()
        if i % 3:
            two.replay()
        for x, y in zip(r1 + r2, want):
            assert torch.equal(bits(x), bits(y))
    assert c.get_error() == 0


def test_outputs_aligned_to_16_bytes_and_no_more():
    lens = [500, 40]
    c, table, g, k, v = make(2, 8, 2, 64, BF16, 16, lens, seed=24)
    for new in (1, 30):
        n = 2 * new * 8 * 64
        q = randn(g, 2 * new, 8, 64, dtype=BF16)
        src, dst = torch.empty(n + 8, dtype=BF16, device="cuda"), torch.empty(n + 8, dtype=BF16, device="cuda")
        qa, out = src[8:].view(2 * new, 8, 64), dst[8:].view(2 * new, 8, 64)
        qa.copy_(q)
        lse = torch.empty(2 * new * 8 + 1, device="cuda")[1:].view(2 * new, 8)
        c.attend(qa, out=out, lse=lse, flags=paged.CAUSAL)
        assert c.get_error() == 0
        check(out, lse, expect(c, k, v, q, lens, None, True), "alignment")


@pytest.mark.parametrize("what", ["decode", "chunk", "chunk in waves"])
def test_calls_between_a_wait_that_ran_out_and_the_report(what):
    """They return; the bit stays until it is asked for; and what follows the report is right, calls and replays alike."""
    lens = [5000, 3000]
    heads, kv_heads = (24, 24) if "waves" in what else (8, 2)
    new = 300 if "chunk" in what else 1
    c, g, _, _ = big(lens, heads, kv_heads, 128, BF16, 16, seed=41)
    q = torch.randn(2, new, heads, 128, device="cuda", generator=g).to(BF16)
    run = lambda: c.attend(q, lse=True, flags=paged.CAUSAL)  # noqa: E731
    want = run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = run()
    assert c.get_error() == 0
    for _ in range(2):
        paged4.kvc_paged4_debug_stall_waits(c.handle, 200_000)
        run()
        paged4.kvc_paged4_debug_stall_waits(c.handle, 0)
        run()
        graph.replay()
        run()
        assert c.get_error() & paged.DEV_TIMEOUT
        assert c.get_error() == 0
        for x in replayed:
            x.fill_(7)
        graph.replay()
        got = run()
        assert c.get_error() == 0
        for x, y, z in zip(want, got, replayed):
            assert torch.equal(x, y) and torch.equal(x, z)


def test_reading_keys_or_values_alone_and_queries_turned_in_place():
    """By the C entry: either output may be missing.  q_out may be q where its rows are dense."""
    c, table, g, k, v = make(2, 4, 2, 64, BF16, 16, [20, 37], seed=26)
    cu, n = ints([0, 20, 57]), 57
    want = c.read(n, cu=cu)
    for i in range(2):
        out = torch.full((n, 2, 64), 7.0, dtype=BF16, device="cuda")
        ptr = [None, None]
        ptr[i] = out.data_ptr()
        assert kvc._lib.kvc_paged4_read(c.handle, *ptr, n, cu.data_ptr(), torch.cuda.current_stream().cuda_stream) == kvc.OK
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(want[i]))
    assert kvc._lib.kvc_paged4_read(c.handle, None, None, n, cu.data_ptr(), None) == kvc.ERR_ARG
    q = randn(g, n, 4, 64, dtype=BF16).cuda()
    kn, rope = randn(g, n, 2, 64, dtype=BF16).cuda(), wl.rope_table(64, 64).cuda()
    pos = torch.randint(0, 64, (n, 2), generator=g, dtype=torch.int32).cuda()
    for kw in (dict(), dict(positions=pos, axes=paged.rope_axes([j % 2 for j in range(32)])), dict(positions=pos, axes=paged.rope_axes([0] * 16 + [1] * 16))):
        turned_q = c.append(kn, kn, cu_new=cu, rope=rope, q=q, **kw)
        same = q.clone()
        assert c.append(kn, kn, cu_new=cu, rope=rope, q=same, q_out=same, **kw) is same
        assert torch.equal(bits(same), bits(turned_q))
    assert c.get_error() == 0


def test_refusals():
    c, table, g, k, v = make(2, 4, 2, 64, BF16, 16, [20, 20], seed=25)
    q = randn(g, 2, 4, 64, dtype=BF16).cuda()
    for flags in (256, 2, 512):                            # no FMA kernel, no other flag
        with pytest.raises(kvc.KvcError):
            c.attend(q, flags=flags)
    with pytest.raises(kvc.KvcError):
        c.attend(q, cu_q=ints([0, 1, 2]), max_q=0)
    with pytest.raises(kvc.KvcError):
        c.attend(torch.zeros(3, 4, 64, dtype=BF16, device="cuda"))          # three tokens for two rows
    with pytest.raises(ValueError):
        c.read(3)
    with pytest.raises(kvc.KvcError):
        c.read(0)
    for call in (c.attend_shared, c.attend_sparse):
        with pytest.raises(kvc.KvcError):
            call(q, 1)
    with pytest.raises(kvc.KvcError):
        paged4.PagedKVCache4(2, 4, 2, 64, torch.float32, page_size=16, n_pages=4, max_pages=2)
    with pytest.raises(ValueError):
        paged4.PagedKVCache4(2, 4, 2, 64, BF16, page_size=16, n_pages=4, max_pages=2, pages=torch.zeros(4, 2, 16 * 64, dtype=torch.uint8, device="cuda"))
    assert c.get_error() == 0
