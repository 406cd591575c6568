"""GPU tests of the paged cache as a server runs it: calls back to back under load, captured graphs on one handle, outputs
that are aligned no better than the interface asks, long chunks, and waits that run out.

A wait that runs out is made by the testing hook (a wait on a barrier that nothing signals, 200 us): the kernels return and
report it, nothing faults or hangs.
"""
import numpy as np
import pytest
import torch

from diffusion_serving_gb300 import workloads as wl
from tests import paged_ref as ref
from tests.helpers import to64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from diffusion_serving_gb300 import kvc, paged

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SIMT = 256


def bits(t):
    t = t.contiguous()
    return t.view(torch.int16) if t.element_size() == 2 else t.view(torch.int32)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def big(lens, heads, kv_heads, dim, dtype, page, *, seed, bounds=False, max_tokens=0):
    """Rows of `lens` tokens in pages in random order, all on the device."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    c = paged.PagedKVCache(len(lens), heads, kv_heads, dim, dtype, page_size=page, n_pages=sum(need), max_pages=max(need),
                           bounds=bounds, max_tokens=max_tokens)
    c.k_pages.normal_(generator=g)
    c.v_pages.normal_(generator=g)
    perm = torch.randperm(sum(need), generator=g, device="cuda").int()
    at = 0
    for b, p in enumerate(need):
        c.block_table[b, :p] = perm[at:at + p]
        at += p
    c.kv_len.copy_(ints(lens))
    if bounds:
        c.bounds.copy_(torch.stack([c.k_pages.amax(1), c.k_pages.amin(1)], 2))
    return c, g


def same_sums(lse, other):
    """Both kernels sum the weights in fp32, unrounded, of scores whose fp32 sums of 128 products of |x| < 6 are off by less
    than 128 2^-24 of a few hundred times the scale: 2^-12 holds both and the exponentials' own errors."""
    torch.testing.assert_close(lse, other, rtol=0, atol=2.0 ** -12)


@pytest.mark.parametrize("dtype,heads,kv_heads,dim,page,lens,new", [
    (BF16, 32, 8, 128, 64, [4500, 7000], [700, 1024]),
    (F16, 40, 40, 64, 16, [5200, 3000], [333, 300]),
    (BF16, 64, 64, 128, 128, [300, 9000, 40], [290, 129, 40]),       # one long row among short ones
])
def test_long_chunks_of_whole_and_cut_items(dtype, heads, kv_heads, dim, page, lens, new):
    """More items than blocks over long rows: whole ones first, the rest cut anywhere."""
    c, g = big(lens, heads, kv_heads, dim, dtype, page, seed=5)
    cu = wl.seqlens_to_cu(new)
    q = torch.randn(cu[-1], heads, dim, device="cuda", generator=g).to(dtype)
    args = dict(cu_q=ints(cu), max_q=max(new), lse=True)
    out, lse = c.attend(q, flags=paged.CAUSAL, **args)
    simt, lse_simt = c.attend(q, flags=paged.CAUSAL | SIMT, **args)
    assert c.get_error() == 0
    same_sums(lse, lse_simt)
    k, v, table = to64(c.k_pages), to64(c.v_pages), c.block_table.cpu().numpy()
    for b, n in enumerate(lens):
        kk, vv = ref.gather(k, table[b], 0, n), ref.gather(v, table[b], 0, n)
        for i in range(b, new[b], 97):
            t = cu[b] + i
            see = ref.visible_mask(n, 0, new[b], n, True)[i:i + 1]
            ref.check(out[t:t + 1], lse[t:t + 1], ref.attend_rows(to64(q[t:t + 1]), kk, vv, see, dim ** -0.5, dtype), f"token {t}")


@pytest.mark.parametrize("dtype,heads,kv_heads,dim", [(F16, 24, 24, 64), (BF16, 40, 8, 128)])
def test_long_chunks_behind_a_shared_prefix(dtype, heads, kv_heads, dim):
    """Items cut and joined next to the prefix's state."""
    lens, new, P = [8000, 700, 256], [300, 200, 33], 256
    c, g = big(lens, heads, kv_heads, dim, dtype, 32, seed=15, max_tokens=540)
    pages = c.block_table[0, :P // 32].clone()
    c.block_table[:, :P // 32] = pages
    cu = wl.seqlens_to_cu(new)
    q = torch.randn(cu[-1], heads, dim, device="cuda", generator=g).to(dtype)
    args = dict(cu_q=ints(cu), max_q=max(new), lse=True)
    out, lse = c.attend_shared(q, pages, ints([P]), flags=paged.CAUSAL, **args)
    _, lse_simt = c.attend(q, flags=paged.CAUSAL | SIMT, **args)
    assert c.get_error() == 0
    same_sums(lse, lse_simt)
    k, v, table = to64(c.k_pages), to64(c.v_pages), c.block_table.cpu().numpy()
    for b, n in enumerate(lens):
        kk, vv = ref.gather(k, table[b], 0, n), ref.gather(v, table[b], 0, n)
        for i in range(b, new[b], 41):
            t = cu[b] + i
            see = ref.visible_mask(n, 0, new[b], n, True)[i:i + 1]
            ref.check(out[t:t + 1], lse[t:t + 1], ref.attend_rows(to64(q[t:t + 1]), kk, vv, see, dim ** -0.5, dtype), f"token {t}")


@pytest.mark.parametrize("new", [1, 4])
def test_decode_back_to_back_under_load(new):
    """Calls on two handles follow each other without a pause, rows from short to long, more data than L2 holds."""
    lens = [17 + 449 * i for i in range(20)]
    cs = [big(lens, 32, 8, 128, dt, 16, seed=6 + i) for i, dt in enumerate((BF16, F16))]
    want, bufs, qs = [], [], []
    for (c, g), dt in zip(cs, (BF16, F16)):
        q = torch.randn(len(lens), new, 32, 128, device="cuda", generator=g).to(dt)
        want.append(c.attend(q, lse=True, flags=paged.CAUSAL))
        same_sums(want[-1][1], c.attend(q, lse=True, flags=paged.CAUSAL | SIMT)[1])
        qs.append(q)
        bufs.append([torch.empty_like(q) for _ in range(25)])
    torch.cuda.synchronize()
    for _ in range(4):
        for i in range(25):
            for (c, _), q, b in zip(cs, qs, bufs):
                c.attend(q, out=b[i], flags=paged.CAUSAL)
    torch.cuda.synchronize()
    for (c, _), w, b in zip(cs, want, bufs):
        assert c.get_error() == 0
        for x in b:
            assert torch.equal(bits(x), bits(w[0]))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_two_graphs_of_one_handle_replayed_in_turn(dtype):
    """A decode step (append, shared, sparse) and a chunk, each captured, replayed in turn on one workspace as the lengths
    on the device grow; the same calls made one by one give the same bits."""
    B, heads, kv_heads, dim, page, P = 3, 8, 2, 128, 16, 64
    rope = wl.rope_table(512, dim).cuda()

    def cache():
        c = paged.PagedKVCache(B, heads, kv_heads, dim, dtype, page_size=page, n_pages=80, max_pages=24, bounds=True, max_tokens=64)
        g = torch.Generator(device="cuda").manual_seed(8)
        for t in (c.k_pages, c.v_pages, c.bounds):
            t.zero_()
        table = torch.full((B, 24), -1, dtype=torch.int32)
        for b in range(B):
            table[b, :4] = torch.arange(4)
            table[b, 4:24] = 4 + b * 20 + torch.arange(20)
        c.block_table.copy_(table)
        c.kv_len.copy_(ints([P, 0, 0]))
        c.append(torch.randn(P, kv_heads, dim, device="cuda", generator=g).to(dtype),
                 torch.randn(P, kv_heads, dim, device="cuda", generator=g).to(dtype), cu_new=ints([0, P, P, P]), rope=rope)
        c.kv_len.fill_(P)
        return c, g

    shared, plen, cu = ints([0, 1, 2, 3]), ints([P]), ints([0, 17, 17, 40])

    def buffers():
        z = lambda *s: torch.zeros(*s, device="cuda").to(dtype)  # noqa: E731
        return dict(k=z(B, 1, kv_heads, dim), v=z(B, 1, kv_heads, dim), q=z(B, 1, heads, dim), qr=z(B, 1, heads, dim),
                    o1=z(B, 1, heads, dim), o2=z(B, heads, dim), sel=torch.zeros(B, kv_heads, 3, dtype=torch.int32, device="cuda"),
                    ck=z(40, kv_heads, dim), cv=z(40, kv_heads, dim), cq=z(40, heads, dim), cqr=z(40, heads, dim), co=z(40, heads, dim))

    def step(c, s):
        c.kv_len.add_(1)
        c.append(s["k"], s["v"], rope=rope, q=s["q"], q_out=s["qr"])
        c.attend_shared(s["qr"], shared, plen, out=s["o1"])
        c.attend_sparse(s["qr"].view(B, heads, dim), 3, out=s["o2"], selected=s["sel"])

    grow = ints([17, 0, 23])

    def chunk(c, s):
        c.kv_len.add_(grow)
        c.append(s["ck"], s["cv"], cu_new=cu, rope=rope, q=s["cq"], q_out=s["cqr"])
        c.attend(s["cqr"], cu_q=cu, max_q=23, out=s["co"], flags=paged.CAUSAL)

    (c, _), (d, _) = cache(), cache()
    sc, sd = buffers(), buffers()
    at = c.kv_len.clone()
    graphs = []
    pool = [t.clone() for t in (c.k_pages, c.v_pages, c.bounds)]
    side = torch.cuda.Stream()
    for f in (step, chunk):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            f(c, sc)                                             # (warm-up)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f(c, sc)
        graphs.append(graph)
    c.kv_len.copy_(at)
    for t, x in zip((c.k_pages, c.v_pages, c.bounds), pool):
        t.copy_(x)
    g = torch.Generator(device="cuda").manual_seed(9)
    for turn in range(8):
        for key in ("k", "v", "q", "ck", "cv", "cq"):
            sc[key].copy_(torch.randn(sc[key].shape, device="cuda", generator=g))
            sd[key].copy_(sc[key])
        which = 1 if turn in (2, 5) else 0
        graphs[which].replay()
        (step, chunk)[which](d, sd)
        assert torch.equal(c.kv_len, d.kv_len)
        for key in (("co", "cqr") if which else ("o1", "o2", "sel", "qr")):
            assert torch.equal(bits(sc[key]), bits(sd[key])), (turn, key)
        for x, y in ((c.k_pages, d.k_pages), (c.v_pages, d.v_pages), (c.bounds, d.bounds)):
            assert torch.equal(bits(x), bits(y)), turn
    assert c.get_error() == 0 and d.get_error() == 0


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("new", [1, 33])
def test_buffers_aligned_to_16_bytes_only(dtype, new):
    """Queries and outputs at every multiple of 16 bytes, sums at every multiple of 4."""
    lens = [300, 77]
    c, g = big(lens, 8, 2, 64, dtype, 16, seed=11, bounds=True, max_tokens=80)
    n = 2 * new
    vec = 16 // torch.empty(0, dtype=dtype).element_size()
    q = torch.randn(n, 8, 64, device="cuda", generator=g).to(dtype)
    pages, plen = c.block_table[0, :4].clone(), ints([64])
    c.block_table[1, :4] = pages
    want = [c.attend(q, lse=True, flags=paged.CAUSAL), c.attend_shared(q, pages, plen, lse=True, flags=paged.CAUSAL)]
    for off in (1, 2, 3):
        qb = torch.zeros(q.numel() + 8 * vec, dtype=dtype, device="cuda")
        ob = torch.full_like(qb, 7.0)
        lb = torch.full((n * 8 + 8,), 7.0, device="cuda")
        qv, ov = (t[off * vec:off * vec + q.numel()].view_as(q) for t in (qb, ob))
        lv = lb[off:off + n * 8].view(n, 8)
        qv.copy_(q)
        for i in range(2):
            if i == 0:
                c.attend(qv, out=ov, lse=lv, flags=paged.CAUSAL)
            else:
                c.attend_shared(qv, pages, plen, out=ov, lse=lv, flags=paged.CAUSAL)
            assert torch.equal(bits(ov), bits(want[i][0])) and torch.equal(lv, want[i][1])
            assert torch.all(ob[:off * vec] == 7.0) and torch.all(ob[off * vec + q.numel():] == 7.0)
            assert torch.all(lb[:off] == 7.0) and torch.all(lb[off + n * 8:] == 7.0)
        if new == 1:
            a = c.attend_sparse(q, 4)
            b = c.attend_sparse(qv, 4, out=ov)
            assert torch.equal(bits(a[0]), bits(ov)) and torch.equal(a[1], b[1])
    assert c.get_error() == 0


def against_plain(c, q, out, lse, cu, causal, rows, sel=None):
    """Rows `rows` of a call against the plain form."""
    k, v, table, lens = to64(c.k_pages), to64(c.v_pages), c.block_table.cpu().numpy(), c.kv_len.tolist()
    for b in rows:
        n, t0, t1 = lens[b], cu[b], cu[b + 1]
        kk, vv = ref.gather(k, table[b], 0, n), ref.gather(v, table[b], 0, n)
        see = ref.visible_mask(n, 0, t1 - t0, n, causal)
        want = ref.attend_rows(to64(q[t0:t1]), kk, vv, see, c.head_dim ** -0.5, c.dtype)
        ref.check(out[t0:t1], lse[t0:t1], want, f"row {b}")


@pytest.mark.parametrize("dtype,heads,kv_heads,dim", [(BF16, 4, 2, 128), (F16, 6, 1, 64), (F32, 2, 2, 64)])
def test_the_largest_batch(dtype, heads, kv_heads, dim):
    """1024 rows: single tokens, ragged chunks, a shared prefix both ways, chosen pages, appends."""
    B, page = 1024, 16
    lens = [1 + (37 * b) % 90 for b in range(B)]
    c, g = big(lens, heads, kv_heads, dim, dtype, page, seed=21, bounds=True, max_tokens=4 * B)
    some = list(range(0, B, 61)) + [B - 1]
    q = torch.randn(B, heads, dim, device="cuda", generator=g).to(dtype)
    one = list(range(B + 1))
    out, lse = c.attend(q, lse=True)
    against_plain(c, q, out, lse, one, False, some)
    new = [b % 5 if b % 7 else 70 for b in range(B)]
    new = [min(n, m) for n, m in zip(new, lens)]
    cu = wl.seqlens_to_cu(new)
    qc = torch.randn(cu[-1], heads, dim, device="cuda", generator=g).to(dtype)
    for most in (max(new), 1 << 30):
        out, lse = c.attend(qc, cu_q=ints(cu), max_q=most, lse=True, flags=paged.CAUSAL)
        against_plain(c, qc, out, lse, cu, True, [b for b in some if new[b]])
    pages = torch.arange(2, dtype=torch.int32, device="cuda")
    c.block_table[:, :2] = pages                                 # (rows of one page see the first slots of a full one)
    for P in (32, 0):
        out, lse = c.attend_shared(q, pages, ints([P]), lse=True)
        against_plain(c, q, out, lse, one, False, some)
        q4 = torch.randn(4 * B, heads, dim, device="cuda", generator=g).to(dtype)
        out, lse = c.attend_shared(q4, pages, ints([P]), lse=True, flags=paged.CAUSAL)
        against_plain(c, q4, out, lse, list(range(0, 4 * B + 1, 4)), True, some)
    out, lse, sel = c.attend_sparse(q, 3, lse=True)
    full = c.kv_len.cpu().numpy() <= 3 * page
    assert all(sel[b, :, :-(-lens[b] // page)].tolist() == [list(range(-(-lens[b] // page)))] * kv_heads for b in some if full[b])
    against_plain(c, q, out, lse, one, False, [b for b in some if full[b]])
    assert c.get_error() == 0


@pytest.mark.parametrize("heads,kv_heads", [(71, 1), (96, 1), (128, 2)])
def test_wide_groups(heads, kv_heads):
    """Groups of 71 (a prime), 96 and 64 heads."""
    lens, new = [900, 130, 47], [3, 40, 1]
    c, g = big(lens, heads, kv_heads, 64, BF16, 32, seed=22, bounds=True)
    q = torch.randn(3, heads, 64, device="cuda", generator=g).to(BF16)
    out, lse = c.attend(q, lse=True)
    against_plain(c, q, out, lse, [0, 1, 2, 3], False, range(3))
    cu = wl.seqlens_to_cu(new)
    qc = torch.randn(cu[-1], heads, 64, device="cuda", generator=g).to(BF16)
    out, lse = c.attend(qc, cu_q=ints(cu), max_q=40, lse=True, flags=paged.CAUSAL)
    against_plain(c, qc, out, lse, cu, True, range(3))
    # more places than any row has pages: everything is attended
    out, lse, sel = c.attend_sparse(q, c.cfg.max_pages + 9, lse=True)
    against_plain(c, q, out, lse, [0, 1, 2, 3], False, range(3))
    assert sel[0, 0].tolist() == list(range(29)) + [-1] * (sel.shape[2] - 29)
    # one place
    _, sel = c.attend_sparse(q, 1, first=0, recent=0)
    bd, table = to64(c.bounds), c.block_table.cpu().numpy()
    for b, n in enumerate(lens):
        assert sel[b].tolist() == ref.select(to64(q[b]), bd, table[b], -(-n // 32), 1, 0, 0)
    assert c.get_error() == 0


def test_as_many_pages_as_selection_takes():
    """32768 columns, and one more refused."""
    page, n = 16, 32768
    c, g = big([n * page - 5, 1], 8, 1, 64, BF16, page, seed=23, bounds=True)
    q = torch.randn(2, 8, 64, device="cuda", generator=g).to(BF16)
    out, sel = c.attend_sparse(q, 600)
    bd, table = to64(c.bounds), c.block_table.cpu().numpy()
    assert sel[0].tolist() == ref.select(to64(q[0]), bd, table[0], n, 600, 1, 1)
    assert sel[1, 0, 0] == 0 and torch.all(sel[1, 0, 1:] == -1)
    assert c.get_error() == 0
    d = paged.PagedKVCache(1, 8, 1, 64, BF16, page_size=page, n_pages=4, max_pages=n + 1, bounds=True)
    with pytest.raises(kvc.KvcError) as e:
        d.attend_sparse(q[:1], 4)
    assert e.value.code == kvc.ERR_RANGE


def test_what_the_entry_points_refuse():
    c, g = big([100, 60], 8, 2, 64, BF16, 16, seed=12, max_tokens=4)
    q = torch.randn(2, 8, 64, device="cuda", generator=g).to(BF16)
    pages, plen = c.block_table[0, :2].clone(), ints([32])
    keep = torch.full_like(q, 7.0)

    def refused(code, f):
        with pytest.raises(kvc.KvcError) as e:
            f()
        assert e.value.code == code
        torch.cuda.synchronize()
        assert torch.all(keep == 7.0)

    refused(kvc.ERR_UNSUPPORTED, lambda: c.attend_sparse(q, 4, out=keep))                    # no bounds
    c2, _ = big([100, 60], 8, 2, 64, BF16, 16, seed=12, bounds=True)
    refused(kvc.ERR_ARG, lambda: c2.attend_sparse(q, 4, first=3, recent=2, out=keep))
    refused(kvc.ERR_ARG, lambda: c2.attend_sparse(q, 4, first=-1, out=keep))
    refused(kvc.ERR_ARG, lambda: c2.attend_sparse(q, 4, out=keep, flags=paged.CAUSAL))
    refused(kvc.ERR_ARG, lambda: c.attend(q, out=keep, flags=2))
    refused(kvc.ERR_ARG, lambda: c.attend(q, cu_q=ints([0, 1, 2]), max_q=0, out=keep))
    refused(kvc.ERR_ARG, lambda: c.attend_shared(q, ints([0] * 40), plen, out=keep))          # longer than the table
    q6 = torch.randn(6, 8, 64, device="cuda", generator=g).to(BF16)
    refused(kvc.ERR_RANGE, lambda: c.attend_shared(q6, pages, plen))                          # more than max_tokens
    k = torch.randn(2, 2, 64, device="cuda", generator=g).to(BF16)
    refused(kvc.ERR_ARG, lambda: c.append(k, k, q=q, q_out=keep))                             # queries without a table
    assert c.get_error() == 0 and c2.get_error() == 0


def test_shared_prefix_in_a_pass_of_its_own_refuses_bad_lengths():
    lens, P = [4100 + i for i in range(26)], 4096
    c, g = big(lens, 8, 2, 128, BF16, 16, seed=14, max_tokens=26)
    q = torch.randn(26, 8, 128, device="cuda", generator=g).to(BF16)
    pages = c.block_table[0, :P // 16].clone()
    c.block_table[:, :P // 16] = pages
    want, lse = c.attend(q, lse=True)
    for bad in (-16, 8, P + 16, -2 ** 31):
        out = torch.full_like(q, 7.0)
        c.attend_shared(q, pages, ints([bad]), out=out)
        assert c.get_error() & paged.DEV_BAD_KVLEN
        assert torch.all(out == 7.0)
    got, lse2 = c.attend_shared(q, pages, ints([P]), lse=True)
    assert c.get_error() == 0
    same_sums(lse, lse2)
    got, lse2 = c.attend_shared(q, pages, ints([0]), lse=True)   # the prefix may shrink to nothing on the device
    assert c.get_error() == 0
    same_sums(lse, lse2)


@pytest.mark.parametrize("what", ["decode", "decode over many blocks", "chunk", "chunk in waves", "shared", "shared of many rows"])
def test_wait_that_runs_out_returns_and_reports(what):
    lens = [5000, 3000] if "many blocks" in what else [700, 400] + [500] * (100 if "many rows" in what else 0)
    heads, kv_heads = (24, 24) if "waves" in what else (32, 8) if "rows" in what else (8, 2)
    new = 300 if "chunk" in what else 1
    c, g = big(lens, heads, kv_heads, 128, BF16, 16, seed=13, max_tokens=len(lens))
    q = torch.randn(len(lens), new, heads, 128, device="cuda", generator=g).to(BF16)
    pages, plen = c.block_table[0, :20].clone(), ints([320])
    c.block_table[:, :20] = pages
    run = (lambda: c.attend_shared(q, pages, plen, lse=True)) if "shared" in what else \
        (lambda: c.attend(q, lse=True, flags=paged.CAUSAL))
    want = run()
    assert c.get_error() == 0
    paged.kvc_paged_debug_stall_waits(c.handle, 200_000)
    run()                                              # returns; its output is not defined
    assert c.get_error() & paged.DEV_TIMEOUT
    assert c.get_error() == 0                          # reported once, then cleared
    paged.kvc_paged_debug_stall_waits(c.handle, 0)
    for _ in range(2):
        out, lse = run()
        assert c.get_error() == 0
        assert torch.equal(bits(out), bits(want[0])) and torch.equal(lse, want[1])
