"""GPU tests of the paged cache: append, attention of tokens and chunks, over a shared prefix, over selected pages.

Everything is compared with plain 64-bit forms (tests/paged_ref.py), stores and rotations bit for bit.
"""
import numpy as np
import pytest
import torch

from diffusion_serving_gb300 import workloads as wl
from oracle import kvc_oracle as orc
from tests import paged_ref as ref
from tests.helpers import to64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from diffusion_serving_gb300 import paged

FMT = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SIMT = 256


def bits(t):
    t = t.contiguous()
    return t.view(torch.int16) if t.element_size() == 2 else t.view(torch.int32)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(batch, heads, kv_heads, dim, dtype, page, lens, *, seed=1, extra=2, bounds=None, max_tokens=0, fill=True,
         shared=0, scale=0.0):
    """A cache whose rows hold `lens` tokens in pages handed out in random order; rows share their first `shared` pages.
    Slots that no row fills hold NaN."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    n_pages = shared + sum(max(0, p - shared) for p in need) + extra
    c = paged.PagedKVCache(batch, heads, kv_heads, dim, dtype, page_size=page, n_pages=n_pages,
                           max_pages=max(max(need), shared, 1) + 1, bounds=bounds, max_tokens=max_tokens, softmax_scale=scale)
    perm = torch.randperm(n_pages, generator=g).tolist()
    table = np.full((batch, c.cfg.max_pages), -7, dtype=np.int64)
    at = shared
    for b, p in enumerate(need):
        table[b, :min(p, shared)] = perm[:min(p, shared)]
        for j in range(shared, p):
            table[b, j] = perm[at]
            at += 1
    c.block_table.copy_(torch.from_numpy(table).int())
    c.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
    k = torch.full((n_pages, page, kv_heads, dim), float("nan"))
    v = torch.full((n_pages, page, kv_heads, dim), float("nan"))
    if fill:
        for b, n in enumerate(lens):
            for j in range(need[b]):
                m = min(page, n - j * page)
                pg = table[b, j]
                have = int((~torch.isnan(k[pg, :, 0, 0])).sum())
                if have < m:
                    k[pg, have:m] = torch.randn(m - have, kv_heads, dim, generator=g)
                    v[pg, have:m] = torch.randn(m - have, kv_heads, dim, generator=g)
    c.k_pages.copy_(k.to(dtype))
    c.v_pages.copy_(v.to(dtype))
    c.perm = perm
    return c, table, g


def randn(g, *shape, dtype):
    return torch.randn(*shape, generator=g).to(dtype)


def rows_of(cu, b, n_tokens, batch):
    if cu is None:
        n = n_tokens // batch
        return b * n, n
    return cu[b], cu[b + 1] - cu[b]


def expect(c, table, q, lens, cu, causal, start=0):
    """(out, lse, bounds) of every token by the plain form; rows one by one."""
    k, v = to64(c.k_pages), to64(c.v_pages)
    qn = to64(q).reshape(-1, c.heads, c.head_dim)
    scale = c.cfg.softmax_scale or c.head_dim ** -0.5
    out = [np.zeros(qn.shape), np.full(qn.shape[:2], -np.inf), np.zeros(qn.shape), np.zeros(qn.shape[:2])]
    for b, n in enumerate(lens):
        t0, m = rows_of(cu, b, len(qn), c.batch)
        kk, vv = ref.gather(k, table[b], 0, n), ref.gather(v, table[b], 0, n)
        got = ref.attend_rows(qn[t0:t0 + m], kk, vv, ref.visible_mask(n, 0, m, n, causal), scale, c.dtype)
        for dst, x in zip(out, got):
            dst[t0:t0 + m] = x
    return out


def check(got, lse, want, what, n=None):
    n = want[0].shape[0] if n is None else n
    got = got.reshape(-1, *want[0].shape[1:])[:n]
    lse = None if lse is None else lse.reshape(-1, want[1].shape[1])[:n]
    ref.check(got, lse, [x[:n] for x in want], what)


# ------------------------------------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dim,kv_heads,page", [(128, 8, 16), (64, 3, 64), (128, 20, 32), (64, 1, 128)])
def test_append_packed_rows_rotated_bit_exact(dtype, half, dim, kv_heads, page):
    heads = 2 * kv_heads
    lens, new = [37, 1, 300, 64, 129], [20, 1, 0, 64, 3]
    c, table, g = make(5, heads, kv_heads, dim, dtype, page, lens, bounds=True, seed=3)
    before_k, before_v = c.k_pages.clone(), c.v_pages.clone()
    # pages of the old tokens have their bounds; those of new tokens hold nonsense
    c.bounds.fill_(99.0)
    kp = to64(c.k_pages)
    for b, (n, m) in enumerate(zip(lens, new)):
        if (n - m) % page:
            pg, f = table[b, (n - m) // page], (n - m) % page
            c.bounds[pg].copy_(torch.from_numpy(ref.page_bounds(kp, pg, f).swapaxes(0, 1)).to(dtype))
    before_b = c.bounds.clone()
    cu = wl.seqlens_to_cu(new)
    total = cu[-1] + 4                                  # rows behind the last sequence
    joint = randn(g, total, heads + 2 * kv_heads, dim, dtype=dtype).cuda()
    q, k, v = joint[:, :heads], joint[:, heads:heads + kv_heads], joint[:, heads + kv_heads:]
    table_rope = wl.rope_table(400, dim)
    q_out = torch.full((total, heads, dim), 7.0, dtype=dtype, device="cuda")
    c.append(k, v, cu_new=ints(cu), rope=table_rope.cuda(), half=half, q=q, q_out=q_out)
    assert c.get_error() == 0

    def turned(x, pos):
        """orc.rope_store turns interleaved pairs: halves are interleaved for it, and taken apart again."""
        x = to64(x)
        if half:
            x = np.stack([x[..., :dim // 2], x[..., dim // 2:]], -1).reshape(x.shape)
        y = orc.rope_store(x, pos, table_rope.numpy(), FMT[dtype])
        if half:
            y = np.concatenate([y[..., 0::2], y[..., 1::2]], -1)
        return torch.from_numpy(y).to(dtype)

    want_k, want_v = before_k.cpu(), before_v.cpu()
    for b, (n, m) in enumerate(zip(lens, new)):
        pos = list(range(n - m, n))
        kb = turned(k[cu[b]:cu[b] + m], pos) if m else None
        for i, p in enumerate(pos):
            want_k[table[b, p // page], p % page] = kb[i]
            want_v[table[b, p // page], p % page] = v[cu[b] + i].cpu()
        if m:
            assert torch.equal(bits(q_out[cu[b]:cu[b] + m].cpu()), bits(turned(q[cu[b]:cu[b] + m], pos)))
    assert torch.equal(bits(c.k_pages.cpu()), bits(want_k))
    assert torch.equal(bits(c.v_pages.cpu()), bits(want_v))
    assert torch.all(q_out[cu[-1]:] == 7.0)
    kp = to64(c.k_pages)
    touched = {}
    for b, (n, m) in enumerate(zip(lens, new)):
        for p in range(n - m, n):
            touched[table[b, p // page]] = p % page + 1
    for pg in range(c.cfg.n_pages):
        if pg in touched:
            want = ref.page_bounds(kp, pg, touched[pg]).swapaxes(0, 1)
            assert np.array_equal(to64(c.bounds[pg]), want), pg
        else:
            assert torch.equal(bits(c.bounds[pg]), bits(before_b[pg]))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append_even_rows_without_rotation_and_token_by_token(dtype):
    """[batch, n, ...] rows as they come; a prompt, then single tokens, equal to one append of all."""
    lens = [45, 45, 45]
    c, table, g = make(3, 4, 2, 64, dtype, 16, lens, bounds=True, seed=5)
    d, _, _ = make(3, 4, 2, 64, dtype, 16, lens, bounds=True, seed=5)
    k, v = randn(g, 3, 45, 2, 64, dtype=dtype).cuda(), randn(g, 3, 45, 2, 64, dtype=dtype).cuda()
    c.append(k, v)
    for lo, hi in [(0, 30)] + [(i, i + 1) for i in range(30, 45)]:
        d.kv_len.fill_(hi)
        d.append(k[:, lo:hi].contiguous(), v[:, lo:hi].contiguous())
    assert c.get_error() == 0 and d.get_error() == 0
    for b in range(3):
        got = ref.gather(to64(c.k_pages), table[b], 0, 45)
        assert np.array_equal(got, to64(k[b]))
    for x, y in ((c.k_pages, d.k_pages), (c.v_pages, d.v_pages)):
        assert torch.equal(bits(x), bits(y))
    used = sorted({int(p) for b in range(3) for p in table[b, :3]})
    assert torch.equal(bits(c.bounds[used]), bits(d.bounds[used]))


def test_append_reports_bad_rows_and_leaves_them():
    lens = [20, 20, 20, 20]
    c, table, g = make(4, 4, 2, 64, BF16, 16, lens, seed=6)
    k = randn(g, 8, 2, 64, dtype=BF16).cuda()
    before = c.k_pages.clone()
    rope = wl.rope_table(19, 64).cuda()                 # position 19 is outside
    c.kv_len.copy_(ints([20, 1, 500, 20]))              # row 1 shorter than its tokens, row 2 past the table's columns
    c.block_table[3, 1] = 10 ** 6
    c.append(k, k, cu_new=ints([0, 2, 4, 6, 8]), rope=rope)
    assert c.get_error() == paged.DEV_BAD_KVLEN | paged.DEV_BAD_PAGE | paged.DEV_BAD_POS
    want = before.clone()
    got = c.k_pages
    pg = int(table[0, 1])
    assert not torch.equal(bits(got[pg, 2]), bits(before[pg, 2]))      # row 0, position 18: written
    want[pg, 2] = got[pg, 2]
    assert torch.equal(bits(got), bits(want))
    c.kv_len.copy_(ints(lens))
    c.append(k, k, cu_new=ints([0, 3, 1, 9, 8]))        # row 1 goes backward, row 2 past the tokens, row 3 backward
    assert c.get_error() & paged.DEV_BAD_CUSEQ


def test_append_in_place_queries_and_graph_replay():
    """q_out may be q; a captured step of length update, append and attention follows the device's lengths."""
    lens = [3, 17]
    c, table, g = make(2, 4, 2, 64, F16, 16, [60, 60], seed=8, fill=False)
    c.k_pages.zero_()
    c.v_pages.zero_()
    c.kv_len.copy_(ints([0, 14]))
    rope = wl.rope_table(64, 64).cuda()
    k, v, q = (torch.zeros(2, 1, n, 64, dtype=F16, device="cuda") for n in (2, 2, 4))
    out, lse = torch.empty_like(q), torch.empty(2, 1, 4, device="cuda")

    def step():
        c.kv_len.add_(1)
        c.append(k, v, rope=rope, q=q, q_out=q)
        c.attend(q, out=out, lse=lse)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()                                          # (not captured: writes zeros)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    c.kv_len.copy_(ints([0, 14]))
    lens = [0, 14]
    for _ in range(20):
        k.copy_(randn(g, 2, 1, 2, 64, dtype=F16))
        v.copy_(randn(g, 2, 1, 2, 64, dtype=F16))
        q.copy_(randn(g, 2, 1, 4, 64, dtype=F16))
        q0 = q.clone()
        graph.replay()
        lens = [n + 1 for n in lens]
        for b in range(2):
            turned = orc.rope_store(to64(q0[b]), [lens[b] - 1], rope.cpu().numpy(), "f16")
            assert np.array_equal(to64(q[b]), turned)
        check(out, lse, expect(c, table, q, lens, None, False), f"replay at {lens}")
    assert c.get_error() == 0


# ------------------------------------------------------------------------------------------------ attend
ATTEND = [
    # heads, kv_heads, dim, page, lens, new (None: one each), causal
    (32, 8, 128, 16, [490], None, False),
    (4, 4, 128, 64, [1, 2, 63, 64, 65, 127, 128, 129], None, False),
    (8, 1, 64, 16, [0, 5, 1000, 0, 333], None, False),
    (12, 4, 64, 32, [700, 31, 33], [1, 4, 0], True),
    (40, 8, 128, 128, [300, 140, 2], [3, 1, 2], True),
    (6, 2, 64, 16, [200, 64], [60, 64], True),
    (8, 2, 128, 32, [513, 129, 40, 300], [130, 129, 1, 0], True),
    (4, 2, 128, 64, [1100], [300], False),
    (4, 4, 64, 128, [3, 0, 260], [5, 2, 200], True),        # more tokens than slots: the first see nothing
    (36, 2, 64, 16, [90, 17], [2, 9], True),                # groups of 18 heads
    (34, 2, 128, 16, [70], [40], True),                     # a group of 17
    (16, 1, 128, 16, [2000], [33], True),
    (16, 8, 64, 64, [150, 290, 160, 30, 133], [140, 150, 150, 0, 133], True),   # more items than blocks
    (12, 12, 128, 16, [400, 131], [260, 129], False),
    (16, 8, 64, 64, [1500, 1400], [700, 700], False),       # and the rest of them cut in the middle of long rows
    (24, 24, 128, 32, [900, 1000], [400, 500], True),
]


@pytest.mark.parametrize("simt", [0, SIMT])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attend(case, dtype, simt):
    heads, kv_heads, dim, page, lens, new, causal = ATTEND[case]
    c, table, g = make(len(lens), heads, kv_heads, dim, dtype, page, lens, seed=10 + case)
    cu = None if new is None else wl.seqlens_to_cu(new)
    total = len(lens) if cu is None else cu[-1] + 3
    q = randn(g, total, heads, dim, dtype=dtype).cuda()
    out = torch.full_like(q, 7.0)
    lse = torch.full((total, heads), 7.0, device="cuda")
    flags = simt | (paged.CAUSAL if causal else 0)
    c.attend(q, cu_q=None if cu is None else ints(cu), max_q=None if new is None else max(new), out=out, lse=lse, flags=flags)
    assert c.get_error() == 0
    want = expect(c, table, q, lens, cu, causal)
    n = total if cu is None else cu[-1]
    check(out, lse, want, f"case {case}", n)
    assert torch.all(out[n:] == 7.0) and torch.all(lse[n:] == 7.0)
    again = c.attend(q, cu_q=None if cu is None else ints(cu), max_q=None if new is None else max(new), flags=flags)
    assert torch.equal(bits(again[:n]), bits(out[:n]))       # the same call, the same bits


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens,new", [([6000, 1], [1, 1]), ([3000, 2900, 17], [16, 3, 1]), ([5000], [150])])
def test_attend_long_rows_split_over_blocks(dtype, lens, new):
    c, table, g = make(len(lens), 8, 2, 128, dtype, 16, lens, seed=31)
    cu = wl.seqlens_to_cu(new)
    q = (3 * randn(g, cu[-1], 8, 128, dtype=dtype).float()).to(dtype).cuda()
    out, lse = c.attend(q, cu_q=ints(cu), max_q=max(new), lse=True, flags=paged.CAUSAL)
    assert c.get_error() == 0
    check(out, lse, expect(c, table, q, lens, cu, True), f"{lens}")


@pytest.mark.parametrize("dtype", [F16, F32])
def test_attend_leaves_bad_rows_and_bad_pages_out(dtype):
    lens = [100, 100, 100]
    c, table, g = make(3, 4, 2, 64, dtype, 16, lens, seed=33)
    q = randn(g, 3, 4, 64, dtype=dtype).cuda()
    good = c.attend(q)
    c.kv_len.copy_(ints([100, -1, 10 ** 6]))
    out = torch.full_like(q, 7.0)
    c.attend(q, out=out)
    assert c.get_error() == paged.DEV_BAD_KVLEN
    assert torch.equal(bits(out[0]), bits(good[0])) and torch.all(out[1:] == 7.0)
    c.kv_len.copy_(ints(lens))
    c.block_table[1, 2] = c.cfg.n_pages                  # one bad page: its 16 slots are left out
    c.block_table[2, :7] = -1                            # no good page at all
    out, lse = c.attend(q, lse=True)
    assert c.get_error() == paged.DEV_BAD_PAGE
    assert torch.equal(bits(out[0]), bits(good[0]))
    kk = ref.gather(to64(c.k_pages), table[1], 0, 100)
    vv = ref.gather(to64(c.v_pages), table[1], 0, 100)
    see = np.ones((1, 100), bool)
    see[0, 32:48] = False
    want = ref.attend_rows(to64(q[1:2]), kk, vv, see, 64 ** -0.5, dtype)
    ref.check(out[1:2], lse[1:2], want, "bad page")
    assert torch.all(out[2] == 0) and torch.all(torch.isneginf(lse[2]))
    out.fill_(7.0)
    c.attend(q, cu_q=ints([0, 1, 3, 3]), max_q=1, out=out)     # row 1 has more tokens than max_q
    assert c.get_error() & paged.DEV_BAD_CUSEQ
    assert torch.equal(bits(out[0]), bits(good[0])) and torch.all(out[1:] == 7.0)


@pytest.mark.parametrize("dtype,new", [(BF16, 1), (BF16, 40), (F32, 1)])
def test_attend_on_another_stream_and_two_handles_at_once(dtype, new):
    """Two handles with a workspace each over one pool, on two streams."""
    lens = [900, 400]
    c, table, g = make(2, 8, 2, 128, dtype, 32, lens, seed=35)
    d = paged.PagedKVCache(2, 8, 2, 128, dtype, page_size=32, n_pages=c.cfg.n_pages, max_pages=c.cfg.max_pages,
                           k_pages=c.k_pages, v_pages=c.v_pages, block_table=c.block_table, kv_len=c.kv_len)
    q = randn(g, 2, new, 8, 128, dtype=dtype).cuda()
    want = c.attend(q)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(20):
        outs.append((torch.empty_like(q), torch.empty_like(q)))
    torch.cuda.synchronize()
    for x, y in outs:
        c.attend(q, out=x, stream=s1)
        d.attend(q, out=y, stream=s2)
    torch.cuda.synchronize()
    for x, y in outs:
        assert torch.equal(bits(x), bits(want)) and torch.equal(bits(y), bits(want))


def test_offsets_past_32_bits():
    """A pool of more than 2^31 elements: its last pages are found."""
    page, kv_heads, dim = 128, 8, 128
    n_pages = 2 ** 31 // (page * kv_heads * dim) + 40
    pool = torch.zeros(2, n_pages, page, kv_heads, dim, dtype=BF16, device="cuda")
    c = paged.PagedKVCache(1, 8, 8, dim, BF16, page_size=page, n_pages=n_pages, max_pages=4, k_pages=pool[0], v_pages=pool[1],
                           bounds=True)
    g = torch.Generator().manual_seed(36)
    c.block_table.copy_(ints([[n_pages - 1, 0, n_pages - 3, n_pages - 2]]))
    table = c.block_table.cpu().numpy()
    c.kv_len.fill_(400)
    k, v = randn(g, 400, kv_heads, dim, dtype=BF16).cuda(), randn(g, 400, kv_heads, dim, dtype=BF16).cuda()
    c.append(k, v)
    for n in (1, 30):
        q = randn(g, n, 8, dim, dtype=BF16).cuda()
        out = c.attend(q)
        want = ref.attend_rows(to64(q), to64(k), to64(v), np.ones((n, 400), bool), dim ** -0.5, BF16)
        ref.check(out, None, want, "far pages")
    q = randn(g, 1, 8, dim, dtype=BF16).cuda()
    out, sel = c.attend_sparse(q, 3)
    assert c.get_error() == 0 and torch.all(sel[..., 0] == 0) and torch.all(sel[..., 2] == 3)
    del pool, c


# ------------------------------------------------------------------------------------------------ shared prefix
SHARED = [
    # heads, kv_heads, dim, page, prefix, lens, new, causal
    (8, 2, 128, 16, 512, [513, 600, 530], [1, 1, 1], False),
    (32, 8, 128, 64, 1024, [1030, 1500, 1025, 1100], [1, 1, 1, 1], True),
    (40, 8, 64, 32, 320, [325, 400, 321, 330], [5, 1, 1, 4], True),
    (4, 4, 64, 128, 128, [130, 200], [2, 70], True),            # the second row's tokens are a chunk
    (8, 1, 128, 16, 64, [64, 40, 0, 70, 64], [1, 1, 1, 1, 2], True),   # rows within the prefix, one empty
    (6, 2, 128, 16, 0, [20, 9], [1, 1], False),                 # no prefix
    (12, 12, 128, 32, 2048, [2049 + i for i in range(40)], [1] * 40, False),
    (34, 2, 64, 16, 160, [161, 170], [1, 3], True),             # groups of 17 heads
    # more than rows read one by one: the prefix in a pass of its own
    (8, 2, 128, 16, 4096, [4097 + 9 * i for i in range(25)] + [4096], [1, 2] * 13, True),
    (34, 2, 64, 16, 6400, [6404, 6415], [1, 3], True),
    (40, 8, 64, 32, 3200, [3205, 100, 0, 3201, 3300, 3217, 3199, 3230, 3264, 3250, 3260], [5, 1, 1, 4, 2, 5, 1, 1, 0, 1, 3], True),
    (12, 12, 128, 128, 1408, [1409 + 31 * i for i in range(12)], [1] * 12, False),
]


@pytest.mark.parametrize("simt", [0, SIMT])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("case", range(len(SHARED)))
def test_attend_shared(case, dtype, simt):
    heads, kv_heads, dim, page, prefix, lens, new, causal = SHARED[case]
    cu = wl.seqlens_to_cu(new)
    total = cu[-1] + 2
    c, table, g = make(len(lens), heads, kv_heads, dim, dtype, page, lens, seed=50 + case, shared=prefix // page, max_tokens=total)
    if prefix:                                                   # rows shorter than the prefix leave its pages unfilled
        full = torch.randn(prefix // page, page, kv_heads, dim, generator=g).to(dtype).cuda()
        idx = torch.tensor(c.perm[:prefix // page], device="cuda")
        c.k_pages[idx] = full
        c.v_pages[idx] = full.flip(0)
    pages = ints(c.perm[:prefix // page] or [0])
    # the columns of the prefix are not read from the rows' own tables
    ptable = table.copy()
    c.block_table[:, :prefix // page] = -1
    q = randn(g, total, heads, dim, dtype=dtype).cuda()
    out, lse = torch.full_like(q, 7.0), torch.full((total, heads), 7.0, device="cuda")
    flags = simt | (paged.CAUSAL if causal else 0)
    c.attend_shared(q, pages, ints([prefix]), cu_q=ints(cu), max_q=max(new), out=out, lse=lse, flags=flags)
    assert c.get_error() == 0
    check(out, lse, expect(c, ptable, q, lens, cu, causal), f"case {case}", cu[-1])
    assert torch.all(out[cu[-1]:] == 7.0) and torch.all(lse[cu[-1]:] == 7.0)
    again = c.attend_shared(q, pages, ints([prefix]), cu_q=ints(cu), max_q=max(new), flags=flags)
    assert torch.equal(bits(again[:cu[-1]]), bits(out[:cu[-1]]))


def test_attend_shared_refuses_bad_prefixes_on_the_device():
    c, table, g = make(2, 4, 2, 64, BF16, 16, [50, 60], seed=70, shared=2)
    q = randn(g, 2, 4, 64, dtype=BF16).cuda()
    for bad in (-16, 8, 48):
        out = torch.full_like(q, 7.0)
        c.attend_shared(q, ints(c.perm[:2]), ints([bad]), out=out)
        assert c.get_error() & paged.DEV_BAD_KVLEN
        assert torch.all(out == 7.0)
    out = c.attend_shared(q, ints(c.perm[:2]), ints([32]))
    assert c.get_error() == 0
    check(out, None, expect(c, table, q, [50, 60], None, False), "after")


# ------------------------------------------------------------------------------------------------ selected pages
SPARSE = [
    # heads, kv_heads, dim, page, lens, n_select, first, recent
    (32, 8, 128, 16, [2000], 16, 1, 1),
    (8, 2, 64, 64, [1000, 64, 0, 3000, 500], 6, 1, 1),
    (6, 2, 128, 32, [999, 1500], 9, 0, 0),
    (16, 1, 64, 16, [700, 350], 12, 3, 2),
    (4, 4, 128, 128, [1500, 1300], 4, 2, 2),
    (34, 2, 128, 16, [400], 7, 1, 1),
    (12, 4, 64, 16, [9000], 40, 1, 1),
]


@pytest.mark.parametrize("simt", [0, SIMT])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("case", range(len(SPARSE)))
def test_attend_sparse(case, dtype, simt):
    heads, kv_heads, dim, page, lens, n_select, first, recent = SPARSE[case]
    B = len(lens)
    c, table, g = make(B, heads, kv_heads, dim, dtype, page, lens, seed=80 + case, bounds=True)
    kp = to64(c.k_pages)
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            x = ref.page_bounds(kp, table[b, j], min(page, n - j * page)).swapaxes(0, 1)
            c.bounds[table[b, j]].copy_(torch.from_numpy(x).to(dtype))
    q = randn(g, B, heads, dim, dtype=dtype).cuda()
    for call in range(2):                                        # (counters are left as found)
        out, lse, sel = c.attend_sparse(q, n_select, first=first, recent=recent, lse=True, flags=simt)
        assert c.get_error() == 0
        bd = to64(c.bounds)
        v = to64(c.v_pages)
        for b, n in enumerate(lens):
            np_row = -(-n // page)
            want = ref.select(to64(q[b]), bd, table[b], np_row, n_select, first, recent)
            for e in range(kv_heads):
                assert sel[b, e].tolist() == want[e] + [-1] * (n_select - len(want[e])), (b, e)
            kk, vv = ref.gather(kp, table[b], 0, n), ref.gather(v, table[b], 0, n)
            G = heads // kv_heads
            for e in range(kv_heads):
                see = np.isin(np.arange(n) // page, want[e])[None]
                r = ref.attend_rows(to64(q[b:b + 1, e * G:(e + 1) * G]), kk[:, e:e + 1], vv[:, e:e + 1], see, dim ** -0.5, dtype)
                ref.check(out[b:b + 1, e * G:(e + 1) * G], lse[b:b + 1, e * G:(e + 1) * G], r, f"row {b} head {e}")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sparse_ties_go_to_the_lowest_column(dtype):
    """Equal bounds everywhere: more candidates at the border than places; and some pages a hair above."""
    B, page, n_cols = 2, 16, 1500
    lens = [n_cols * page, 600 * page - 5]
    c, table, g = make(B, 4, 2, 64, dtype, page, lens, seed=95, bounds=True)
    one = torch.randn(2, 2, 64, generator=g).to(dtype)
    c.bounds.copy_(torch.maximum(one[:, :1], one[:, 1:]).expand(2, 2, 64).cuda())
    q = randn(g, B, 4, 64, dtype=dtype).cuda()
    _, sel = c.attend_sparse(q, 10, first=1, recent=2)
    for b, cols in enumerate((n_cols, 600)):
        for e in range(2):
            assert sel[b, e].tolist() == list(range(8)) + [cols - 2, cols - 1]
    step = {BF16: 2.0 ** -8, F32: 2.0 ** -23}[dtype]
    for j in (7, 100, 599 - 90):                                 # the least step up in one channel of both bounds
        pg = int(table[0, j])
        x = c.bounds[pg, :, :, 5]
        c.bounds[pg, :, :, 5] = (x.float() * (1 + step) + 0.0).to(dtype)
    bd = to64(c.bounds)
    _, sel = c.attend_sparse(q, 10, first=1, recent=2)
    for b, cols in enumerate((n_cols, 600)):
        want = ref.select(to64(q[b]), bd, table[b], cols, 10, 1, 2)
        for e in range(2):
            assert sel[b, e].tolist() == want[e]
    assert c.get_error() == 0


# ------------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_serving_run_prompt_shared_then_sparse(dtype):
    """A common prompt stored once; three rows continue it with prompts of their own (a chunk), then single tokens by
    shared and by sparse attention, all against one chronological history per row."""
    heads, kv_heads, dim, page, P = 8, 2, 64, 16, 96
    own_prompt = [40, 7, 1]
    B, steps = 3, 6
    rope = wl.rope_table(256, dim)
    n_pages = 64
    c = paged.PagedKVCache(B, heads, kv_heads, dim, dtype, page_size=page, n_pages=n_pages, max_pages=16, bounds=True, max_tokens=64)
    for t in (c.k_pages, c.v_pages, c.bounds):
        t.fill_(float("nan"))
    g = torch.Generator().manual_seed(99)
    perm = torch.randperm(n_pages, generator=g).tolist()
    shared = perm[:P // page]
    table = np.full((B, 16), -1)
    for b in range(B):
        table[b, :P // page] = shared
        table[b, P // page:14] = perm[10 + b * 8:10 + b * 8 + 14 - P // page]
    c.block_table.copy_(torch.from_numpy(table).int())
    hist_k, hist_v = [[] for _ in range(B)], [[] for _ in range(B)]
    d_rope = rope.cuda()

    def record(b, k, v, pos):
        kr = orc.rope_store(to64(k), pos, rope.numpy(), FMT[dtype])
        hist_k[b].extend(kr)
        hist_v[b].extend(to64(v))

    def reference(q, b, n, n_q, cols=None, e=None):
        kk, vv = np.stack(hist_k[b]), np.stack(hist_v[b])
        return ref.attend_rows(to64(q), kk, vv, ref.visible_mask(n, 0, n_q, n, True), dim ** -0.5, dtype)

    # the common prompt goes in through row 0 alone
    c.kv_len.copy_(ints([P, 0, 0]))
    k, v = randn(g, P, kv_heads, dim, dtype=dtype), randn(g, P, kv_heads, dim, dtype=dtype)
    c.append(k.cuda(), v.cuda(), cu_new=ints([0, P, P, P]), rope=d_rope)
    for b in range(B):
        record(b, k, v, list(range(P)))
    # each row's own prompt, packed, one call
    cu = wl.seqlens_to_cu(own_prompt)
    lens = [P + n for n in own_prompt]
    c.kv_len.copy_(ints(lens))
    k, v, q = (randn(g, cu[-1], h, dim, dtype=dtype) for h in (kv_heads, kv_heads, heads))
    qr = c.append(k.cuda(), v.cuda(), cu_new=ints(cu), rope=d_rope, q=q.cuda())
    for b in range(B):
        record(b, k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]], list(range(P, lens[b])))
    plain, lse_p = c.attend(qr, cu_q=ints(cu), max_q=40, lse=True, flags=paged.CAUSAL)
    both, lse_s = c.attend_shared(qr, ints(shared), ints([P]), cu_q=ints(cu), max_q=40, lse=True, flags=paged.CAUSAL)
    for b in range(B):
        want = reference(qr[cu[b]:cu[b + 1]], b, lens[b], own_prompt[b])
        for o, L in ((plain, lse_p), (both, lse_s)):
            ref.check(o[cu[b]:cu[b + 1]], L[cu[b]:cu[b + 1]], want, f"prompt of row {b}")
    for step in range(steps):
        lens = [n + 1 for n in lens]
        c.kv_len.add_(1)
        k, v, q = (randn(g, B, 1, h, dim, dtype=dtype) for h in (kv_heads, kv_heads, heads))
        qr = c.append(k.cuda(), v.cuda(), rope=d_rope, q=q.cuda())
        for b in range(B):
            record(b, k[b], v[b], [lens[b] - 1])
        out, lse = c.attend_shared(qr, ints(shared), ints([P]), lse=True)
        so, sl, sel = c.attend_sparse(qr, 4, lse=True)
        for b in range(B):
            want = reference(qr[b], b, lens[b], 1)
            ref.check(out[b], lse[b], want, f"step {step} row {b}")
            kk, vv = np.stack(hist_k[b]), np.stack(hist_v[b])
            for e in range(kv_heads):
                cols = [j for j in sel[b, e].tolist() if j >= 0]
                assert len(cols) == 4 and cols[0] == 0 and cols[-1] == (lens[b] - 1) // page
                see = np.isin(np.arange(lens[b]) // page, cols)[None]
                G = heads // kv_heads
                r = ref.attend_rows(to64(qr[b][:, e * G:(e + 1) * G]), kk[:, e:e + 1], vv[:, e:e + 1], see, dim ** -0.5, dtype)
                ref.check(so[b][:, e * G:(e + 1) * G], sl[b][:, e * G:(e + 1) * G], r, f"sparse step {step} row {b}")
    assert c.get_error() == 0
