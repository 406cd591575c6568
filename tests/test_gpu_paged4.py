"""GPU tests of the 4-bit paged cache: what append stores and read returns, bit for bit; attention against plain 64-bit forms."""
import numpy as np
import pytest
import torch

from diffusion_serving_gb300 import workloads as wl
from tests import paged4_ref as ref4
from tests import paged_ref as ref
from tests.helpers import to64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from diffusion_serving_gb300 import paged, paged4
    from tests.test_gpu_paged import bits, ints, randn, rows_of
    from tests.test_gpu_paged_axes import layouts, turned

BF16, F16 = torch.bfloat16, torch.float16


def make(batch, heads, kv_heads, dim, dtype, page, lens, *, seed=1, extra=2, fill=True, spread=None, scale=0.0, n_pages=None):
    """A 4-bit cache whose rows hold `lens` tokens in pages handed out in random order.  Bytes that no token stands in
    are 0xff: codes of 15 under scales of NaN.  Returns (cache, table, generator, k, v): k[b], v[b] the held values."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    n_pages = n_pages or sum(need) + extra
    c = paged4.PagedKVCache4(batch, heads, kv_heads, dim, dtype, page_size=page, n_pages=n_pages, max_pages=max(max(need), 1) + 1,
                             softmax_scale=scale)
    c.pages.fill_(255)
    perm = torch.randperm(n_pages, generator=g)[:sum(need)].tolist()
    table = np.full((batch, c.cfg.max_pages), -7, dtype=np.int64)
    for b, p in enumerate(need):
        table[b, :p] = [perm.pop() for _ in range(p)]
    c.block_table.copy_(torch.from_numpy(table).int())
    c.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
    k, v = ([randn(g, n, kv_heads, dim, dtype=dtype) * (spread or 1) for n in lens] for _ in range(2))
    if fill and sum(lens):
        c.append(torch.cat(k).cuda(), torch.cat(v).cuda(), cu_new=ints(wl.seqlens_to_cu(lens)))
        assert c.get_error() == 0
        k, v = [ref4.held(to64(x)) for x in k], [ref4.held(to64(x)) for x in v]
    return c, table, g, k, v


def expect(c, k, v, q, lens, cu, causal):
    """(out, lse, bounds) of every token by the plain form.  Weights are rounded to fp16, 2^8 too large: those below its
    normal range are off by half its least step, 2^-25 2^-8 of the largest (paged_ref's bound has it for a store of fp16)."""
    qn = to64(q).reshape(-1, c.heads, c.head_dim)
    scale = c.cfg.softmax_scale or c.head_dim ** -0.5
    out = [np.zeros(qn.shape), np.full(qn.shape[:2], -np.inf), np.zeros(qn.shape), np.zeros(qn.shape[:2])]
    for b, n in enumerate(lens):
        t0, m = rows_of(cu, b, len(qn), c.batch)
        if m == 0:
            continue
        got = ref.attend_rows(qn[t0:t0 + m], k[b][:n], v[b][:n], ref.visible_mask(n, 0, m, n, causal), scale, c.dtype)
        if n:
            got[2][:] += 2.0 ** -33 * np.repeat(np.abs(v[b][:n]).sum(0), c.heads // c.kv_heads, 0)
        for dst, x in zip(out, got):
            dst[t0:t0 + m] = x
    return out


def check(got, lse, want, what, n=None):
    n = want[0].shape[0] if n is None else n
    got = got.reshape(-1, *want[0].shape[1:])[:n]
    lse = None if lse is None else lse.reshape(-1, want[1].shape[1])[:n]
    ref.check(got, lse, [x[:n] for x in want], what)


# ------------------------------------------------------------------------------------------------ append, read
def store(before, table, lens, new, cu, kv, page, dim):
    """What a pool's unpacked parts are after an append: `kv` (k, v) packed rows of values in 64 bits."""
    parts = [x.copy() for x in ref4.unpack(before, page, dim)]
    for (code, bit), x in zip(((0, 1), (2, 3)), kv):
        cc, bb = ref4.codes(x)
        for b, (n, m) in enumerate(zip(lens, new)):
            for i in range(m):
                p = n - m + i
                parts[code][table[b, p // page], p % page] = cc[cu[b] + i]
                parts[bit][table[b, p // page], p % page] = bb[cu[b] + i]
    return parts


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dim,kv_heads,page,layout", [(128, 8, 16, None), (64, 3, 64, "turns"), (128, 5, 32, "sections"), (64, 9, 16, None),
                                                      (128, 1, 128, "four"), (64, 1, 32, None), (64, 2, 128, "odd sections")])
def test_append_and_read_bit_exact(dtype, half, dim, kv_heads, page, layout):
    heads = 2 * kv_heads
    lens, new = [37, 1, 300, 64, 129], [20, 1, 0, 64, 3]
    c, table, g, _, _ = make(5, heads, kv_heads, dim, dtype, page, lens, fill=False, seed=3)
    c.pages.copy_(torch.randint(0, 256, c.pages.shape, generator=g, dtype=torch.uint8))
    before = c.pages.cpu().numpy()
    cu = wl.seqlens_to_cu(new)
    n, total = cu[-1], cu[-1] + 4                       # rows behind the last sequence
    angles = torch.randn(320, dim // 2, generator=g, dtype=torch.float64) * 3
    rope = torch.stack([angles.cos(), angles.sin()], -1).float()
    joint = randn(g, total, heads + 2 * kv_heads, dim, dtype=dtype).cuda()
    joint[:, :, ::17] *= 6
    q, k, v = joint[:, :heads], joint[:, heads:heads + kv_heads], joint[:, heads + kv_heads:]
    kw = {}
    if layout is None:
        pos = np.concatenate([np.arange(x - m, x) for x, m in zip(lens, new)])[:, None]
        pair_axis = [0] * (dim // 2)
    else:
        pair_axis = layouts(dim)[layout]
        kw["axes"] = paged.rope_axes(pair_axis)
        kw["positions"] = torch.randint(0, 320, (total, kw["axes"].n_axes), generator=g, dtype=torch.int32).cuda()
        pos = kw["positions"].cpu().numpy()[:n]
    q_out = torch.full((total, heads, dim), 7.0, dtype=dtype, device="cuda")
    c.append(k, v, cu_new=ints(cu), rope=rope.cuda(), half=half, q=q, q_out=q_out, **kw)
    assert c.get_error() == 0
    kt = turned(k[:n], pos, pair_axis, rope.numpy(), half, dtype)
    assert torch.equal(bits(q_out[:n].cpu()), bits(turned(q[:n], pos, pair_axis, rope.numpy(), half, dtype)))
    assert torch.all(q_out[n:] == 7.0)
    want = store(before, table, lens, new, cu, (to64(kt), to64(v[:n])), page, dim)
    got = ref4.unpack(c.pages.cpu().numpy(), page, dim)
    for x, y in zip(got, want):
        assert np.array_equal(x, y)
    k_out, v_out = (torch.full((total, kv_heads, dim), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    c.read(total, cu=ints(cu), k_out=k_out, v_out=v_out)
    assert c.get_error() == 0
    assert np.array_equal(to64(k_out[:n]), ref4.held(to64(kt))) and np.array_equal(to64(v_out[:n]), ref4.held(to64(v[:n])))
    assert torch.all(k_out[n:] == 7.0) and torch.all(v_out[n:] == 7.0)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("dim", [64, 128])
def test_every_magnitude_and_what_is_not_a_number(dtype, dim):
    """Groups of every magnitude of the type down to its least, ties between codes and between scales, zeros, infinities, NaN."""
    g = torch.Generator().manual_seed(4)
    tops = torch.arange(0, 32768, 13, dtype=torch.int32).to(torch.int16).view(dtype)
    tops = tops[torch.isfinite(tops)]
    n = len(tops)
    x = (torch.rand(n, 32, generator=g) * 2 - 1)
    x = (x * tops.float()[:, None]).to(dtype)
    x[torch.arange(n), torch.randint(0, 32, (n,), generator=g)] = tops
    ties = torch.arange(-15, 17).float()[None] / 2 * torch.from_numpy(ref4.E4M3[8:119]).float()[:, None]   # (c - 8) s and halfway
    ties = torch.cat([ties, torch.where(ties.abs() > 7 * ties[:, -3:-2] / 7, 0, ties)]).to(dtype)
    odd = torch.zeros(8, 32, dtype=dtype)
    odd[1, 3], odd[2, 5], odd[3, 31] = float("nan"), float("inf"), -float("inf")
    odd[4, 0], odd[4, 1] = float("nan"), float("inf")
    odd[5], odd[6], odd[7, 7] = float("inf"), 3136.0, -0.0
    odd[2, 6], odd[3, 6] = 448 * 1.5, 447.0
    x = torch.cat([x, ties, odd])
    per = dim // 32 * 2
    x = torch.cat([x, torch.zeros(-len(x) % per, 32, dtype=dtype)]).reshape(-1, 2, dim)
    v = x.flip(0).contiguous()
    n = len(x)
    c, table, _, _, _ = make(1, 2, 2, dim, dtype, 32, [n], fill=False)
    c.append(x.cuda(), v.cuda())
    k_out, v_out = c.read(n)
    assert c.get_error() == 0
    got = ref4.unpack(c.pages.cpu().numpy()[table[0, :-1]], 32, dim)
    for (code, bit), y, out in (((0, 1), x, k_out), ((2, 3), v, v_out)):
        cc, bb = ref4.codes(to64(y))
        assert np.array_equal(got[bit].reshape(-1, 2, dim // 32)[:n], bb)
        nan = np.repeat(bb == 127, 32, -1)
        assert np.array_equal(got[code].reshape(-1, 2, dim)[:n][~nan], cc[~nan])
        want = ref4.value(cc, bb)
        assert np.array_equal(np.isnan(to64(out)), nan) and np.array_equal(to64(out)[~nan], want[~nan])


def test_token_by_token_is_one_append():
    lens = [45, 45, 45]
    c, table, g, _, _ = make(3, 4, 2, 64, BF16, 16, lens, fill=False, seed=5)
    d, _, _, _, _ = make(3, 4, 2, 64, BF16, 16, lens, fill=False, seed=5)
    k, v = randn(g, 3, 45, 2, 64, dtype=BF16).cuda(), randn(g, 3, 45, 2, 64, dtype=BF16).cuda()
    c.append(k, v)
    for lo, hi in [(0, 30)] + [(i, i + 1) for i in range(30, 45)]:
        d.kv_len.fill_(hi)
        d.append(k[:, lo:hi].contiguous(), v[:, lo:hi].contiguous())
    assert c.get_error() == 0 and d.get_error() == 0
    assert torch.equal(c.pages, d.pages)
    ko, vo = c.read(3 * 45, k_out=torch.empty_like(k), v_out=torch.empty_like(v))
    assert np.array_equal(to64(ko), ref4.held(to64(k))) and np.array_equal(to64(vo), ref4.held(to64(v)))


def test_append_and_read_report_bad_rows_and_leave_them():
    lens = [20, 20, 20, 20]
    c, table, g, _, _ = make(4, 4, 2, 64, BF16, 16, lens, fill=False, seed=6)
    k = randn(g, 8, 2, 64, dtype=BF16).cuda()
    before = c.pages.clone()
    rope = wl.rope_table(19, 64).cuda()                 # position 19 is outside
    c.kv_len.copy_(ints([20, 1, 500, 20]))              # row 1 shorter than its tokens, row 2 past the table's columns
    c.block_table[3, 1] = 10 ** 6
    c.append(k, k, cu_new=ints([0, 2, 4, 6, 8]), rope=rope)
    assert c.get_error() == paged.DEV_BAD_KVLEN | paged.DEV_BAD_PAGE | paged.DEV_BAD_POS
    a, b = ref4.unpack(before.cpu().numpy(), 16, 64), ref4.unpack(c.pages.cpu().numpy(), 16, 64)
    for x, y in zip(a, b):
        same = np.array([[np.array_equal(x[i, s], y[i, s]) for s in range(16)] for i in range(len(x))])
        assert not same[table[0, 1], 2] and same.sum() == same.size - 1        # row 0, position 18 alone
    out = torch.full((8, 2, 64), 7.0, dtype=BF16, device="cuda")
    c.read(8, cu=ints([0, 2, 4, 6, 8]), k_out=out, v_out=out.clone())
    assert c.get_error() == paged.DEV_BAD_KVLEN | paged.DEV_BAD_PAGE
    assert torch.all(out[2:] == 7.0) and not torch.any(out[:2] == 7.0)
    c.kv_len.copy_(ints(lens))
    c.read(8, cu=ints([0, 2, 1, 6, 9]), k_out=out.fill_(7.0), v_out=out.clone())
    assert c.get_error() & paged.DEV_BAD_CUSEQ and torch.all(out[6:] == 7.0)
    pos = ints([[0], [19], [18], [-1], [0], [0], [0], [0]])
    c.block_table.copy_(torch.from_numpy(table).int())
    before = c.pages.clone()
    c.append(k, k, rope=rope, positions=pos)
    assert c.get_error() == paged.DEV_BAD_POS
    a, b = ref4.unpack(before.cpu().numpy(), 16, 64), ref4.unpack(c.pages.cpu().numpy(), 16, 64)
    for r in range(4):
        for i in range(2):
            p = 18 + i
            same = all(np.array_equal(x[table[r, p // 16], p % 16], y[table[r, p // 16], p % 16]) for x, y in zip(a, b))
            assert same == ((r, i) in ((0, 1), (1, 1))), (r, i)


# ------------------------------------------------------------------------------------------------ attend
SHAPES = [(32, 8, 128), (8, 8, 64), (12, 4, 64), (40, 8, 128), (16, 1, 128), (6, 3, 128), (64, 2, 64), (71, 1, 128)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,kv_heads,dim", SHAPES)
def test_single_tokens(dtype, page, heads, kv_heads, dim):
    lens = [1, 300, 16, 0, 131, 1100, 128, 15]
    c, table, g, k, v = make(len(lens), heads, kv_heads, dim, dtype, page, lens, seed=page + heads)
    q = randn(g, len(lens), heads, dim, dtype=dtype)
    out, lse = c.attend(q.cuda(), lse=True)
    assert c.get_error() == 0
    check(out, lse, expect(c, k, v, q, lens, None, False), "single tokens")


@pytest.mark.parametrize("dtype,page", [(BF16, 16), (F16, 64), (BF16, 128), (F16, 32)])
@pytest.mark.parametrize("heads,kv_heads,dim", SHAPES[:6])
@pytest.mark.parametrize("causal", [False, True])
def test_tokens_and_chunks(dtype, page, heads, kv_heads, dim, causal):
    """Rows with no token, with one, more than they have slots, odd lengths; rows behind the last are left as they were."""
    lens, new = [700, 5, 0, 260, 129, 1], [33, 5, 3, 0, 129, 2]
    c, table, g, k, v = make(len(lens), heads, kv_heads, dim, dtype, page, lens, seed=page + heads)
    cu = wl.seqlens_to_cu(new)
    q = randn(g, cu[-1] + 3, heads, dim, dtype=dtype).cuda()
    q[cu[-1]:] = float("nan")
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    c.attend(q, cu_q=ints(cu), max_q=max(new), out=out, lse=lse, flags=paged.CAUSAL if causal else 0)
    assert c.get_error() == 0
    check(out, lse, expect(c, k, v, q[:cu[-1]], lens, cu, causal), "chunks", cu[-1])
    assert torch.all(out[cu[-1]:] == 7.0) and torch.all(lse[cu[-1]:] == 7.0)


@pytest.mark.parametrize("dim,heads,kv_heads,n", [(128, 8, 2, 20011), (64, 4, 4, 9000), (128, 1, 1, 33333)])
def test_long_rows_cut_among_blocks(dim, heads, kv_heads, n):
    lens = [n, 17, n // 3]
    c, table, g, k, v = make(3, heads, kv_heads, dim, F16, 64, lens, seed=7, spread=2)
    q = randn(g, 3, heads, dim, dtype=F16)
    out, lse = c.attend(q.cuda(), lse=True)
    want = expect(c, k, v, q, lens, None, False)
    check(out, lse, want, "long rows")
    for _ in range(3):
        again, lse2 = c.attend(q.cuda(), lse=True)
        assert torch.equal(bits(again), bits(out)) and torch.equal(bits(lse2), bits(lse))
    assert c.get_error() == 0


@pytest.mark.parametrize("heads,kv_heads,dim,page,new,causal", [(32, 8, 128, 64, 300, True), (12, 12, 64, 16, 260, False),
                                                               (16, 2, 128, 128, 129, True), (5, 1, 64, 32, 400, True)])
def test_long_chunks(heads, kv_heads, dim, page, new, causal):
    lens = [2500, new + 1]
    c, table, g, k, v = make(2, heads, kv_heads, dim, BF16, page, lens, seed=8)
    q = randn(g, 2 * new, heads, dim, dtype=BF16)
    out, lse = c.attend(q.cuda(), lse=True, flags=paged.CAUSAL if causal else 0)
    assert c.get_error() == 0
    check(out, lse, expect(c, k, v, q, lens, None, causal), "long chunks")


def test_growing_scores_move_the_reference():
    """Scores that grow along the row by far more than the headroom of the weights, and a few that stand out."""
    n, dim = 900, 128
    for new in (1, 40):
        c, table, g, _, _ = make(1, 2, 1, dim, F16, 16, [n], seed=9, fill=False)
        q = randn(g, new, 2, dim, dtype=F16)
        k = randn(g, n, 1, dim, dtype=F16) * 0.1 + q[0, :1] * torch.linspace(-4, 4, n)[:, None, None].half()
        v = randn(g, n, 1, dim, dtype=F16)
        c.append(k.cuda(), v.cuda())
        out, lse = c.attend(q.cuda(), lse=True)
        assert c.get_error() == 0
        check(out, lse, expect(c, [ref4.held(to64(k))], [ref4.held(to64(v))], q, [n], None, False), "growing scores")


def test_a_nan_reaches_what_sees_it_and_nothing_else():
    lens = [200, 200]
    for new, flags in ((1, 0), (40, paged.CAUSAL)):
        c, table, g, _, _ = make(2, 4, 2, 128, BF16, 16, lens, seed=10, fill=False)
        k, v = randn(g, 400, 2, 128, dtype=BF16), randn(g, 400, 2, 128, dtype=BF16)
        k[37, 0, 5] = float("nan")                      # row 0, kv head 0
        c.append(k.cuda(), v.cuda())
        q = randn(g, 2 * new, 4, 128, dtype=BF16)
        out, lse = c.attend(q.cuda(), lse=True, flags=flags)
        assert c.get_error() == 0
        bad = torch.isnan(out).any(-1).reshape(2, new, 4)
        assert bad[0, :, :2].all() and not bad[0, :, 2:].any() and not bad[1].any()
        assert torch.isnan(out.reshape(2, new, 4, 128)[0, :, :2]).all() and torch.isnan(lse.reshape(2, new, 4)[0, :, :2]).all()


@pytest.mark.parametrize("new", [1, 50])
def test_bad_pages_and_lengths(new):
    lens = [300, 300, 300, 100]
    c, table, g, k, v = make(4, 4, 2, 128, BF16, 64, lens, seed=11)
    q = randn(g, 4 * new, 4, 128, dtype=BF16)
    c.block_table[0, 1] = c.cfg.n_pages                 # slots 64 .. 127 left out
    c.block_table[3, :2] = -1                           # all of row 3's
    c.kv_len.copy_(ints([300, -1, c.cfg.max_pages * 64 + 1, 100]))
    out = torch.full((4 * new, 4, 128), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((4 * new, 4), 7.0, device="cuda")
    c.attend(q.cuda(), out=out, lse=lse)
    assert c.get_error() == paged.DEV_BAD_PAGE | paged.DEV_BAD_KVLEN
    assert torch.all(out[new:3 * new] == 7.0) and torch.all(lse[new:3 * new] == 7.0)
    assert torch.all(out[3 * new:] == 0) and torch.all(torch.isneginf(lse[3 * new:]))
    keep = np.r_[0:64, 128:300]
    want = expect(c, [k[0][keep]], [v[0][keep]], q[:new], [len(keep)], [0, new], False)
    check(out[:new], lse[:new], want, "a page left out")
    c.kv_len.copy_(ints(lens))
    c.attend(q.cuda(), cu_q=ints([0, new, 2 * new, new, 4 * new + 1]), max_q=new, out=out.fill_(7.0))
    assert c.get_error() & paged.DEV_BAD_CUSEQ
    c.attend(q.cuda(), cu_q=ints([0, 4 * new, 4 * new, 4 * new, 4 * new]), max_q=new, out=out.fill_(7.0))
    assert c.get_error() == paged.DEV_BAD_CUSEQ and torch.all(out == 7.0)


def test_records_beyond_32_bits_of_the_pool():
    """Pages at the end of a pool of more than 4 GB: written, read back and attended."""
    page, kv_heads, dim = 64, 40, 128
    n_pages = 2 ** 32 // (kv_heads * page * (dim + dim // 16)) + 40
    c = paged4.PagedKVCache4(2, kv_heads, kv_heads, dim, F16, page_size=page, n_pages=n_pages, max_pages=8)
    assert c.pages.numel() > 2 ** 32
    c.block_table.copy_(torch.arange(n_pages - 16, n_pages, dtype=torch.int32).flip(0).reshape(2, 8))
    lens, g = [500, 77], torch.Generator().manual_seed(12)
    c.kv_len.copy_(ints(lens))
    k, v, q = (randn(g, n, kv_heads, dim, dtype=F16) for n in (577, 577, 2))
    cu = ints([0, 500, 577])
    c.append(k.cuda(), v.cuda(), cu_new=cu)
    ko, vo = c.read(577, cu=cu)
    out, lse = c.attend(q.cuda(), lse=True)
    assert c.get_error() == 0
    kh, vh = ref4.held(to64(k)), ref4.held(to64(v))
    assert np.array_equal(to64(ko), kh) and np.array_equal(to64(vo), vh)
    check(out, lse, expect(c, [kh[:500], kh[500:]], [vh[:500], vh[500:]], q, lens, None, False), "far records")
