"""GPU tests of rotary positions with several axes in the paged append: stores and queries bit for bit."""
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
    from tests.test_gpu_paged import FMT, bits, ints, make, randn

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
POSITIONS = 300


def turned(x, pos, pair_axis, table, half, dtype):
    """x [n, heads, D] turned at pos [n, axes]: a table of its own for the tokens, pair by pair, and the one-axis rotation."""
    dim = x.shape[-1]
    own = np.stack([table[pos[:, a], j] for j, a in enumerate(pair_axis)], 1)            # [n, D/2, 2]
    x = to64(x)
    if half:
        x = np.stack([x[..., :dim // 2], x[..., dim // 2:]], -1).reshape(x.shape)
    y = orc.rope_store(x, np.arange(len(x)), own, FMT[dtype])
    if half:
        y = np.concatenate([y[..., 0::2], y[..., 1::2]], -1)
    return torch.from_numpy(y).to(dtype)


def layouts(dim):
    n = dim // 2
    return {"one": [0] * n, "sections": [0] * (n // 4) + [1] * (3 * n // 8) + [2] * (n - n // 4 - 3 * n // 8),
            "turns": [j % 3 for j in range(n)], "odd sections": [0] * 5 + [1] * 7 + [3] * (n - 12),
            "four": [(j * 7 + j // 5) % 4 for j in range(n)]}


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dim,kv_heads,page,layout", [(128, 8, 16, "sections"), (64, 3, 64, "turns"), (128, 2, 32, "four"),
                                                      (64, 1, 128, "odd sections"), (128, 20, 16, "one")])
def test_packed_rows_bit_exact(dtype, half, dim, kv_heads, page, layout):
    heads = 2 * kv_heads
    lens, new = [37, 1, 300, 64, 129], [20, 1, 0, 64, 3]
    c, table, g = make(5, heads, kv_heads, dim, dtype, page, lens, bounds=True, seed=3)
    pair_axis = layouts(dim)[layout]
    axes = paged.rope_axes(pair_axis)
    cu = wl.seqlens_to_cu(new)
    total = cu[-1] + 4                                  # rows behind the last sequence: their positions may be anything
    pos = torch.randint(0, POSITIONS, (total, axes.n_axes), generator=g, dtype=torch.int32)
    pos[0], pos[1] = 0, POSITIONS - 1
    pos[cu[-1]:] = -5
    angles = torch.randn(POSITIONS, dim // 2, generator=g, dtype=torch.float64) * 3
    rope = torch.stack([angles.cos(), angles.sin()], -1).float()
    joint = randn(g, total, heads + 2 * kv_heads, dim, dtype=dtype).cuda()
    q, k, v = joint[:, :heads], joint[:, heads:heads + kv_heads], joint[:, heads + kv_heads:]
    want_k, want_v = c.k_pages.cpu().clone(), c.v_pages.cpu().clone()
    old_bounds = to64(c.bounds.fill_(0.0))
    q_out = torch.full((total, heads, dim), 7.0, dtype=dtype, device="cuda")
    c.append(k, v, cu_new=ints(cu), rope=rope.cuda(), half=half, q=q, q_out=q_out, positions=pos.cuda(),
             axes=None if layout == "one" else axes)
    assert c.get_error() == 0
    kt = turned(k[:cu[-1]], pos[:cu[-1]].numpy(), pair_axis, rope.numpy(), half, dtype)
    qt = turned(q[:cu[-1]], pos[:cu[-1]].numpy(), pair_axis, rope.numpy(), half, dtype)
    touched = {}
    for b, (n, m) in enumerate(zip(lens, new)):
        for i in range(m):
            p = n - m + i
            want_k[table[b, p // page], p % page] = kt[cu[b] + i]
            want_v[table[b, p // page], p % page] = v[cu[b] + i].cpu()
            touched.setdefault(int(table[b, p // page]), []).append(p % page)
    assert torch.equal(bits(q_out[:cu[-1]].cpu()), bits(qt)) and torch.all(q_out[cu[-1]:] == 7.0)
    assert torch.equal(bits(c.k_pages.cpu()), bits(want_k))
    assert torch.equal(bits(c.v_pages.cpu()), bits(want_v))
    kp, got = to64(want_k), to64(c.bounds)
    for pg in range(c.cfg.n_pages):
        want = old_bounds[pg]
        if pg in touched:
            x = kp[pg, touched[pg]]
            hi, lo = x.max(0), x.min(0)
            if 0 not in touched[pg]:                    # widened from what was there (0)
                hi, lo = np.maximum(hi, want[:, 0]), np.minimum(lo, want[:, 1])
            want = np.stack([hi, lo], 1)
        assert np.array_equal(got[pg], want), pg


def test_equal_axes_are_one_position():
    """All axes at the slot: the plain append, bit for bit; [batch, n, axes] positions."""
    lens = [45, 45]
    c, table, g = make(2, 4, 2, 64, BF16, 16, lens, seed=5)
    d, _, _ = make(2, 4, 2, 64, BF16, 16, lens, seed=5)
    k, v, q = (randn(g, 2, 9, h, 64, dtype=BF16).cuda() for h in (2, 2, 4))
    rope = wl.rope_table(64, 64).cuda()
    pos = torch.arange(36, 45, dtype=torch.int32)[None, :, None].expand(2, 9, 3).contiguous().cuda()
    a = c.append(k, v, rope=rope, q=q, half=True)
    b = d.append(k, v, rope=rope, q=q, half=True, positions=pos, axes=paged.rope_axes([j % 3 for j in range(32)]))
    assert c.get_error() == 0 and d.get_error() == 0
    assert torch.equal(bits(a), bits(b)) and torch.equal(bits(c.k_pages), bits(d.k_pages)) and torch.equal(bits(c.v_pages), bits(d.v_pages))


@pytest.mark.parametrize("page", [16, 64])
def test_tokens_out_of_the_table_are_left_out(page):
    """They are not written, nor their queries, and count in no bound; a page with none of the others keeps its bounds."""
    lens = [3 * page]
    c, table, g = make(1, 4, 2, 64, F16, page, lens, bounds=True, seed=8)
    n = 3 * page
    k, v, q = (randn(g, n, h, 64, dtype=F16).cuda() for h in (2, 2, 4))
    k[5] = 50.0                                         # would show in the bounds
    pos = torch.randint(0, 40, (n, 2), generator=g, dtype=torch.int32)
    out = [5] + list(range(page, 2 * page)) + [2 * page, 3 * page - 1]
    for i, t in enumerate(out):
        pos[t, i % 2] = (-1, 40, 2 ** 31 - 1, -2 ** 31)[i % 4]
    c.bounds.fill_(99.0)
    before_k, before_v = c.k_pages.clone(), c.v_pages.clone()
    q_out = torch.full((n, 4, 64), 7.0, dtype=F16, device="cuda")
    c.append(k, v, rope=wl.rope_table(40, 64).cuda(), q=q, q_out=q_out, positions=pos.cuda(), axes=paged.rope_axes([0] * 16 + [1] * 16))
    assert c.get_error() == paged.DEV_BAD_POS
    kp = to64(c.k_pages)
    for t in range(n):
        pg, s = int(table[0, t // page]), t % page
        if t in out:
            assert torch.equal(bits(c.k_pages[pg, s]), bits(before_k[pg, s])) and torch.equal(bits(c.v_pages[pg, s]), bits(before_v[pg, s]))
            assert torch.all(q_out[t] == 7.0)
        else:
            assert torch.equal(bits(c.v_pages[pg, s]), bits(v[t])) and not torch.any(q_out[t] == 7.0)
    for col in range(3):
        pg = int(table[0, col])
        good = [t % page for t in range(col * page, (col + 1) * page) if t not in out]
        got = to64(c.bounds[pg])
        if not good:
            assert np.all(got == 99.0)
        else:
            assert np.array_equal(got[:, 0], kp[pg, good].max(0)) and np.array_equal(got[:, 1], kp[pg, good].min(0))


def test_image_tokens_then_text_attend():
    """An image's grid and a text step behind it, appended and attended: as the 64-bit form over what is stored; captured and replayed."""
    dim, page, lens = 128, 16, [70]
    c, table, g = make(1, 8, 2, dim, BF16, page, lens, seed=9)
    axes = paged.rope_axes([0] * 16 + [1] * 24 + [2] * 24)
    grid = torch.tensor([[4, 4 + i // 9, 4 + i % 9] for i in range(63)] + [[13 + i] * 3 for i in range(7)], dtype=torch.int32)
    k, v, q = (randn(g, 70, h, dim, dtype=BF16).cuda() for h in (2, 2, 8))
    rope, pos = wl.rope_table(64, dim).cuda(), grid.cuda()
    q_out, out = torch.empty_like(q), torch.empty_like(q)

    def step():
        c.append(k, v, rope=rope, q=q, q_out=q_out, positions=pos, axes=axes)
        c.attend(q_out, out=out, flags=paged.CAUSAL)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    k.copy_(randn(g, 70, 2, dim, dtype=BF16))
    pos.add_(1)
    out.zero_()
    graph.replay()
    assert c.get_error() == 0
    kt = turned(k, pos.cpu().numpy(), [0] * 16 + [1] * 24 + [2] * 24, wl.rope_table(64, dim).numpy(), False, BF16)
    got = ref.gather(to64(c.k_pages), table[0], 0, 70)
    assert np.array_equal(got, to64(kt))
    want = ref.attend_rows(to64(q_out), got, to64(v), ref.visible_mask(70, 0, 70, 70, True), dim ** -0.5, BF16)
    ref.check(out, None, want, "image and text")
