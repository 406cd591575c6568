"""The paged cache's rotary positions with several axes and its 4-bit store, measured: what each operator is called with, its
plain form, and its work.

 axes     new tokens appended to a 16 or 32 bit store, keys and queries rotated at given positions of several axes
 append4  new tokens quantised into a 4-bit store (keys rotated first, queries beside them), and what it then holds of them
 attend4  softmax attention of one token, a few, or a chunk per row over a 4-bit store

A 4-bit store holds, per 32 neighbouring dims of a token and head, an e4m3 scale s and codes c of 4 bits, which stand for
(c - 8) s.  Its pool is uint8 [pages, kv_heads, page * (dim + dim / 16)], a record per page and head:
 K codes  [page][dim / 2]    a word of 32 bits holds dims 8 w .. 8 w + 7: dim 2 i in bits 4 i .., dim 2 i + 1 in bits 16 + 4 i ..
 V codes  [page][dim / 2]    the same, but the 16-byte piece x of slot p stands at piece x ^ ((p / 4) mod (dim / 32))
 K scales [page][dim / 32]
 V scales [dim / 32][page]

Rows' lengths follow from the case alone (evenly spread between two ends), so that the work does too; values and the
order of the pages in the pool come from the seed.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of 32 requests whose prompts held images: every axis at the text's position (latency)
        dict(name="axes_step", op="axes", dtype="f16", batch=32, heads=32, kv_heads=8, dim=128, page=16, len_lo=234,
             len_hi=4096, new_lo=1, new_hi=1, half=True, axes="sections"),
        # a frame of 30 x 52 tokens for each of two streams, every head with its own keys
        dict(name="axes_frame", op="axes", dtype="bf16", batch=2, heads=40, kv_heads=40, dim=128, page=64, len_lo=1560,
             len_hi=9360, new_lo=1560, new_hi=1560, half=False, axes="sections"),
        # images of different sizes behind what is stored, the axes' pairs in turn, 32-bit store
        dict(name="axes_images", op="axes", dtype="f32", batch=3, heads=12, kv_heads=4, dim=64, page=32, len_lo=777,
             len_hi=4097, new_lo=333, new_hi=777, half=True, axes="turns"),
        # a decode step of 32 requests into 4 bits (latency)
        dict(name="append4_step", op="append4", dtype="bf16", batch=32, heads=32, kv_heads=8, dim=128, page=16, len_lo=234,
             len_hi=4096, new_lo=1, new_hi=1, half=True, axes="none"),
        # prompts of different lengths admitted in one call
        dict(name="append4_prompts", op="append4", dtype="bf16", batch=8, heads=32, kv_heads=8, dim=128, page=64, len_lo=512,
             len_hi=1560, new_lo=512, new_hi=1560, half=True, axes="none"),
        # three frames for each of two streams, small heads
        dict(name="append4_frames", op="append4", dtype="f16", batch=2, heads=12, kv_heads=12, dim=64, page=32, len_lo=4680,
             len_hi=9361, new_lo=4680, new_hi=4680, half=False, axes="sections"),
        # one request's decode step at the middle of a short answer (latency)
        dict(name="attend4_one", op="attend4", dtype="f16", batch=1, heads=32, kv_heads=8, dim=128, page=16, len_lo=490,
             len_hi=490, new_lo=1, new_hi=1, causal=False),
        # a decode step of 32 requests between a short prompt and a full context
        dict(name="attend4_batch", op="attend4", dtype="bf16", batch=32, heads=32, kv_heads=8, dim=128, page=16, len_lo=234,
             len_hi=16384, new_lo=1, new_hi=1, causal=False),
        # two requests deep in very long contexts
        dict(name="attend4_long", op="attend4", dtype="f16", batch=2, heads=32, kv_heads=8, dim=128, page=64, len_lo=100001,
             len_hi=131072, new_lo=1, new_hi=1, causal=False),
        # drafted tokens checked together, odd group of five small heads
        dict(name="attend4_draft", op="attend4", dtype="bf16", batch=16, heads=40, kv_heads=8, dim=64, page=32, len_lo=900,
             len_hi=9001, new_lo=1, new_hi=5, causal=True),
        # chunks of two prompts over a long context, causal
        dict(name="attend4_chunk", op="attend4", dtype="bf16", batch=2, heads=32, kv_heads=8, dim=128, page=64, len_lo=9000,
             len_hi=16384, new_lo=700, new_hi=1024, causal=True),
        # a frame's tokens over a window of 21 frames, every head with its own keys
        dict(name="attend4_window", op="attend4", dtype="bf16", batch=1, heads=12, kv_heads=12, dim=128, page=128,
             len_lo=32760, len_hi=32760, new_lo=1560, new_hi=1560, causal=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["axes", "append4", "attend4", "attend4", "chunk"])
    heads, kv_heads = rng.choice([(32, 8), (40, 40), (12, 12), (40, 8), (12, 4), (16, 2), (8, 1)])
    c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), heads=heads, kv_heads=kv_heads, dim=rng.choice([64, 128]),
             page=rng.choice([16, 32, 64, 128]))
    if op in ("axes", "append4"):
        if op == "axes":
            c["dtype"] = rng.choice(["bf16", "f16", "f32"])
        c["batch"] = _log(rng, 1, 64)
        top = rng.choice([1, min(1560, 3100 * 40 // kv_heads // c["batch"])])
        c["new_hi"] = max(1, _log(rng, 1, max(1, top)))
        c["new_lo"] = rng.randint(1, c["new_hi"])
        c["len_lo"] = c["new_hi"] + rng.randint(0, 2000)
        c["len_hi"] = c["len_lo"] + rng.randint(0, 2000)
        c.update(half=rng.random() < 0.5, axes=rng.choice(["sections", "turns"] + ["none"] * (op == "append4")))
        return c
    c["op"] = "attend4"
    if op == "chunk":
        c.update(causal=rng.random() < 0.8, batch=rng.randint(1, 3))
        c["new_hi"] = _log(rng, 8, 900)
        c["new_lo"] = rng.randint(1, c["new_hi"])
        c["len_hi"] = c["new_hi"] + _log(rng, 1, 8000)
        c["len_lo"] = rng.randint(c["new_hi"], c["len_hi"])
        return c
    c["batch"] = _log(rng, 1, 40)
    c["len_hi"] = _log(rng, 1, 1000000 // (c["batch"] * kv_heads // 4 + 8))
    c["len_lo"] = rng.randint(1, c["len_hi"])
    c["new_hi"] = rng.choice([1, 1, 1, min(3, c["len_lo"])])
    c.update(new_lo=1, causal=True)
    return c


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spread, not in order."""
    v = [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]
    return v[::2] + v[1::2][::-1]


def _rows(c):
    return _spread(c["len_lo"], c["len_hi"], c["batch"]), _spread(c["new_lo"], c["new_hi"], c["batch"])


def _table_rows(c):
    """Rows of the table of angles: slots, or 600 positions that begin anywhere and what a grid of the new tokens adds."""
    return c["len_hi"] if c["axes"] == "none" else 600 + c["new_hi"]


def work(c):
    lens, new = _rows(c)
    h, hkv, d = c["heads"], c["kv_heads"], c["dim"]
    eb = 4 if c["dtype"] == "f32" else 2
    t = sum(new)
    held = 2 * hkv * (d // 2 + d // 32)                    # one slot's key and value in 4 bits
    qo = 2 * t * h * d * eb                                # queries in, queries or outputs out
    if c["op"] == "attend4":
        seen = sum(m * n - (m * (m - 1) // 2 if c["causal"] else 0) for n, m in zip(lens, new))
        return dict(bytes=sum(lens) * held + qo + 4 * t * h, flops=4 * h * d * seen)
    kv = 2 * hkv * d * eb
    angles = min(t, _table_rows(c)) * d * 4 + (0 if c["axes"] == "none" else 12 * t)
    moved = 2 * t * kv if c["op"] == "axes" else t * (2 * kv + 2 * held)     # (held: written, and read back)
    return dict(bytes=moved + qo + angles, flops=3 * t * (h + hkv) * d)


# --------------------------------------------------------------------------------------------------------- inputs
def _pair_axis(c):
    """The axis (0 time, 1 height, 2 width) that each of the dim / 2 pairs goes by: a quarter of them to time and the rest
    evenly to height and width, side by side or in turns."""
    n = c["dim"] // 2
    if c["axes"] == "sections":
        return [0] * (n // 4) + [1] * (3 * n // 8) + [2] * (3 * n // 8)
    return [j % 3 for j in range(n)]


def _grid(m, start):
    """Positions of m tokens: one is text; more are an image's rows or a video's frames of at most 30 x 52."""
    if m == 1:
        return [[start] * 3]
    w = min(52, max(1, math.isqrt(m)))
    return [[start + i // (30 * w), start + i // w % 30, start + i % w] for i in range(m)]


def prepare(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    lens, new = _rows(c)
    b, h, hkv, d, ps = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    pages = [-(-n // ps) for n in lens]
    n_pages = sum(pages) + 3                               # a pool with a few free pages
    max_pages = max(pages) + 1
    randn = lambda *s: torch.randn(s, generator=g, device=dev, dtype=torch.float32)  # noqa: E731
    perm = torch.randperm(n_pages, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    table = torch.full((b, max_pages), -1, dtype=torch.int32, device=dev)
    at = 0
    for i, p in enumerate(pages):
        table[i, :p] = perm[at:at + p]
        at += p
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    s = dict(c=c, table=table, kv_len=ints(lens), cu=ints(cu) if c["new_hi"] > 1 else None, total=cu[-1], max_q=max(new))
    if c["op"] == "attend4":
        s["q"] = randn(cu[-1], h, d).to(dt)
        s["pool"] = torch.empty(n_pages, hkv, ps * (d + d // 16), dtype=torch.uint8, device=dev)
        for lo in range(0, n_pages, 512):                  # keys have a few channels of larger values
            n = min(512, n_pages - lo)
            k, v = randn(n, ps, hkv, d), randn(n, ps, hkv, d)
            k[..., ::29] *= 4
            s["pool"][lo:lo + n] = _pack(_quantised(k.to(dt)), _quantised(v.to(dt)))
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(cu[-1], h, dtype=torch.float32, device=dev)
    else:
        inv = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64, device=dev) / d)
        ang = torch.arange(_table_rows(c), dtype=torch.float64, device=dev)[:, None] * inv
        s["rope"] = torch.stack([ang.cos(), ang.sin()], -1).float().contiguous()
        # keys, values and queries as a model's joint projection leaves them: slices of one buffer
        joint = randn(cu[-1], h + 2 * hkv, d).to(dt)
        s["q"], s["k_new"], s["v_new"] = joint[:, :h], joint[:, h:h + hkv], joint[:, h + hkv:]
        s["q_out"] = torch.empty(cu[-1], h, d, dtype=dt, device=dev)
        row = torch.repeat_interleave(torch.arange(b, device=dev), ints(new).long())
        s["slot"] = ints(lens).long()[row] - ints(new).long()[row] + torch.arange(cu[-1], device=dev) - ints(cu).long()[row]
        s["row"] = row
        if c["axes"] != "none":
            start = torch.randint(0, 500, (b,), generator=g, device=dev).tolist()
            s["pos"] = ints([p for m, x in zip(new, start) for p in _grid(m, x)])
            s["pair_axis"] = _pair_axis(c)
        if c["op"] == "axes":
            s["k"], s["v"] = randn(n_pages, ps, hkv, d).to(dt), randn(n_pages, ps, hkv, d).to(dt)
        else:
            s["pool"] = torch.randint(0, 120, (n_pages, hkv, ps * (d + d // 16)), generator=g, device=dev, dtype=torch.uint8)
            s["k_out"], s["v_out"] = (torch.empty(cu[-1], hkv, d, dtype=dt, device=dev) for _ in range(2))
    if own:
        from diffusion_serving_gb300 import paged, paged4
        size = dict(page_size=ps, n_pages=n_pages, max_pages=max_pages, max_tokens=cu[-1], block_table=table, kv_len=s["kv_len"])
        if c["op"] == "axes":
            s["cache"] = paged.PagedKVCache(b, h, hkv, d, dt, k_pages=s["k"], v_pages=s["v"], **size)
        else:
            s["cache"] = paged4.PagedKVCache4(b, h, hkv, d, dt, pages=s["pool"], **size)
        s["axes"] = paged.rope_axes(s["pair_axis"]) if "pair_axis" in s else None
    return s


# ------------------------------------------------------------------------------------------------------------ run
def run(s):
    op = s["c"]["op"]
    if own:
        cache, c = s["cache"], s["c"]
        if op == "attend4":
            return cache.attend(s["q"], cu_q=s["cu"], max_q=s["max_q"], out=s["out"], lse=s["lse"],
                                flags=1 if c["causal"] else 0)               # paged.CAUSAL
        cache.append(s["k_new"], s["v_new"], cu_new=s["cu"], rope=s["rope"], half=c["half"], q=s["q"], q_out=s["q_out"],
                     positions=s.get("pos"), axes=s["axes"])
        if op == "axes":
            return [s["k"], s["v"], s["q_out"]]
        cache.read(s["total"], cu=s["cu"], k_out=s["k_out"], v_out=s["v_out"])
        return [s["k_out"], s["v_out"], s["q_out"]]
    if op == "axes":
        return _plain_axes(s)
    return _plain_append4(s) if op == "append4" else _plain_attend4(s)


def _rotated(s, x):
    """x [tokens, heads, dim] turned at its positions, in its own type.  In 64 bits and rounded once, as what is next to
    a border between two codes must not depend on 32 bits' rounding."""
    c, n = s["c"], s["c"]["dim"] // 2
    if "pos" in s:
        axis = torch.tensor(s["pair_axis"], device=x.device)
        cs = s["rope"][s["pos"].long()[:, axis], torch.arange(n, device=x.device)]       # [tokens, n, 2]
    else:
        cs = s["rope"][s["slot"]]
    cos, sin = cs[:, None, :, 0].double(), cs[:, None, :, 1].double()
    y = x.double()
    a, b = (y[..., :n], y[..., n:]) if c["half"] else (y[..., 0::2], y[..., 1::2])
    a, b = a * cos - b * sin, a * sin + b * cos
    return _rounded(torch.cat([a, b], -1) if c["half"] else torch.stack([a, b], -1).flatten(-2), x.dtype)


def _rounded(y, dt):
    """64 bits to `dt` in one rounding: to odd in 32 bits first where dt is narrower."""
    z = y.float()
    if dt == torch.float32:
        return z
    over = z.double().abs() > y.abs()
    bits = z.view(torch.int32) - over.int()                # toward zero
    bits = torch.where(bits.view(torch.float32).double() != y, bits | 1, bits)
    return bits.view(torch.float32).to(dt)


def _plain_axes(s):
    page, off = s["table"][s["row"], s["slot"] // s["c"]["page"]].long(), s["slot"] % s["c"]["page"]
    s["k"][page, off] = _rotated(s, s["k_new"])
    s["v"][page, off] = s["v_new"]
    s["q_out"].copy_(_rotated(s, s["q"]))
    return [s["k"], s["v"], s["q_out"]]


def _quantised(x):
    """Codes [..., dim] (whole numbers from 1 to 15) and scales [..., dim / 32] of x [..., dim]."""
    g = x.float().unflatten(-1, (-1, 32))
    top = g.abs().amax(-1)
    top = top / torch.full_like(top, 7)                    # (divided: torch multiplies by a number's reciprocal)
    scale = top.clamp(max=448).to(torch.float8_e4m3fn)
    f = scale.float()[..., None]
    code = torch.where(f > 0, torch.round(g / f), torch.zeros_like(g)).clamp(-7, 7) + 8
    return code.flatten(-2).to(torch.uint8), scale


def _words(code):
    """Codes [..., dim] as bytes [..., dim / 2]."""
    w = code.to(torch.int32).unflatten(-1, (-1, 4, 2))     # [..., word, i, half]
    at = torch.arange(4, device=code.device)[:, None] * 4 + torch.arange(2, device=code.device) * 16
    return (w << at).sum((-2, -1), dtype=torch.int32).view(torch.uint8)


def _place(ps, d, device):
    """Where the 16-byte piece x of a value's codes stands, for each slot: [page, dim / 32]."""
    n = d // 32
    return torch.arange(n, device=device) ^ ((torch.arange(ps, device=device)[:, None] >> 2) % n)


def _pack(k, v):
    """Records [pages, kv_heads, bytes] from the codes and scales of keys and values, [pages, page, kv_heads, ...] each."""
    (kc, ks), (vc, vs) = k, v
    ps, d = kc.shape[1], kc.shape[-1]
    kc, ks, vc, vs = (x.transpose(1, 2) for x in (_words(kc), ks.view(torch.uint8), _words(vc), vs.view(torch.uint8)))
    vc = vc.unflatten(-1, (-1, 16))
    at = _place(ps, d, vc.device)[..., None].expand(vc.shape)              # (its own inverse)
    vc = torch.gather(vc, 3, at)
    return torch.cat([x.flatten(2) for x in (kc, vc, ks, vs.transpose(2, 3))], -1)


def _unpacked(pool, ps, d):
    """Keys and values [pages, page, kv_heads, dim] in 32 bits from records."""
    n = ps * d // 2
    pages, hkv = pool.shape[:2]
    kc = pool[..., :n].reshape(pages, hkv, ps, d // 2)
    vc = pool[..., n:2 * n].reshape(pages, hkv, ps, d // 32, 16)
    vc = torch.gather(vc, 3, _place(ps, d, pool.device)[..., None].expand(vc.shape)).flatten(3)
    ks = pool[..., 2 * n:2 * n + ps * d // 32].reshape(pages, hkv, ps, d // 32)
    vs = pool[..., 2 * n + ps * d // 32:].reshape(pages, hkv, d // 32, ps).transpose(2, 3)
    at = torch.arange(4, device=pool.device)[:, None] * 4 + torch.arange(2, device=pool.device) * 16
    out = []
    for code, scale in ((kc, ks), (vc, vs)):
        w = code.contiguous().view(torch.int32)
        x = ((w[..., None, None] >> at) & 15).flatten(-3).float() - 8
        x = x.unflatten(-1, (-1, 32)) * scale.contiguous().view(torch.float8_e4m3fn).float()[..., None]
        out.append(x.flatten(-2).transpose(1, 2))
    return out


def _plain_append4(s):
    c = s["c"]
    ps, d, hkv = c["page"], c["dim"], c["kv_heads"]
    k, v = _quantised(_rotated(s, s["k_new"])), _quantised(s["v_new"])
    s["q_out"].copy_(_rotated(s, s["q"]))
    # codes and scales into the slots' places within their records
    page, off = s["table"][s["row"], s["slot"] // ps].long()[:, None], (s["slot"] % ps)[:, None]
    head = torch.arange(hkv, device=page.device)[None]
    n = ps * d // 2
    pool = s["pool"]
    pool[..., :n].unflatten(-1, (ps, d // 2))[page, head, off] = _words(k[0])
    at = _place(ps, d, page.device)[off[:, 0]][:, None, :, None].expand(-1, hkv, -1, 16)
    vc = torch.gather(_words(v[0]).unflatten(-1, (-1, 16)), 2, at).flatten(2)
    pool[..., n:2 * n].unflatten(-1, (ps, d // 2))[page, head, off] = vc
    pool[..., 2 * n:2 * n + ps * d // 32].unflatten(-1, (ps, d // 32))[page, head, off] = k[1].view(torch.uint8)
    pool[..., 2 * n + ps * d // 32:].unflatten(-1, (d // 32, ps)).transpose(2, 3)[page, head, off] = v[1].view(torch.uint8)
    # and what the slots then hold
    for (code, scale), out in ((k, s["k_out"]), (v, s["v_out"])):
        x = (code.float() - 8).unflatten(-1, (-1, 32)) * scale.float()[..., None]
        out.copy_(x.flatten(-2))
    return [s["k_out"], s["v_out"], s["q_out"]]


def _plain_attend4(s):
    c, ps = s["c"], s["c"]["page"]
    h, hkv, d = c["heads"], c["kv_heads"], c["dim"]
    lens = s["kv_len"].long()
    b, n = c["batch"], s["max_q"]
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(b + 1, device=lens.device)
    row = torch.repeat_interleave(torch.arange(b, device=lens.device), cu[1:] - cu[:-1], output_size=s["total"])
    i = torch.arange(s["total"], device=lens.device) - cu[row]
    q = torch.zeros(b, n, h, d, device=lens.device)
    q[row, i] = s["q"].float()
    k, v = _unpacked(s["pool"], ps, d)
    pages = s["table"].clamp(min=0).long()
    k = k[pages].flatten(1, 2).permute(0, 2, 3, 1)                                    # [b, hkv, d, slots]
    v = v[pages].flatten(1, 2).permute(0, 2, 1, 3)                                    # [b, hkv, slots, d]
    q = q.view(b, n, hkv, h // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)  # [b, hkv, g n, d]
    x = torch.matmul(q, k) * d ** -0.5
    slot = torch.arange(x.shape[-1], device=x.device)
    end = lens[:, None].expand(b, n)
    if c["causal"]:
        end = (lens - (cu[1:] - cu[:-1]))[:, None] + torch.arange(n, device=x.device) + 1
    dead = slot >= end[..., None]                                                     # [b, n, slots]
    x.view(b, hkv, h // hkv, n, -1).masked_fill_(dead[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    v = v.masked_fill((slot >= lens[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(x, v) / total
    lse = (m + torch.log(total))[..., 0]
    o = o.view(b, hkv, h // hkv, n, d).permute(0, 3, 1, 2, 4).reshape(b, n, h, d)
    lse = lse.view(b, hkv, h // hkv, n).permute(0, 3, 1, 2).reshape(b, n, h)
    return o[row, i].to(s["q"].dtype), lse[row, i]


# ---------------------------------------------------------------------------------------------------------- exact
def exact(c, seed):
    """The definitions row by row in 64 bits."""
    global own
    was, own = own, False
    s = prepare(c, seed)
    own = was
    lens, new = _rows(c)
    h, hkv, d, ps = c["heads"], c["kv_heads"], c["dim"], c["page"]
    table = s["table"].tolist()
    if c["op"] != "attend4":
        z = torch.complex(s["rope"][..., 0].double(), s["rope"][..., 1].double())

        def turn(x, at, p):                                # tokens at .. of the call, at slots p
            if "pos" in s:
                where = s["pos"][at:at + len(p)].long()
                zz = torch.stack([z[where[:, a], j] for j, a in enumerate(s["pair_axis"])], -1)
            else:
                zz = z[p]
            pair = torch.stack([x[..., :d // 2], x[..., d // 2:]], -1) if c["half"] else x.unflatten(-1, (d // 2, 2))
            y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * zz[:, None])
            return torch.cat([y[..., 0], y[..., 1]], -1) if c["half"] else y.flatten(-2)

        q = s["q"].double()
        k_new, v_new = s["k_new"].double(), s["v_new"].double()
        k, v = (s["k"].double(), s["v"].double()) if c["op"] == "axes" else (None, None)
        at = 0
        for i, (n, m) in enumerate(zip(lens, new)):
            p = torch.arange(n - m, n, device=q.device)
            k_new[at:at + m] = turn(k_new[at:at + m], at, p)
            q[at:at + m] = turn(q[at:at + m], at, p)
            if k is not None:
                for col in range((n - m) // ps, (n - 1) // ps + 1):
                    lo, hi = max(n - m, col * ps), min(n, col * ps + ps)
                    k[table[i][col], lo - col * ps:hi - col * ps] = k_new[at + lo - n + m:at + hi - n + m]
                    v[table[i][col], lo - col * ps:hi - col * ps] = v_new[at + lo - n + m:at + hi - n + m]
            at += m
        if c["op"] == "axes":
            return [k, v, q]
        # what is held depends on the rotated keys' rounding to 16 bits first
        step = 2.0 ** (-7 if c["dtype"] == "bf16" else -10)

        def held(x):
            e = torch.floor(torch.log2(x.abs().clamp(min=1e-30)))
            e = torch.where(torch.exp2(e) > x.abs(), e - 1, e)
            e = e.clamp(min=-126 if c["dtype"] == "bf16" else -14)
            ulp = torch.exp2(e) * step
            x = torch.round(x / ulp) * ulp
            g = x.reshape(*x.shape[:-1], d // 32, 32)
            top = g.abs().amax(-1, keepdim=True)
            top = top / torch.full_like(top, 7)            # (a number's reciprocal would not be exact)
            e = torch.floor(torch.log2(top.clamp(min=2.0 ** -40))).clamp(min=-6)     # e4m3: 3 bits behind the point, from 2^-6
            sc = (torch.round(top / torch.exp2(e - 3)) * torch.exp2(e - 3)).clamp(max=448)
            y = torch.where(sc > 0, torch.round(g / sc.clamp(min=2.0 ** -9)).clamp(-7, 7) * sc, torch.zeros_like(g))
            return y.reshape(x.shape)

        return [held(k_new), held(v_new), q]
    out = torch.zeros(s["total"], h, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["total"], h, dtype=torch.float64, device="cuda")
    g = h // hkv
    # where dim t of a word stands: bits 16 (t odd) + 4 (t / 2)
    bit = torch.tensor([16 * (t % 2) + 4 * (t // 2) for t in range(8)], device="cuda")
    dims = torch.arange(d, device="cuda")
    byte, shift = dims // 8 * 4 + bit[dims % 8] // 8, bit[dims % 8] % 8
    codes = ps * d // 2

    def e4m3(u):                                           # from its bits
        u = u.long()
        e, f = u >> 3 & 15, (u & 7).double()
        return torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2(e.double() - 10))

    at = 0
    for i, (n, m) in enumerate(zip(lens, new)):
        pages = torch.tensor(table[i][:-(-n // ps)], device="cuda")
        slots = torch.arange(n, device="cuda")
        off = slots % ps
        for e in range(hkv):
            rec = s["pool"][pages, e][slots // ps]                                    # [n, bytes]
            kb = torch.gather(rec, 1, off[:, None] * (d // 2) + byte)
            piece = (byte // 16) ^ ((off[:, None] // 4) % (d // 32))
            vb = torch.gather(rec, 1, codes + off[:, None] * (d // 2) + piece * 16 + byte % 16)
            ks = torch.gather(rec, 1, 2 * codes + off[:, None] * (d // 32) + dims // 32)
            vs = torch.gather(rec, 1, 2 * codes + ps * d // 32 + dims // 32 * ps + off[:, None])
            kk = ((kb >> shift & 15).double() - 8) * e4m3(ks)
            vv = ((vb >> shift & 15).double() - 8) * e4m3(vs)
            del rec, kb, vb, ks, vs
            for lo in range(0, m, 256):
                hi = min(m, lo + 256)
                qq = s["q"][at + lo:at + hi, e * g:(e + 1) * g].double()              # [tokens, g, d]
                x = torch.einsum("mgd,sd->mgs", qq, kk) / math.sqrt(d)
                if c["causal"]:
                    x = x.masked_fill(slots > torch.arange(n - m + lo, n - m + hi, device="cuda")[:, None, None], -math.inf)
                lse[at + lo:at + hi, e * g:(e + 1) * g] = torch.logsumexp(x, -1)
                out[at + lo:at + hi, e * g:(e + 1) * g] = torch.einsum("mgs,sd->mgd", torch.softmax(x, -1), vv)
        at += m
    return [out, lse]
