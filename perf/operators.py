"""The paged K/V cache's operators, measured: what each is called with, its plain form, and its work.

 append   new tokens' keys (rotated at their positions) and values into the pages of their rows, the queries rotated
          beside them, and each touched page's channelwise key bounds kept
 attend   softmax attention of one token, a few, or a chunk per row over the row's pages
 shared   the same for rows whose first slots are one list of pages
 sparse   single tokens over the pages whose key bounds promise the largest scores

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
        # a decode step of 32 requests: one token each, queries rotated too (latency)
        dict(name="append_step", op="append", dtype="f16", batch=32, heads=32, kv_heads=8, dim=128, page=16,
             len_lo=234, len_hi=4096, new_lo=1, new_hi=1, half=True, bounds=True),
        # prompts of different lengths admitted in one call, every head with its own keys
        dict(name="append_prompts", op="append", dtype="bf16", batch=8, heads=40, kv_heads=40, dim=128, page=64,
             len_lo=512, len_hi=1560, new_lo=512, new_hi=1560, half=False, bounds=False),
        # a chunk of each prompt behind what is stored, odd sizes, bounds kept, 32-bit store
        dict(name="append_chunk", op="append", dtype="f32", batch=3, heads=12, kv_heads=4, dim=64, page=32,
             len_lo=777, len_hi=4097, new_lo=333, new_hi=777, half=True, bounds=True),
        # one request's decode step at the middle of a short answer (latency)
        dict(name="attend_one", op="attend", dtype="f16", batch=1, heads=32, kv_heads=8, dim=128, page=16,
             len_lo=490, len_hi=490, new_lo=1, new_hi=1, causal=False),
        # a decode step of 32 requests between a short prompt and a full context
        dict(name="attend_batch", op="attend", dtype="bf16", batch=32, heads=32, kv_heads=8, dim=128, page=16,
             len_lo=234, len_hi=16384, new_lo=1, new_hi=1, causal=False),
        # chunks of two prompts over a long context, causal
        dict(name="attend_chunk", op="attend", dtype="bf16", batch=2, heads=32, kv_heads=8, dim=128, page=64,
             len_lo=9000, len_hi=16384, new_lo=700, new_hi=1024, causal=True),
        # a few requests behind one system prompt
        dict(name="shared_few", op="shared", dtype="f16", batch=8, heads=32, kv_heads=8, dim=128, page=16,
             prefix=4096, len_lo=4112, len_hi=4500, new_lo=1, new_hi=1, causal=False),
        # many requests behind one long document
        dict(name="shared_many", op="shared", dtype="bf16", batch=64, heads=32, kv_heads=8, dim=128, page=64,
             prefix=32768, len_lo=32800, len_hi=33792, new_lo=1, new_hi=1, causal=False),
        # drafted tokens checked together, odd group of five heads
        dict(name="shared_draft", op="shared", dtype="bf16", batch=16, heads=40, kv_heads=8, dim=64, page=32,
             prefix=8192, len_lo=8200, len_hi=9001, new_lo=1, new_hi=5, causal=True),
        # one request deep in a long context
        dict(name="sparse_one", op="sparse", dtype="f16", batch=1, heads=32, kv_heads=8, dim=128, page=16,
             len_lo=32768, len_hi=32768, new_lo=1, new_hi=1, select=64),
        # a batch of long contexts
        dict(name="sparse_batch", op="sparse", dtype="bf16", batch=16, heads=32, kv_heads=8, dim=128, page=16,
             len_lo=8000, len_hi=32768, new_lo=1, new_hi=1, select=128),
        # wide pages, small heads, some rows shorter than what is selected
        dict(name="sparse_wide", op="sparse", dtype="bf16", batch=12, heads=16, kv_heads=4, dim=64, page=64,
             len_lo=500, len_hi=30001, new_lo=1, new_hi=1, select=24),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend_chunk", "shared", "sparse"])
    heads, kv_heads = rng.choice([(32, 8), (40, 40), (12, 12), (40, 8), (12, 4), (16, 2), (8, 1)])
    c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), heads=heads, kv_heads=kv_heads, dim=rng.choice([64, 128]),
             page=rng.choice([16, 32, 64, 128]))
    if op == "append":
        c["dtype"] = rng.choice(["bf16", "f16", "f32"])
        c["batch"] = _log(rng, 1, 64)
        top = rng.choice([1, min(1560, 12000 // c["batch"])])
        c["new_hi"] = max(1, _log(rng, 1, top))
        c["new_lo"] = rng.randint(1, c["new_hi"])
        c["len_lo"] = c["new_hi"] + rng.randint(0, 2000)
        c["len_hi"] = c["len_lo"] + rng.randint(0, 2000)
        c.update(half=rng.random() < 0.5, bounds=rng.random() < 0.5)
        return c
    if op == "attend_chunk":
        c.update(op="attend", causal=rng.random() < 0.8, batch=rng.randint(1, 3))
        c["new_hi"] = _log(rng, 8, 900)
        c["new_lo"] = rng.randint(1, c["new_hi"])
        c["len_hi"] = c["new_hi"] + _log(rng, 1, 8000)
        c["len_lo"] = rng.randint(c["new_hi"], c["len_hi"])
        return c
    c["batch"] = _log(rng, 1, 40)
    if op == "attend":
        c["len_hi"] = _log(rng, 1, 260000 // (c["batch"] * c["kv_heads"] // 4 + 8))
        c["len_lo"] = rng.randint(1, c["len_hi"])
        c["new_hi"] = rng.choice([1, 1, 1, min(3, c["len_lo"])])
        c.update(new_lo=1, causal=True)
    elif op == "shared":
        c["prefix"] = c["page"] * max(1, _log(rng, 128, 24000 // (1 + c["batch"] * c["kv_heads"] // 200)) // c["page"])
        c["len_lo"] = c["prefix"] + rng.randint(8, 200)
        c["len_hi"] = c["len_lo"] + rng.randint(0, 900)
        c["new_hi"] = rng.choice([1, 1, 4])
        c.update(new_lo=1, causal=True)
    else:
        c["len_hi"] = _log(rng, 200, min(40000, 2000000 // (c["batch"] * c["kv_heads"])))
        c["len_lo"] = rng.randint(1, c["len_hi"])
        c["select"] = rng.randint(2, 2048 // c["page"])
        c.update(new_lo=1, new_hi=1)
    return c


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spread, not in order."""
    v = [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]
    return v[::2] + v[1::2][::-1]


def _rows(c):
    return _spread(c["len_lo"], c["len_hi"], c["batch"]), _spread(c["new_lo"], c["new_hi"], c["batch"])


def work(c):
    lens, new = _rows(c)
    h, hkv, d, ps = c["heads"], c["kv_heads"], c["dim"], c["page"]
    eb = 4 if c["dtype"] == "f32" else 2
    kv = 2 * hkv * d * eb                                  # one slot's key and value
    t = sum(new)
    qo = 2 * t * h * d * eb                                # queries in, outputs out
    pages = [-(-n // ps) for n in lens]
    if c["op"] == "append":
        touched = sum((n - 1) // ps - (n - m) // ps + 1 for n, m in zip(lens, new)) if c["bounds"] else 0
        return dict(bytes=2 * t * kv + qo + t * d * 4 + touched * hkv * 2 * d * eb * 2, flops=3 * t * (h + hkv) * d)
    seen = sum(m * n - (m * (m - 1) // 2 if c.get("causal") else 0) for n, m in zip(lens, new))
    if c["op"] == "attend":
        return dict(bytes=sum(lens) * kv + qo + 4 * t * h, flops=4 * h * d * seen)
    if c["op"] == "shared":
        return dict(bytes=(c["prefix"] + sum(n - c["prefix"] for n in lens)) * kv + qo + 4 * t * h, flops=4 * h * d * seen)
    sel = [min(n, c["select"] * ps) for n in lens]
    return dict(bytes=sum(pages) * kv + sum(sel) * kv + qo + 4 * t * h + 4 * c["batch"] * hkv * c["select"],
                flops=4 * h * d * (sum(pages) + sum(sel)))


# --------------------------------------------------------------------------------------------------------- inputs
def prepare(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    lens, new = _rows(c)
    b, h, hkv, d, ps = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    pages = [-(-n // ps) for n in lens]
    shared = c.get("prefix", 0) // ps
    total = shared + sum(p - shared for p in pages)
    n_pages = total + 3                                    # a pool with a few free pages
    max_pages = max(pages) + 1
    randn = lambda *s: torch.randn(s, generator=g, device=dev, dtype=torch.float32)  # noqa: E731
    # keys of a page lie near one another: a part common to the page, a part of each slot's own
    k = (0.6 * randn(n_pages, 1, hkv, d) + 0.8 * randn(n_pages, ps, hkv, d)).to(dt)
    v = randn(n_pages, ps, hkv, d).to(dt)
    perm = torch.randperm(n_pages, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    table = torch.full((b, max_pages), -1, dtype=torch.int32, device=dev)
    at = shared
    for i, p in enumerate(pages):
        table[i, :shared] = perm[:shared]
        table[i, shared:p] = perm[at:at + p - shared]
        at += p - shared
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    s = dict(c=c, k=k, v=v, table=table, kv_len=ints(lens), cu=ints(cu) if c["new_hi"] > 1 else None, total=cu[-1],
             q=randn(cu[-1], h, d).to(dt), max_q=max(new))
    if c["op"] == "append":
        n_pos = max(lens)
        inv = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64, device=dev) / d)
        ang = torch.arange(n_pos, dtype=torch.float64, device=dev)[:, None] * inv
        s["rope"] = torch.stack([ang.cos(), ang.sin()], -1).float().contiguous()
        # keys, values and queries as a model's joint projection leaves them: slices of one buffer
        joint = randn(cu[-1], h + 2 * hkv, d).to(dt)
        s["q"], s["k_new"], s["v_new"] = joint[:, :h], joint[:, h:h + hkv], joint[:, h + hkv:]
        s["q_out"] = torch.empty(cu[-1], h, d, dtype=dt, device=dev)
        row = torch.repeat_interleave(torch.arange(b, device=dev), ints(new).long())
        s["pos"] = ints(lens).long()[row] - ints(new).long()[row] + torch.arange(cu[-1], device=dev) - ints(cu).long()[row]
        s["row"] = row
    else:
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(cu[-1], h, dtype=torch.float32, device=dev)
    if c["op"] == "shared":
        s["prefix_pages"], s["prefix_len"] = perm[:shared].contiguous(), ints([c["prefix"]])
    if c["op"] == "sparse":
        s["selected"] = torch.empty(b, hkv, c["select"], dtype=torch.int32, device=dev)
    if c["op"] == "sparse" or c.get("bounds"):
        s["bounds"] = _bounds(s, lens, new if c["op"] == "append" else [0] * b)
    if own:
        from diffusion_serving_gb300 import paged
        s["cache"] = paged.PagedKVCache(b, h, hkv, d, dt, page_size=ps, n_pages=n_pages, max_pages=max_pages,
                                        max_tokens=cu[-1], k_pages=k, v_pages=v, block_table=table,
                                        kv_len=s["kv_len"], bounds=s.get("bounds"))
    return s


def _bounds(s, lens, new):
    """Each page's key maximum and minimum per channel over the slots that are filled: [pages, kv_heads, 2, dim]."""
    k, table, ps = s["k"], s["table"], s["c"]["page"]
    filled = torch.tensor([n - m for n, m in zip(lens, new)], device=k.device)
    count = (filled[:, None] - torch.arange(table.shape[1], device=k.device) * ps).clamp(0, ps)     # per row and column
    slots = torch.zeros(k.shape[0], dtype=torch.long, device=k.device)
    slots[table[table >= 0].long()] = count[table >= 0]
    ok = (torch.arange(ps, device=k.device) < slots[:, None])[:, :, None, None]
    low, high = k.masked_fill(~ok, float("inf")).amin(1), k.masked_fill(~ok, float("-inf")).amax(1)
    return torch.stack([high, low], 2).contiguous()


# ------------------------------------------------------------------------------------------------------------ run
def run(s):
    c = s["c"]
    op = c["op"]
    if own:
        cache = s["cache"]
        if op == "append":
            cache.append(s["k_new"], s["v_new"], cu_new=s["cu"], rope=s["rope"], half=c["half"], q=s["q"], q_out=s["q_out"])
            return [s["k"], s["v"], s["q_out"]] + ([s["bounds"]] if c["bounds"] else [])
        flags = 1 if c.get("causal") else 0                # paged.CAUSAL
        if op == "attend":
            return cache.attend(s["q"], cu_q=s["cu"], max_q=s["max_q"], out=s["out"], lse=s["lse"], flags=flags)
        if op == "shared":
            return cache.attend_shared(s["q"], s["prefix_pages"], s["prefix_len"], cu_q=s["cu"], max_q=s["max_q"],
                                       out=s["out"], lse=s["lse"], flags=flags)
        return cache.attend_sparse(s["q"], c["select"], out=s["out"], lse=s["lse"], selected=s["selected"])
    if op == "append":
        return _plain_append(s)
    if op == "sparse":
        return _plain_sparse(s)
    return _plain_attend(s)


def _rotate(x, cs, half):
    """x [n, heads, d] turned by cs [n, d/2, 2], in 32 bits."""
    x = x.float()
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    n = x.shape[-1] // 2
    a, b = (x[..., :n], x[..., n:]) if half else (x[..., 0::2], x[..., 1::2])
    a, b = a * cos - b * sin, a * sin + b * cos
    return torch.cat([a, b], -1) if half else torch.stack([a, b], -1).flatten(-2)


def _plain_append(s):
    c, dt, ps = s["c"], s["k"].dtype, s["c"]["page"]
    pos, row = s["pos"], s["row"]
    cs = s["rope"][pos]
    page, off = s["table"][row, pos // ps].long(), pos % ps
    k_new = _rotate(s["k_new"], cs, c["half"]).to(dt)
    s["k"][page, off] = k_new
    s["v"][page, off] = s["v_new"]
    s["q_out"].copy_(_rotate(s["q"], cs, c["half"]).to(dt))
    if not c["bounds"]:
        return [s["k"], s["v"], s["q_out"]]
    # a page that these tokens begin starts anew; others widen
    old = s["bounds"].float()
    begun = page[off == 0]
    old[begun, :, 0], old[begun, :, 1] = float("-inf"), float("inf")
    to = page[:, None, None].expand(-1, *k_new.shape[1:])
    high = old[:, :, 0].clone().scatter_reduce(0, to, k_new.float(), "amax")
    low = old[:, :, 1].clone().scatter_reduce(0, to, k_new.float(), "amin")
    s["bounds"].copy_(torch.stack([high, low], 2).to(dt))
    return [s["k"], s["v"], s["q_out"], s["bounds"]]


def _padded(s, x, fill):
    """Packed rows [total, ...] as [batch, max_q, ...]; and each packed row's place in it."""
    b, n = s["c"]["batch"], s["max_q"]
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(b + 1, device=x.device)
    row = torch.repeat_interleave(torch.arange(b, device=x.device), cu[1:] - cu[:-1], output_size=s["total"])
    i = torch.arange(s["total"], device=x.device) - cu[row]
    p = x.new_full((b, n) + tuple(x.shape[1:]), fill)
    p[row, i] = x
    return p, row, i, cu[1:] - cu[:-1]


def _plain_attend(s):
    c, ps = s["c"], s["c"]["page"]
    h, hkv, d = c["heads"], c["kv_heads"], c["dim"]
    q, row, i, n_new = _padded(s, s["q"].float(), 0.0)
    b, n = q.shape[:2]
    lens = s["kv_len"].long()
    pages = s["table"].clamp(min=0).long()
    k = s["k"][pages].flatten(1, 2).float().permute(0, 2, 3, 1)                       # [b, hkv, d, slots]
    v = s["v"][pages].flatten(1, 2).float().permute(0, 2, 1, 3)                       # [b, hkv, slots, d]
    q = q.view(b, n, hkv, h // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)  # [b, hkv, g n, d]
    x = torch.matmul(q, k) * d ** -0.5
    slot = torch.arange(x.shape[-1], device=x.device)
    end = lens[:, None].expand(b, n)
    if c["causal"]:
        end = (lens - n_new)[:, None] + torch.arange(n, device=x.device) + 1
    dead = slot >= end[..., None]                                                     # [b, n, slots]
    x.view(b, hkv, h // hkv, n, -1).masked_fill_(dead[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = torch.exp(x - m)
    total = x.sum(-1, keepdim=True)
    v = v.masked_fill((slot >= lens[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(x, v) / total
    lse = (m + torch.log(total))[..., 0]
    o = o.view(b, hkv, h // hkv, n, d).permute(0, 3, 1, 2, 4).reshape(b, n, h, d)
    lse = lse.view(b, hkv, h // hkv, n).permute(0, 3, 1, 2).reshape(b, n, h)
    return o[row, i].to(s["q"].dtype), lse[row, i]


def _plain_sparse(s):
    c, ps = s["c"], s["c"]["page"]
    b, h, hkv, d, take = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["select"]
    lens = s["kv_len"].long()
    n_row = (lens + ps - 1) // ps
    pages = s["table"].clamp(min=0).long()                                            # [b, columns]
    column = torch.arange(pages.shape[1], device=pages.device)
    # scores next to the last one taken decide what is read: in 64 bits
    q = s["q"].double().view(b, hkv, h // hkv, d)
    bd = s["bounds"].double()[pages]                                                  # [b, columns, hkv, 2, d]
    up = torch.einsum("bhgd,bchd->bhgc", q.clamp(min=0), bd[:, :, :, 0])
    up = (up + torch.einsum("bhgd,bchd->bhgc", q.clamp(max=0), bd[:, :, :, 1])).amax(2)
    kept = (column == 0) | (column == n_row[:, None] - 1)                             # the first and the newest page
    up = up.masked_fill(kept[:, None], float("inf"))
    up = up.masked_fill((column >= n_row[:, None])[:, None], float("-inf"))
    order = torch.sort(up, dim=-1, descending=True, stable=True)[1]
    sel = torch.full((b, hkv, take), pages.shape[1], dtype=torch.long, device=up.device)
    sel[:, :, :order.shape[-1]] = order[:, :, :take]
    sel = torch.where(torch.arange(take, device=up.device) < n_row[:, None, None], sel, pages.shape[1]).sort(-1)[0]
    none = sel >= pages.shape[1]
    at = torch.gather(pages[:, None].expand(b, hkv, -1), 2, sel.clamp(max=pages.shape[1] - 1))
    head = torch.arange(hkv, device=up.device)[None, :, None]
    k = s["k"].transpose(1, 2)[at, head].flatten(2, 3).float()                        # [b, hkv, take page, d]
    v = s["v"].transpose(1, 2)[at, head].flatten(2, 3).float()
    slot = (sel[..., None] * ps + torch.arange(ps, device=up.device)).flatten(2)
    dead = (slot >= lens[:, None, None])
    x = torch.matmul(s["q"].float().view(b, hkv, h // hkv, d), k.transpose(2, 3)) * d ** -0.5
    x = x.masked_fill(dead[:, :, None], float("-inf"))
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = torch.exp(x - m)
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v.masked_fill(dead[..., None], 0.0)) / total
    lse = (m + torch.log(total)).view(b, h)
    return o.reshape(b, h, d).to(s["q"].dtype), lse, sel.masked_fill(none, -1).int()


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
    if c["op"] == "append":
        k, v, q = s["k"].double(), s["v"].double(), s["q"].double()
        bounds = s["bounds"].double() if c["bounds"] else None
        z = torch.complex(s["rope"][..., 0].double(), s["rope"][..., 1].double())

        def turn(x, p):
            pair = torch.stack([x[..., :d // 2], x[..., d // 2:]], -1) if c["half"] else x.unflatten(-1, (d // 2, 2))
            y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z[p][:, None])
            return torch.cat([y[..., 0], y[..., 1]], -1) if c["half"] else y.flatten(-2)

        at = 0
        for i, (n, m) in enumerate(zip(lens, new)):
            p = torch.arange(n - m, n, device=k.device)
            kn, vn = turn(s["k_new"][at:at + m].double(), p), s["v_new"][at:at + m].double()
            q[at:at + m] = turn(s["q"][at:at + m].double(), p)
            for col in range((n - m) // ps, (n - 1) // ps + 1):
                lo, hi = max(n - m, col * ps), min(n, col * ps + ps)
                piece, page = kn[lo - n + m:hi - n + m], table[i][col]
                k[page, lo - col * ps:hi - col * ps] = piece
                v[page, lo - col * ps:hi - col * ps] = vn[lo - n + m:hi - n + m]
                if bounds is not None:
                    high, low = piece.amax(0), piece.amin(0)
                    if lo > col * ps:
                        high, low = torch.maximum(high, bounds[page, :, 0]), torch.minimum(low, bounds[page, :, 1])
                    bounds[page, :, 0], bounds[page, :, 1] = high, low
            at += m
        return [k, v, q] + ([bounds] if bounds is not None else [])
    out = torch.zeros(s["total"], h, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["total"], h, dtype=torch.float64, device="cuda")
    g = h // hkv
    at = 0
    for i, (n, m) in enumerate(zip(lens, new)):
        pages = torch.tensor(table[i][:-(-n // ps)], device="cuda")
        for e in range(hkv):
            qq = s["q"][at:at + m, e * g:(e + 1) * g].double()                        # [m, g, d]
            if c["op"] == "sparse":
                bd = s["bounds"][pages, e].double()
                up = torch.maximum(qq[0][:, None] * bd[None, :, 0], qq[0][:, None] * bd[None, :, 1]).sum(-1).amax(0).tolist()
                up[0] = up[-1] = math.inf
                best = sorted(sorted(range(len(up)), key=lambda j: (-up[j], j))[:c["select"]])
                slots = torch.cat([torch.arange(j * ps, min(n, j * ps + ps), device="cuda") for j in best])
            else:
                slots = torch.arange(n, device="cuda")
            kk = s["k"][pages[slots // ps], slots % ps, e].double()
            vv = s["v"][pages[slots // ps], slots % ps, e].double()
            x = torch.einsum("mgd,sd->mgs", qq, kk) / math.sqrt(d)
            if c.get("causal"):
                x = x.masked_fill(slots > torch.arange(n - m, n, device="cuda")[:, None, None], -math.inf)
            lse[at:at + m, e * g:(e + 1) * g] = torch.logsumexp(x, -1)
            out[at:at + m, e * g:(e + 1) * g] = torch.einsum("mgs,sd->mgd", torch.softmax(x, -1), vv)
        at += m
    return [out, lse] + ([None] if c["op"] == "sparse" else [])
