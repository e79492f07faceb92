"""The operators of a paged key-value cache, as they are measured: page tables and slot maps from
request lengths, the append of new keys and values, and the attention of one or a few new rows a
request over the cache.

``run`` computes each operator in its plain form (elementary torch operations) or, where ``own`` is
true, by the library's call. 4 streams, 32 heads of 128, windows of 511 and rounds of 5 drafts and
up to 32 rows are those of the draft step; the other sizes are generic."""
import math

import numpy as np
import torch

own = False

F32, BF16, I32, F8 = torch.float32, torch.bfloat16, torch.int32, torch.float8_e4m3fn
EPS, BASE = 1e-6, 10000.0


# ---- cases -----------------------------------------------------------------------------------

def _plan(requests, lo, hi, new, page, prompt=0, **kw):
    """Request lengths lo..hi, 1..new rows each; ``prompt`` of the requests bring 64 times as many."""
    return dict(op="plan", requests=requests, lo=lo, hi=hi, new=new, page=page, prompt=prompt, **kw)


def _append(requests, rows, heads, dim, page, fmt="bf16", **kw):
    """``rows`` rows a request."""
    return dict(op="append", requests=requests, rows=rows, heads=heads, dim=dim, page=page, fmt=fmt,
                **kw)


def _attn(requests, lo, hi, new, q_heads, kv_heads, dim, page, fmt="bf16", window=-1, tree=False,
          ragged=False, **kw):
    """lo..hi cached keys and ``new`` rows a request (ragged: 1..new)."""
    return dict(op="attn", requests=requests, lo=lo, hi=hi, new=new, q_heads=q_heads,
                kv_heads=kv_heads, dim=dim, page=page, fmt=fmt, window=window, tree=tree,
                ragged=ragged, **kw)


def listed():
    return [
        # a round of the measured pass: four streams of five drafts and the token after
        _plan(4, 505, 515, 6, 16, name="plan_pass"),
        # a large batch with verify windows and a few prompt chunks
        _plan(2048, 1, 9000, 32, 16, prompt=16, name="plan_batch"),
        # one draft step's keys and values of four streams
        _append(4, 1, 32, 128, 64, name="append_step"),
        # the verify rows of 48 requests into an 8-bit cache
        _append(48, 6, 8, 128, 16, "e4m3", name="append_verify_e4m3"),
        # prompt chunks of three requests, an odd number of rows
        _append(3, 2731, 8, 128, 16, name="append_prompt"),
        # one request's next token after a short context: latency is all there is
        _attn(1, 777, 777, 1, 32, 8, 128, 16, name="attn_one"),
        # one draft step of four streams, every head with its own keys, the draft head's window
        _attn(4, 511, 515, 1, 32, 32, 128, 64, window=511, name="attn_pass"),
        # one request with a very long context
        _attn(1, 131041, 131041, 1, 32, 8, 128, 64, name="attn_long"),
        # a decode batch over an 8-bit cache
        _attn(64, 300, 9000, 1, 32, 8, 128, 16, "e4m3", name="attn_batch_e4m3"),
        # verify windows of five drafts and the token after, requests of all lengths
        _attn(24, 90, 7000, 6, 32, 8, 128, 16, ragged=True, name="attn_verify"),
        # trees of up to 32 drafts, eight query heads a key head, heads of 64
        _attn(12, 500, 5000, 32, 16, 2, 64, 32, tree=True, name="attn_tree"),
        # a large batch of long contexts, four rows each
        _attn(96, 1000, 16000, 4, 32, 8, 128, 32, name="attn_large"),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "attn"])
    if op == "plan":
        hi = _log_uniform(rng, 32, 9000)
        requests = _log_uniform(rng, 1, 2048)
        return _plan(requests, rng.randint(0, hi), hi, rng.randint(1, 32),
                     rng.choice([8, 16, 24, 32, 64, 128]), rng.choice([0, 0, min(requests, 8)]))
    if op == "append":
        heads, dim = rng.choice([1, 2, 5, 8, 32]), rng.choice([64, 128])
        requests = _log_uniform(rng, 1, 64)
        rows = _log_uniform(rng, 1, max(1, 8_000_000 // (requests * heads * dim)))
        return _append(requests, rows, heads, dim, rng.choice([8, 16, 24, 32, 64, 128]),
                       rng.choice(["bf16", "e4m3"]))
    kv_heads = rng.choice([1, 2, 4, 5, 8, 32])
    group = rng.choice([1, 4, 7, 8] if kv_heads < 32 else [1])
    dim, fmt = rng.choice([64, 128]), rng.choice(["bf16", "bf16", "e4m3"])
    tree = rng.random() < 0.25
    new = rng.randint(2, 32) if tree else rng.choice([1, 1, 1, rng.randint(2, 8), rng.randint(9, 32)])
    hi = _log_uniform(rng, 20, 131072)
    # at most the keys, and the (row, key) products, of the largest case
    most = min(600_000_000 // (hi * kv_heads * dim), 6_000_000_000 // (hi * kv_heads * group * dim * new))
    requests = _log_uniform(rng, 1, max(1, min(128, most)))
    window = -1 if tree else rng.choice([-1, -1, rng.randint(0, 511), rng.randint(512, 8192)])
    return _attn(requests, rng.randint(0, hi), hi, new, kv_heads * group, kv_heads, dim,
                 rng.choice([8, 16, 24, 32, 64, 128]), fmt, window, tree, rng.random() < 0.5)


# ---- inputs ----------------------------------------------------------------------------------

def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _spread(n, lo, hi):
    """n whole numbers spread over lo..hi, the same for every seed (their sum is the case's)."""
    if n == 1:
        return torch.tensor([hi])
    golden = 0.6180339887498949
    return torch.tensor([lo + int((hi + 1 - lo) * ((i * golden) % 1.0)) for i in range(n)])


def _lens_new(c):
    """Cached lengths and new rows a request, in the order before the seed's permutation."""
    n = c["requests"]
    if c["op"] == "append":
        return _spread(n, 3, 400), torch.full((n,), c["rows"])
    lens = _spread(n, c["lo"], c["hi"])
    if c["op"] == "plan":
        new = _spread(n, 1, c["new"])
        new[:c["prompt"]] *= 64
        return lens, new
    return lens, _spread(n, 1, c["new"]) if c["ragged"] else torch.full((n,), c["new"])


def _quantised(x):
    """E4M3 codes of vectors and their scales, largest magnitude / 448."""
    scale = x.abs().amax(-1) / 448.0
    codes = torch.where(scale[..., None] > 0, x / scale[..., None], x).to(F8)
    return codes, scale


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    cpu = torch.Generator().manual_seed(seed * 104729 + 31)
    lens, new = _lens_new(c)
    order = torch.randperm(c["requests"], generator=cpu)
    lens, new = lens[order], new[order]
    R, page = c["requests"], c["page"]
    total = lens + new
    need = (total + page - 1) // page
    width = int(need.max()) + 2
    rows = int(new.sum())
    s = dict(op=c["op"], page=page, lens=lens.to(I32).cuda(), n_new=new.to(I32).cuda())
    if c["op"] == "plan":
        held = (lens + page - 1) // page                 # the pages of what is cached; the rest is free
        pages = int(need.sum()) + 37
        ids = torch.randperm(pages, generator=cpu)
        used = torch.zeros((R, width), dtype=torch.long)
        mine = torch.arange(width)[None, :] < held[:, None]
        used[mine] = ids[:int(held.sum())]
        s["none"] = torch.zeros_like(s["n_new"])
        s["table"], s["held"] = used.to(I32).cuda(), held.to(I32).cuda()
        free = torch.full((pages,), -1, dtype=torch.long)
        left = ids[int(held.sum()):]
        free[:left.numel()] = left
        s["free_ids"] = free.to(I32).cuda()
        s["n_free"] = torch.tensor([left.numel()], dtype=I32, device="cuda")
        spare = 13                                        # rows of the buffers that no request fills
        s["row_start"] = torch.zeros(R + 1, dtype=I32, device="cuda")
        s["slots"] = torch.zeros(rows + spare, dtype=I32, device="cuda")
        s["pos"] = torch.zeros(rows + spare, dtype=I32, device="cuda")
        s["row_start2"] = torch.zeros(R + 1, dtype=I32, device="cuda")
        return s
    H, D = c.get("heads", c.get("kv_heads")), c["dim"]
    pages = int(need.sum()) + 3
    ids = torch.randperm(pages, generator=cpu)
    table = torch.zeros((R, width), dtype=torch.long)
    table[torch.arange(width)[None, :] < need[:, None]] = ids[:int(need.sum())]
    row_start = torch.cat([torch.zeros(1, dtype=torch.long), torch.cumsum(new, 0)])
    s["table"], s["row_start"] = table.to(I32).cuda(), row_start.to(I32).cuda()
    req = torch.repeat_interleave(torch.arange(R), new)
    at = lens[req] + torch.arange(rows) - row_start[req]
    s["eps"], s["base"] = EPS, BASE
    k = _randn(g, pages, page, H, D)
    v = _randn(g, pages, page, H, D)
    if c["fmt"] == "e4m3":
        (k, ks), (v, vs) = _quantised(k), _quantised(v)
        # scales stand [pages][heads][page]
        s["k_scales"], s["v_scales"] = (t.transpose(1, 2).contiguous() for t in (ks, vs))
        s["k"], s["v"] = k.view(torch.uint8), v.view(torch.uint8)
    else:
        s["k"], s["v"], s["k_scales"], s["v_scales"] = k.to(BF16), v.to(BF16), None, None
    del k, v
    s["gamma"] = (1.0 + 0.2 * _randn(g, D)).to(BF16)
    s["pos"] = at.to(I32).cuda()
    if c["op"] == "append":
        slots = table[req, at // page] * page + at % page
        s["slots"] = slots.to(I32).cuda()
        # keys and values as they stand in one projection's output
        kv = _randn(g, rows, 2, H, D).to(BF16)
        s["k_rows"], s["v_rows"] = kv[:, 0], kv[:, 1]
    else:
        s["q"] = _randn(g, rows, c["q_heads"], D).to(BF16)
        s["window"], s["new"], s["tree"] = c["window"], c["new"], None
        if c["tree"]:                                     # every row's ancestors, and its depth
            m = c["new"]
            parent = (torch.rand((R, m), generator=cpu) * torch.arange(m)).long()
            bits, depth = torch.zeros((R, m), dtype=torch.long), torch.zeros((R, m), dtype=torch.long)
            every = torch.arange(R)
            bits[:, 0] = 1
            for j in range(1, m):
                bits[:, j] = bits[every, parent[:, j]] | (1 << j)
                depth[:, j] = depth[every, parent[:, j]] + 1
            j = torch.arange(rows) - row_start[req]
            word = bits[req, j]
            s["tree"] = torch.where(word >= 1 << 31, word - (1 << 32), word).to(I32).cuda()
            s["pos"] = (lens[req] + depth[req, j]).to(I32).cuda()
        s["out"] = torch.empty((rows, c["q_heads"] * D), dtype=BF16, device="cuda")
        s["lse"] = torch.empty((rows, c["q_heads"]), dtype=F32, device="cuda")
    if own:
        from speculative_decoding_draft_row_gb300 import tfd
        s["cache"] = tfd.KvPages(s["k"], s["v"], s["k_scales"], s["v_scales"])
        if c["op"] == "attn":
            s["ws"] = tfd.zeroed_workspace(
                tfd.tfd_paged_attn_workspace(s["new"], c["q_heads"], H, D), "cuda")
    return s


# ---- the operators -----------------------------------------------------------------------------

def _moved(lens, n_new, page, table, held, free, n_free):
    """Each request's pages grown or shrunk to its length: given-back pages go on the free stack (the
    first on top), then missing ones come from its top, both in the order of requests and pages."""
    want = (lens + n_new + page - 1) // page
    at = torch.arange(table.shape[1], device=table.device)[None, :]
    back = (at >= want[:, None]) & (at < held[:, None])
    take = (at >= held[:, None]) & (at < want[:, None])
    stack = torch.arange(free.shape[0], device=free.device)
    top = n_free + back.sum()
    order = torch.cumsum(back.reshape(-1).long(), 0).view(back.shape)
    freed = torch.where(back, top - order, free.shape[0])
    free = torch.cat([free, free[:1]]).scatter(0, freed.reshape(-1), table.reshape(-1))[:stack.numel()]
    order = torch.cumsum(take.reshape(-1).long(), 0).view(take.shape)
    table = torch.where(take, free[(top - order).clamp(min=0)], table)
    return table, want, free, top - take.sum()


def _plain_plan(s):
    lens, new, page = s["lens"].long(), s["n_new"].long(), s["page"]
    table, held, free, n_free = (s[n].long() for n in ("table", "held", "free_ids", "n_free"))
    table, held, free, n_free = _moved(lens, new, page, table, held, free, n_free)
    row_start = torch.cat([torch.zeros_like(lens[:1]), torch.cumsum(new, 0)])
    row = torch.arange(s["slots"].numel(), device=lens.device)
    req = (torch.searchsorted(row_start, row, right=True) - 1).clamp(max=lens.numel() - 1)
    pos = lens[req] + row - row_start[req]
    slot = table[req, (pos // page).clamp(max=table.shape[1] - 1)] * page + pos % page
    inside = row < row_start[-1]
    s["row_start"].copy_(row_start)
    s["slots"].copy_(torch.where(inside, slot, -1))
    s["pos"].copy_(torch.where(inside, pos, -1))
    # all drafts turned down: back to what was cached
    table, held, free, n_free = _moved(lens, torch.zeros_like(new), page, table, held, free, n_free)
    s["table"].copy_(table)
    s["held"].copy_(held)
    s["free_ids"].copy_(free)
    s["n_free"].copy_(n_free)
    s["row_start2"].zero_()


def _plain_rotated(x, gamma, pos, eps, base):
    """RMSNorm of each head with gamma, then RoPE of elements i and i + dim/2; angles in 64 bits."""
    x = x.float()
    half = x.shape[-1] // 2
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.float()
    i = torch.arange(half, device=x.device, dtype=torch.float64)
    turn = pos.double()[:, None] * torch.pow(float(base), -i / half)[None, :]
    cos, sin = torch.cos(turn).float()[:, None, :], torch.sin(turn).float()[:, None, :]
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _plain_append(s):
    slot = s["slots"].long()
    page, at = slot // s["page"], slot % s["page"]
    k = _plain_rotated(s["k_rows"], s["gamma"], s["pos"], s["eps"], s["base"])
    v = s["v_rows"]
    if s["k_scales"] is None:
        s["k"][page, at] = k.to(BF16)
        s["v"][page, at] = v
        return
    (k, ks), (v, vs) = _quantised(k), _quantised(v.float())
    s["k"][page, at], s["v"][page, at] = k.view(torch.uint8), v.view(torch.uint8)
    s["k_scales"][page, :, at], s["v_scales"][page, :, at] = ks, vs


def _plain_paged(pages, scales, table):
    """The table's pages as [requests][heads][keys][dim] in 32 bits."""
    x = pages.view(F8).float() if scales is not None else pages
    if scales is not None:
        x = x * scales.transpose(1, 2)[..., None]
    x = x[table]                                         # [requests][table][page][heads][dim]
    return x.permute(0, 3, 1, 2, 4).reshape(x.shape[0], x.shape[3], -1, x.shape[4]).float()


def _plain_attn(s):
    lens, table = s["lens"].long(), s["table"].long()
    first, m = s["row_start"].long()[:-1], s["new"]
    R, D = lens.numel(), s["k"].shape[-1]
    Hq, H = s["q"].shape[1], s["k"].shape[2]
    n = s["n_new"].long()
    q = _plain_rotated(s["q"], s["gamma"], s["pos"], s["eps"], s["base"])
    j = torch.arange(m, device=lens.device)[None, :]
    row = (first[:, None] + j).clamp(max=q.shape[0] - 1)  # [requests][rows]
    qr = q[row].view(R, m, H, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(R, H, -1, D)
    x = torch.matmul(qr, _plain_paged(s["k"], s["k_scales"], table).transpose(2, 3))
    x = (x / math.sqrt(D)).view(R, H, m, Hq // H, -1)
    key = torch.arange(x.shape[-1], device=lens.device)[None, None, :]
    own_key = key - lens[:, None, None]                  # which of the new rows a key is
    if s["tree"] is None:
        seen = own_key <= j[:, :, None]
        if s["window"] >= 0:
            seen = seen & (own_key >= j[:, :, None] - s["window"])
    else:
        bit = s["tree"].long()[row][:, :, None] >> own_key.clamp(0, 31)
        seen = (own_key < 0) | ((own_key < n[:, None, None]) & ((bit & 1) == 1))
    seen = seen[:, None, :, None, :]
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    v = _plain_paged(s["v"], s["v_scales"], table)
    y = torch.matmul(x.view(R, H, -1, x.shape[-1]), v).view(R, H, m, Hq // H, D)
    y = torch.where(total > 0, y / total, 0.0).permute(0, 2, 1, 3, 4).reshape(R, m, Hq * D)
    lse = (top + torch.log(total))[..., 0].permute(0, 2, 1, 3).reshape(R, m, Hq)
    mine = j < n[:, None]
    s["out"].copy_(y[mine].to(BF16))
    s["lse"].copy_(lse[mine])


def _outputs(s):
    if s["op"] == "plan":
        names = ("row_start", "slots", "pos", "table", "held", "free_ids", "n_free", "row_start2")
        return {n: s[n] for n in names}
    if s["op"] == "attn":
        return {"out": s["out"], "lse": s["lse"]}
    if s["k_scales"] is None:
        return {"k": s["k"], "v": s["v"]}
    return {"k": s["k"].view(F8), "v": s["v"].view(F8), "k_scales": s["k_scales"],
            "v_scales": s["v_scales"]}


def run(state):
    s = state
    if own:
        from speculative_decoding_draft_row_gb300 import tfd
        if s["op"] == "plan":
            # a round's rows, and back to what was cached when all its drafts were turned down
            tfd.tfd_page_plan(s["lens"], s["n_new"], s["page"], s["table"], s["held"], s["free_ids"],
                              s["n_free"], row_start=s["row_start"], slots=s["slots"], pos=s["pos"])
            tfd.tfd_page_plan(s["lens"], s["none"], s["page"], s["table"], s["held"], s["free_ids"],
                              s["n_free"], row_start=s["row_start2"])
        elif s["op"] == "append":
            tfd.tfd_paged_append(s["k_rows"], s["v_rows"], s["slots"], s["pos"], s["cache"],
                                 k_gamma=s["gamma"], eps=s["eps"], rope_base=s["base"])
        else:
            tfd.tfd_paged_attn(s["q"], s["cache"], s["table"], s["lens"], s["row_start"], s["new"],
                               pos=s["pos"], tree=s["tree"], window=s["window"], q_gamma=s["gamma"],
                               eps=s["eps"], rope_base=s["base"], out=s["out"], lse=s["lse"],
                               ws=s["ws"])
    else:
        {"plan": _plain_plan, "append": _plain_append, "attn": _plain_attn}[s["op"]](s)
    return _outputs(s)


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    c = case
    lens, new = _lens_new(c)
    page, rows = c["page"], int(new.sum())
    if c["op"] == "plan":
        moved = int(((lens + new + page - 1) // page - (lens + page - 1) // page).sum())
        # lengths, rows and pages held in and out; a slot and a position a row; the pages that move
        return {"bytes": 2 * c["requests"] * 16 + rows * 8 + moved * 16, "flops": 0}
    D, size = c["dim"], 1 if c["fmt"] == "e4m3" else 2
    if c["op"] == "append":
        e = rows * c["heads"]
        return {"bytes": 2 * e * (D * (2 + size) + (4 if size == 1 else 0)) + rows * 8,
                "flops": 10 * e * D}
    keys = lens + new
    pairs = new * (lens + (new + 1) // 2)
    if c["window"] >= 0:
        keys = torch.minimum(keys, c["window"] + new)
        pairs = torch.minimum(pairs, new * (c["window"] + 1))
    # every visible key and value once, the queries, the outputs
    return {"bytes": int(keys.sum()) * 2 * c["kv_heads"] * (D * size + (4 if size == 1 else 0)) +
            rows * c["q_heads"] * (4 * D + 4),
            "flops": 4 * int(pairs.sum()) * c["q_heads"] * D}


# ---- from the definitions, in 64 bits ------------------------------------------------------------

def _exact_plan(s):
    lens, new, held, page = s["lens"].tolist(), s["n_new"].tolist(), s["held"].tolist(), s["page"]
    table, free = s["table"].cpu().numpy().copy(), s["free_ids"].cpu().numpy().copy()
    stack = free[:int(s["n_free"][0])].tolist()
    start, slots, pos, before = [0], [], [], list(held)
    for r, (a, n) in enumerate(zip(lens, new)):
        while held[r] * page < a + n:
            table[r, held[r]] = stack.pop()
            held[r] += 1
        for i in range(a, a + n):
            slots.append(int(table[r, i // page]) * page + i % page)
            pos.append(i)
        start.append(start[-1] + n)
    # given back in reverse, so that the stack is what it was
    for r in reversed(range(len(lens))):
        while (held[r] - 1) * page >= lens[r]:
            held[r] -= 1
            stack.append(int(table[r, held[r]]))
    assert held == before
    free[:len(stack)] = stack
    pad = [-1] * (s["slots"].numel() - len(slots))
    i4 = np.int32
    return {"row_start": np.array(start, i4), "slots": np.array(slots + pad, i4),
            "pos": np.array(pos + pad, i4), "table": table, "held": np.array(held, i4),
            "free_ids": free, "n_free": np.array([len(stack)], i4),
            "row_start2": np.zeros(len(start), i4)}


def _exact_turned(x, gamma, pos, eps, base):
    x, gamma = x.double(), gamma.double()
    dim = x.shape[-1]
    x = x * gamma * torch.rsqrt(x.square().sum(-1, keepdim=True) / dim + eps)
    pair = torch.arange(dim // 2, device=x.device, dtype=torch.float64)
    angle = torch.outer(pos.double(), base ** (-2.0 * pair / dim))
    z = torch.complex(x[..., :dim // 2], x[..., dim // 2:])
    z = z * torch.polar(torch.ones_like(angle), angle)[:, None, :]
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(s)
    page, eight = case["page"], case["fmt"] == "e4m3"
    if case["op"] == "append":
        new = {"k": _exact_turned(s["k_rows"], s["gamma"], s["pos"], s["eps"], s["base"]),
               "v": s["v_rows"].double()}
        out, slot = {}, s["slots"].long()
        for name, x in new.items():
            pages = (s[name].view(F8) if eight else s[name]).double()
            flat = pages.view(-1, *pages.shape[2:])
            if eight:
                scale = x.abs().max(-1).values / 448
                x = x / scale[..., None]
                scales = s[name + "_scales"].double()
                for h in range(case["heads"]):
                    scales[slot // page, h, slot % page] = scale[:, h]
                out[name + "_scales"] = scales.cpu().numpy()
            flat[slot] = x
            out[name] = pages.cpu().numpy()
        return {n: out[n] for n in ("k", "v", "k_scales", "v_scales") if n in out}
    H, D, group = case["kv_heads"], case["dim"], case["q_heads"] // case["kv_heads"]
    q = _exact_turned(s["q"], s["gamma"], s["pos"], s["eps"], s["base"]) / D ** 0.5
    start = s["row_start"].tolist()
    outs, lses = [], []
    for r, a in enumerate(s["lens"].tolist()):
        lo, hi = start[r], start[r + 1]
        total = a + hi - lo
        ids = s["table"][r, :-(-total // page)].long()
        kv = []
        for name in ("k", "v"):
            x = s[name][ids]
            x = (x.view(F8) if eight else x).double()
            if eight:
                x = x * s[name + "_scales"][ids].double().permute(0, 2, 1).unsqueeze(-1)
            kv.append(x.reshape(-1, H, D)[:total])
        seen = torch.ones((hi - lo, total), dtype=torch.bool)
        if s["tree"] is not None:
            words = s["tree"][lo:hi].tolist()
            seen[:, a:] = torch.tensor([[w >> i & 1 for i in range(hi - lo)] for w in words]).bool()
        else:
            for i in range(hi - lo):
                seen[i, a + i + 1:] = False
                if case["window"] >= 0:
                    seen[i, :max(0, a + i - case["window"])] = False
        bias = torch.zeros(seen.shape, dtype=torch.float64).masked_fill(~seen, -math.inf).cuda()
        x = torch.einsum("ihgd,jhd->hgij", q[lo:hi].view(-1, H, group, D), kv[0]) + bias
        lse = torch.logsumexp(x, -1)
        y = torch.einsum("hgij,jhd->ihgd", torch.exp(x - lse[..., None]), kv[1])
        outs.append(y.reshape(hi - lo, -1))
        lses.append(lse.permute(2, 0, 1).reshape(hi - lo, -1))
    return {"out": torch.cat(outs).cpu().numpy(), "lse": torch.cat(lses).cpu().numpy()}
