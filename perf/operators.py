"""The operators of sampled, per-request drafting, as they are measured: drawing tokens from given
random numbers, the rejection accept of sampled drafts, and low-rank adapters of many requests.

``run`` computes each operator in its plain form (elementary torch operations) or, where ``own`` is
true, by the library's call. The vocabulary (163840 and the 4096 of the smallest workload), the
hidden size (4096), the w2 input (11008), the 4 streams of 5 drafts and the 1-32-row windows are
those of the draft step; the other sizes are generic."""
import math

import numpy as np
import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16


# ---- cases -----------------------------------------------------------------------------------

def _sample(rows, n, dtype="f32", filters="mixed", probs=False, masked=False, **kw):
    return dict(op="sample", rows=rows, n=n, dtype=dtype, filters=filters, probs=probs,
                masked=masked, **kw)


def _accept(streams, win, n, **kw):
    return dict(op="accept", streams=streams, win=win, n=n, **kw)


def _lora(rows, k, n, rank, adapters, dtype="bf16", none=False, **kw):
    return dict(op="lora", rows=rows, k=k, n=n, rank=rank, adapters=adapters, dtype=dtype,
                none=none, **kw)


def listed():
    return [
        # one request over the smallest workload's vocabulary: latency is all there is
        _sample(1, 4096, filters="all", name="sample_one"),
        # one draft step of four streams: drafts drawn, their distributions kept for the accept
        _sample(4, 163840, filters="top_p", probs=True, name="sample_draft_step"),
        # a 16-row decode window with bf16 logits, every request with settings of its own
        _sample(16, 163840, dtype="bf16", filters="mixed", name="sample_window_bf16"),
        # temperature alone over an odd vocabulary with banned tokens (a grammar): all of it counts
        _sample(33, 50021, filters="none", masked=True, name="sample_odd_masked"),
        # the target's distributions of a verify round: 16 streams of 5 drafts and the row after
        _sample(96, 163840, filters="mixed", probs=True, name="sample_verify_rows"),
        # one request, one draft, the smallest vocabulary
        _accept(1, 1, 4096, name="accept_one"),
        # a round of the measured pass: four streams of five drafts
        _accept(4, 5, 163840, name="accept_pass"),
        # a large batch's round
        _accept(48, 5, 163840, name="accept_batch"),
        # one token's output projection with one request's adapter
        _lora(1, 4096, 4096, 16, 1, name="lora_one"),
        # a decode window beside w2: 16 rows of 8 requests' adapters, some rows without one
        _lora(16, 11008, 4096, 32, 8, none=True, name="lora_window_w2"),
        # the vocabulary head's logits of a 16-row window, four adapters
        _lora(16, 4096, 163840, 16, 4, dtype="f32", name="lora_head"),
        # prompt chunks of six requests, an odd number of rows
        _lora(4099, 4096, 4096, 64, 6, name="lora_prompt"),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sample", "accept", "lora"])
    if op == "sample":
        n = _log_uniform(rng, 1000, 200000)
        rows = _log_uniform(rng, 1, max(1, min(256, 15_000_000 // n)))
        return _sample(rows, n, rng.choice(["f32", "bf16"]),
                       rng.choice(["none", "top_k", "top_p", "min_p", "all", "mixed"]),
                       rng.random() < 0.5, rng.random() < 0.3)
    if op == "accept":
        n = _log_uniform(rng, 1000, 200000)
        win = rng.randint(1, 8)
        streams = _log_uniform(rng, 1, max(1, min(64, 40_000_000 // (n * (win + 1)))))
        return _accept(streams, win, n)
    rank = rng.choice([8, 16, 24, 32, 64, 128])
    k = 8 * _log_uniform(rng, 32, 1376)
    if rng.random() < 0.25:                              # beside a vocabulary head
        n, rows = _log_uniform(rng, 20000, 163840), rng.randint(1, 32)
        return _lora(rows, k, n, min(rank, 32), rng.randint(1, 4), rng.choice(["f32", "bf16"]),
                     rng.random() < 0.3)
    n = _log_uniform(rng, 256, 11008)
    rows = _log_uniform(rng, 1, max(1, min(4096, 16_000_000 // (k + n))))
    return _lora(rows, k, n, rank, min(rows, rng.randint(1, 12)), rng.choice(["f32", "bf16"]),
                 rng.random() < 0.3)


# ---- inputs ----------------------------------------------------------------------------------

def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _pick(g, values, rows, dtype):
    t = torch.tensor(values, device="cuda", dtype=dtype)
    return t[torch.randint(0, len(values), (rows,), generator=g, device="cuda")]


def _logits(g, rows, n):
    """Logits as a trained head gives them: a wide bulk and a handful of likely tokens a row."""
    x = 2.5 * _randn(g, rows, n)
    m = min(n, 12)
    at = torch.randint(0, n, (rows, m), generator=g, device="cuda")
    return x.scatter_add_(1, at, 9.0 * _rand(g, rows, m))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    s = dict(op=case["op"])
    if case["op"] == "sample":
        rows, n, f = case["rows"], case["n"], case["filters"]
        x = _logits(g, rows, n)
        if case["masked"]:
            x[_rand(g, rows, n) < 0.1] = -math.inf
        s["logits"] = x.to(BF16) if case["dtype"] == "bf16" else x
        s["u"] = _rand(g, rows)
        s["temperature"] = _pick(g, [0.6, 0.8, 1.0, 1.2] + ([0.0] if f == "mixed" else []), rows,
                                 F32)
        s["top_k"] = _pick(g, [20, 50, 200] + ([0] if f == "mixed" else []), rows, torch.int32) \
            if f in ("top_k", "all", "mixed") else None
        s["top_p"] = _pick(g, [0.8, 0.9, 0.95] + ([1.0] if f == "mixed" else []), rows, F32) \
            if f in ("top_p", "all", "mixed") else None
        s["min_p"] = _pick(g, [0.02, 0.05] + ([0.0] if f == "mixed" else []), rows, F32) \
            if f in ("min_p", "all", "mixed") else None
        s["ids"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        s["prob"] = torch.empty(rows, dtype=F32, device="cuda")
        s["probs"] = torch.empty((rows, n), dtype=F32, device="cuda") if case["probs"] else None
    elif case["op"] == "accept":
        S, W, n = case["streams"], case["win"], case["n"]
        lp = _logits(g, S * (W + 1), n)
        p = torch.softmax(lp, 1).view(S, W + 1, n)
        lq = lp.view(S, W + 1, n)[:, :W] + 0.7 * _randn(g, S, W, n)
        q = torch.softmax(lq, 2)
        c = torch.cumsum(q.double(), 2)
        at = (c <= _rand(g, S, W, 1).double() * c[:, :, -1:]).sum(2).clamp(max=n - 1)
        s["p"], s["q"], s["drafts"] = p, q.contiguous(), at.to(torch.int32)
        s["n_asked"] = torch.full((S,), W, dtype=torch.int32, device="cuda")
        s["u"], s["u_next"] = _rand(g, S, W), _rand(g, S)
        s["n_kept"] = torch.empty(S, dtype=torch.int32, device="cuda")
        s["next_ids"] = torch.empty(S, dtype=torch.int32, device="cuda")
        s["next_prob"] = torch.empty(S, dtype=F32, device="cuda")
    else:
        R, k, n, rank, na = (case[v] for v in ("rows", "k", "n", "rank", "adapters"))
        out = F32 if case["dtype"] == "f32" else BF16
        s["x"] = _randn(g, R, k).to(BF16)
        s["a"] = (_randn(g, na, rank, k) / math.sqrt(k)).to(BF16)
        s["b"] = (0.3 * _randn(g, na, n, rank)).to(BF16)
        s["scales"] = 0.5 + _rand(g, na)
        s["base"] = (2.5 * _randn(g, R, n)).to(out)
        s["y"] = torch.empty_like(s["base"])
        if R <= 64:                                      # decode rows: requests in any order
            ids = torch.arange(R, device="cuda") % na
            ids = ids[torch.randperm(R, generator=g, device="cuda")]
            if case["none"]:
                ids[::5] = -1
        else:                                            # prompt chunks: rows of a request adjoin
            cut = torch.sort(torch.randint(1, R, (na - 1,), generator=g, device="cuda"))[0]
            ids = (torch.arange(R, device="cuda")[:, None] >= cut[None, :]).sum(1)
            if case["none"]:
                ids[ids == na - 1] = -1
        s["adapter_ids"] = ids.to(torch.int32)
    return s


# ---- the operators -----------------------------------------------------------------------------

def _plain_sample(s):
    # 64 bits: a running mass next to u * total or to top_p * total decides a token
    x, u = s["logits"].float(), s["u"].double()[:, None]
    rows, n = x.shape
    t = s["temperature"].double()[:, None]
    greedy = t == 0
    k = s["top_k"].long()[:, None] if s["top_k"] is not None else torch.zeros_like(t).long()
    k = torch.where(greedy, 1, torch.where(k <= 0, n, k))
    top_p = s["top_p"].double()[:, None] if s["top_p"] is not None else torch.ones_like(t)
    min_p = s["min_p"].double()[:, None] if s["min_p"] is not None else torch.zeros_like(t)
    v, at = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((v.double() - v[:, :1].double()) / torch.where(greedy, 1.0, t))
    rank = torch.arange(n, device=x.device)[None, :]
    w = torch.where(rank < k, w, 0.0)
    before = torch.cumsum(w, 1) - w
    keep = (rank == 0) | (top_p >= 1) | (before < top_p * w.sum(1, keepdim=True))
    w = torch.where(keep & (w >= min_p), w, 0.0)
    w = torch.zeros_like(w).scatter_(1, at, w)
    c = torch.cumsum(w, 1)
    total = c[:, -1:]
    pick = (c <= u * total).sum(1, keepdim=True)
    out = {"ids": pick[:, 0].to(torch.int32), "prob": (w.gather(1, pick) / total)[:, 0].float()}
    if s["probs"] is not None:
        out["probs"] = (w / total).float()
    return out


def _plain_accept(s):
    # 64 bits, for the same reason
    p, q, d = s["p"], s["q"], s["drafts"].long()[:, :, None]
    S, W, n = q.shape
    pd, qd = p[:, :W].gather(2, d)[:, :, 0].double(), q.gather(2, d)[:, :, 0].double()
    asked = s["n_asked"].long()
    ok = (s["u"].double() * qd < pd) & (torch.arange(W, device=p.device)[None, :] < asked[:, None])
    kept = torch.cumprod(ok.long(), 1).sum(1)
    at = torch.arange(S, device=p.device)
    pr = p[at, kept].double()
    r = (pr - q[at, kept.clamp(max=W - 1)].double()).clamp(min=0)
    r = torch.where((kept < asked)[:, None], r, pr)
    r = torch.where(r.sum(1, keepdim=True) > 0, r, pr)
    c = torch.cumsum(r, 1)
    total = c[:, -1:]
    pick = (c <= s["u_next"].double()[:, None] * total).sum(1, keepdim=True)
    return {"n_kept": kept.to(torch.int32), "next_ids": pick[:, 0].to(torch.int32),
            "next_prob": (r.gather(1, pick) / total)[:, 0].float()}


def _plain_lora(s):
    # every adapter's low-rank rows at once, the rows of other requests' adapters set to zero
    na, rank, k = s["a"].shape
    n = s["b"].shape[1]
    ids = s["adapter_ids"].long()
    mine = (ids[:, None] == torch.arange(na, device=ids.device)[None, :]).float() * s["scales"]
    h = (s["x"].float() @ s["a"].float().view(na * rank, k).T).view(-1, na, rank)
    h = (h * mine[:, :, None]).view(-1, na * rank)
    b = s["b"].float().permute(0, 2, 1).reshape(na * rank, n)
    return (s["base"].float() + h @ b).to(s["y"].dtype)


def run(state):
    s = state
    if own:
        from speculative_decoding_draft_row_gb300 import tfd
        if s["op"] == "sample":
            ids, prob, probs = tfd.tfd_sample(
                s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                top_p=s["top_p"], min_p=s["min_p"], ids=s["ids"], prob=s["prob"],
                probs=s["probs"])
            out = {"ids": ids, "prob": prob}
            if probs is not None:
                out["probs"] = probs
            return out
        if s["op"] == "accept":
            n_kept, next_ids, next_prob = tfd.tfd_accept_sampled(
                s["p"], s["q"], s["drafts"], s["n_asked"], s["u"], s["u_next"],
                n_kept=s["n_kept"], next_ids=s["next_ids"], next_prob=s["next_prob"])
            return {"n_kept": n_kept, "next_ids": next_ids, "next_prob": next_prob}
        return tfd.tfd_lora(s["x"], s["a"], s["b"], s["adapter_ids"], base=s["base"], y=s["y"],
                            scales=s["scales"])
    return {"sample": _plain_sample, "accept": _plain_accept, "lora": _plain_lora}[s["op"]](s)


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    if case["op"] == "sample":
        size = 4 if case["dtype"] == "f32" else 2
        e = case["rows"] * case["n"]
        # logits read, the distribution written where it is asked for; a weight and a sum an element
        return {"bytes": e * (size + (4 if case["probs"] else 0)) + case["rows"] * 28,
                "flops": 4 * e}
    if case["op"] == "accept":
        # the deciding row of p and, where a draft is turned down (most rounds), that row of q
        e = case["streams"] * case["n"]
        return {"bytes": 8 * e + case["streams"] * (case["win"] * 16 + 24), "flops": 3 * e}
    R, k, n, rank, na = (case[v] for v in ("rows", "k", "n", "rank", "adapters"))
    size = 4 if case["dtype"] == "f32" else 2
    return {"bytes": min(R, na) * (k + n) * rank * 2 + R * k * 2 + 2 * R * n * size + 4 * R,
            "flops": 2 * R * rank * (k + n)}


# ---- from the definitions, in 64 bits ------------------------------------------------------------

def _exact_sample_row(x, t, k, p, mp, u):
    n = x.size
    if t == 0:
        t, k = 1.0, 1
    order = np.lexsort((np.arange(n), -x))
    if k > 0:
        order = order[:k]
    w = np.exp((x[order] - x[order[0]]) / t)
    if p < 1:
        incl = np.cumsum(w)
        cut = int(np.searchsorted(incl, p * incl[-1], side="left")) + 1
        order, w = order[:cut], w[:cut]
    few = w >= mp
    order, w = order[few], w[few]
    full = np.zeros(n)
    full[order] = w / w.sum()
    cols = np.sort(order)
    c = np.cumsum(full[cols])
    j = cols[min(int(np.searchsorted(c, u * c[-1], side="right")), cols.size - 1)]
    return j, full


def exact(case, seed):
    s = prepare(case, seed)

    def h(name):
        return None if s.get(name) is None else s[name].double().cpu().numpy()

    if case["op"] == "sample":
        x, rows = h("logits"), case["rows"]
        t, u = h("temperature"), h("u")
        k = h("top_k") if s["top_k"] is not None else np.zeros(rows)
        p = h("top_p") if s["top_p"] is not None else np.ones(rows)
        mp = h("min_p") if s["min_p"] is not None else np.zeros(rows)
        got = [_exact_sample_row(x[r], t[r], int(k[r]), p[r], mp[r], u[r]) for r in range(rows)]
        out = {"ids": np.array([j for j, _ in got], np.int32),
               "prob": np.array([f[j] for j, f in got])}
        if case["probs"]:
            out["probs"] = np.stack([f for _, f in got])
        return out
    if case["op"] == "accept":
        p, q, d = h("p"), h("q"), s["drafts"].cpu().numpy()
        u, un = h("u"), h("u_next")
        S, W = d.shape
        kept, nxt, prob = [], [], []
        for i in range(S):
            m = 0
            while m < W and u[i, m] * q[i, m, d[i, m]] < p[i, m, d[i, m]]:
                m += 1
            r = np.maximum(p[i, m] - q[i, m], 0) if m < W else p[i, m]
            if not r.any():
                r = p[i, m]
            c = np.cumsum(r)
            j = int(np.searchsorted(c, un[i] * c[-1], side="right"))
            kept.append(m)
            nxt.append(j)
            prob.append(r[j] / c[-1])
        return {"n_kept": np.array(kept, np.int32), "next_ids": np.array(nxt, np.int32),
                "next_prob": np.array(prob)}
    x, a, b, sc, y = h("x"), h("a"), h("b"), h("scales"), h("base")
    ids = s["adapter_ids"].cpu().numpy()
    for i in range(case["adapters"]):
        mine = np.flatnonzero(ids == i)
        y[mine] += sc[i] * ((x[mine] @ a[i].T) @ b[i].T)
    return y
