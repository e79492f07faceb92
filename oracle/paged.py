"""A paged key-value cache: page tables of a round, the append of new rows, attention over the pages.

Oracle (test infrastructure only; see ``oracle/__init__.py``), in float64 and plain loops. The pages keep
a ring a stream (``attn``, ``layer.absorb``); the paged cache is the library's own, with the same qk_norm,
RoPE and rounding of keys. Readings:
* pages given back go on the free stack in the order of requests and pages, the first ending on top (ids
  that are no pages are left out); then missing pages come from its top in the same order;
* a row sees the cached tokens and the new ones up to itself (or those its tree word names), from its
  own depth minus the window on; a row that sees nothing gives zeros and a log-sum of -inf;
* E4M3 keys are quantised from the exact key, by the row rule (largest magnitude / 448).
"""
import numpy as np

from .attn import rmsnorm, rope


def plan(lens, n_new, page_size, table, held, free_ids, n_free, rows):
    """Returns dict(table, held, free_ids, n_free, row_start, slots, pos, bad)."""
    table, held, free = np.array(table), np.array(held), np.array(free_ids)
    R, max_pages = table.shape
    pages, bad = len(free), False
    want, wrong = [], []
    for r in range(R):
        ln, n, hd = int(lens[r]), int(n_new[r]), int(held[r])
        need = -(-(ln + n) // page_size)
        wrong.append(ln < 0 or n < 0 or not 0 <= hd <= max_pages or need > max_pages)
        want.append(hd if wrong[r] else need)
        bad |= wrong[r]
    stack = free[:max(0, int(n_free))].tolist()
    back = [(r, p) for r in range(R) for p in range(want[r], int(held[r]))]
    broken = not 0 <= int(n_free) <= pages or int(n_free) + len(back) > pages
    if broken:
        bad, stack = True, []
    else:
        given = [int(table[r, p]) for r, p in back]
        bad |= any(not 0 <= i < pages for i in given)
        stack += [i for i in given[::-1] if 0 <= i < pages]  # the first given back ends on top
        free[:len(stack)] = stack
        for r in range(R):
            held[r] = min(held[r], want[r])
    left, counted = len(stack), 0
    for r in range(R):
        missing = max(0, want[r] - int(held[r]))
        counted += missing
        if not missing:
            continue
        if counted > len(stack):
            table[r, held[r]:want[r]] = -1
            bad = wrong[r] = True
        else:
            for p in range(held[r], want[r]):
                left -= 1
                table[r, p] = stack[left]
            held[r] = want[r]
    start = np.concatenate([[0], np.cumsum([max(0, int(n)) for n in n_new])])
    slots, pos = np.full(rows, -1), np.full(rows, -1)
    bad |= 0 < rows < start[-1]
    for r in range(R):
        for j in range(max(0, int(n_new[r]))):
            i, p = int(start[r]) + j, int(lens[r]) + j
            if wrong[r] or i >= rows:
                continue
            page = int(table[r, p // page_size])
            pos[i] = p
            if 0 <= page < pages:
                slots[i] = page * page_size + p % page_size
            else:
                bad = True
    return dict(table=table, held=held, free_ids=free, n_free=int(n_free) if broken else left,
                row_start=start, slots=slots, pos=pos, bad=bool(bad))


def turned(x, pos, gamma=None, norm=True, rotate=True, eps=1e-6, base=10000.0):
    """(x [rows][heads][dim] after RMSNorm with gamma and RoPE at pos [rows], and the magnitude of each
    element's rotation pair before the rotation, which bounds its fp32 error)."""
    x = np.asarray(x, dtype=np.float64)
    rows, heads, dim = x.shape
    g = np.ones(dim) if gamma is None else np.asarray(gamma, dtype=np.float64)
    out, pair = np.empty_like(x), np.empty_like(x)
    for i in range(rows):
        for h in range(heads):
            v = rmsnorm(x[i, h], g, eps) if norm else x[i, h]
            pair[i, h] = np.tile(np.hypot(v[:dim // 2], v[dim // 2:]), 2) if rotate else np.abs(v)
            out[i, h] = rope(v, int(pos[i]), base) if rotate else v
    return out, pair


def attend(q, k, v, length, tree=None, window=-1, scale=None, mag=None):
    """One request's attention.

    Args:
      q: [n][q_heads][dim] as it enters the scores; k, v: [tokens][heads][dim], tokens = length + n.
      tree: [n] words or None (causal); window: -1 or the tokens seen before the own one.
      mag: magnitudes of q's elements for the error terms (|q|; before a rotation, their pairs').
    Returns (out [n][q_heads][dim], lse [n][q_heads], terms): terms has, per output, ``abs_out`` =
    sum_j p_j |v_j|, and per row and head ``a`` = the largest A_j = scale sum_e mag_e |k_je| over the seen
    tokens, ``a_most`` the same with every mag_e the largest, ``dev`` [n][q_heads][dim] = sum_j p_j |v_j - out| and ``dev_a`` the same weighted with A_j + max A.
    """
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    n, hq, dim = q.shape
    tokens, heads = k.shape[0], k.shape[1]
    assert tokens == length + n
    scale = 1.0 / np.sqrt(dim) if scale is None else scale
    mag = np.abs(q) if mag is None else mag
    words = None if tree is None else [int(w) & ((1 << n) - 1) for w in tree]
    depth = [length + (j if tree is None else bin(words[j]).count("1") - 1) for j in range(n)]
    out, lse = np.zeros(q.shape), np.full((n, hq), -np.inf)
    terms = {name: np.zeros(q.shape) for name in ("abs_out", "dev", "dev_a")}
    terms["a"], terms["a_most"] = np.zeros((n, hq)), np.zeros((n, hq))
    for j in range(n):
        sees = []
        for t in range(tokens):
            own = t - length
            there = own < 0 or (own <= j if tree is None else words[j] >> own & 1)
            at = t if own < 0 else depth[own]
            if there and (window < 0 or at >= depth[j] - window):
                sees.append(t)
        if not sees:
            continue
        for i in range(hq):
            ks, vs = k[sees, i // (hq // heads)], v[sees, i // (hq // heads)]
            x = scale * (ks @ q[j, i])
            top = x.max()
            w = np.exp(x - top)
            lse[j, i] = top + np.log(w.sum())
            w /= w.sum()
            y = w @ vs
            out[j, i] = y
            a = scale * (np.abs(ks) @ mag[j, i])
            terms["a"][j, i] = a.max()
            terms["a_most"][j, i] = scale * mag[j, i].max() * np.abs(ks).sum(1).max()
            terms["abs_out"][j, i] = w @ np.abs(vs)
            terms["dev"][j, i] = w @ np.abs(vs - y)
            terms["dev_a"][j, i] = (w * (a + a.max())) @ np.abs(vs - y)
    return out, lse, terms
