"""Drawing tokens from logits with given random numbers, and the rejection accept of such drafts.

Oracle (test infrastructure only; see ``oracle/__init__.py``). Float64, one row at a time.

Readings (the pages take the round's draws as inputs, so these are this library's own):
* order for top-k and top-p: value descending, then (mapped) id ascending; top-p after top-k, on the
  mass that top-k leaves; min_p on the weight relative to the largest;
* a token is the first column, in column order, at which the running kept mass exceeds u * total;
* temperature 0 is top-k 1; NaN and -inf have no mass; +inf logits share it; an empty row gives -1.

``margin`` is how near the row came to another answer: the smallest distance, relative to the total
mass, of u * total to a running mass, and of top_p * total to the running masses around its border.
"""
import numpy as np


def filtered(logits, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, id_map=None):
    """(distribution [n] in float64, margin of the top-p border) of one row; None when empty."""
    x = np.asarray(logits, dtype=np.float64)
    n = x.size
    ids = np.arange(n) if id_map is None else np.asarray(id_map, dtype=np.int64)
    if temperature == 0:
        temperature, top_k = 1.0, 1
    top = np.max(np.where(np.isnan(x), -np.inf, x))
    if top == -np.inf:
        return None, 1.0
    with np.errstate(invalid="ignore"):
        d = np.where(x == top, 0.0, x - top) / float(temperature)
    w = np.where(np.isnan(x), 0.0, np.exp(np.where(np.isnan(d), -np.inf, d)))
    order = np.lexsort((ids, np.where(np.isnan(x), np.inf, -x)))
    if top_k > 0:
        order = order[:top_k]
    margin = 1.0
    if top_p < 1:
        incl = np.cumsum(w[order])
        goal = max(float(top_p), 0.0) * incl[-1]
        before = incl - w[order]
        keep = before < goal
        keep[0] = True
        last = int(np.flatnonzero(keep)[-1])
        near = [abs(incl[last] - goal)] + ([abs(before[last] - goal)] if last > 0 else [])
        margin = min(near) / incl[-1]
        order = order[keep]
    order = order[w[order] >= min(max(float(min_p), 0.0), 1.0)]
    full = np.zeros(n)
    full[order] = w[order]
    return full / full.sum(), margin


def draw(dist, u):
    """(column, margin) of the inverse of a distribution's running sum at u."""
    cols = np.flatnonzero(dist)
    c = np.cumsum(dist[cols])
    j = min(int(np.searchsorted(c, float(u) * c[-1], side="right")), cols.size - 1)
    goal = float(u) * c[-1]
    near = [abs(c[j] - goal)] + ([abs(c[j - 1] - goal)] if j > 0 else [])
    return int(cols[j]), min(near) / c[-1]


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, id_map=None):
    """(ids int32 [R], probs float64 [R][n], margin float64 [R]) of the rows of ``logits``."""
    lg = np.atleast_2d(np.asarray(logits, dtype=np.float64))
    R, n = lg.shape

    def at(v, r, default):
        return default if v is None else v[r]

    ids, probs, margins = np.full(R, -1, np.int32), np.zeros((R, n)), np.ones(R)
    for r in range(R):
        t, k = float(at(temperature, r, 1.0)), int(at(top_k, r, 0))
        p, mp, ur = float(at(top_p, r, 1.0)), float(at(min_p, r, 0.0)), float(u[r])
        if not (0 <= t < np.inf) or np.isnan(p) or np.isnan(mp) or not 0 <= ur < 1:
            continue
        dist, m1 = filtered(lg[r], t, k, p, mp, id_map)
        if dist is None:
            continue
        j, m2 = draw(dist, ur)
        ids[r] = j if id_map is None else int(id_map[j])
        probs[r], margins[r] = dist, min(m1, m2)
    return ids, probs, margins


def accept_sampled(p, q, drafts, n_asked, u, u_next, q_map=None):
    """(n_kept int32 [S], next_ids int32 [S], next_prob float64 [S], margin [S], bad [S])."""
    p, q = np.asarray(p, dtype=np.float64), np.asarray(q, dtype=np.float64)
    S, W = np.asarray(drafts).shape
    n = p.shape[2]
    kept, nxt = np.zeros(S, np.int32), np.full(S, -1, np.int32)
    prob, margin, bad = np.zeros(S), np.ones(S), np.zeros(S, bool)

    def clean(v):
        return np.clip(np.where(np.isnan(v), 0.0, v), 0.0, 1.0)

    def q_row(s, t):
        if q_map is None:
            return q[s, t]
        m = np.asarray(q_map, dtype=np.int64)
        ok = (m >= 0) & (m < q.shape[2])
        return np.where(ok, q[s, t][np.where(ok, m, 0)], 0.0)

    for s in range(S):
        na = int(n_asked[s])
        if na < 0 or na > W or not 0 <= u_next[s] < 1 or \
                any(not 0 <= int(d) < n for d in drafts[s][:na]) or \
                any(not 0 <= float(v) < 1 for v in u[s][:na]):
            bad[s] = True
            continue
        m = 0
        while m < na:
            d = int(drafts[s][m])
            if not float(u[s][m]) * q_row(s, m)[d] < p[s, m, d]:
                break
            m += 1
        kept[s] = m
        pr = clean(p[s, m])
        r = np.maximum(pr - clean(q_row(s, m)), 0.0) if m < na else pr
        if not r.any():
            r = pr
        if not r.any():
            continue
        nxt[s], margin[s] = draw(r / r.sum(), u_next[s])
        prob[s] = r[nxt[s]] / r.sum()
    return kept, nxt, prob, margin, bad
