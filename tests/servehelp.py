"""Plain 64-bit forms of the serving operators (include/pi_serve.h) for the
tests: numpy loops written from the definitions, none of the library's code."""
from __future__ import annotations

import numpy as np


def attention(q, k, v, n, scale, window, sinks, hidden=()):
    """One slot and one kv head: q [G][D], k, v [>= n][D] float64 rows by
    position.  Returns (y [G][D], lse [G], the largest |q| . |k| of a visible
    token per head)."""
    t = [i for i in range(n)
         if (window == 0 or i >= n - window or i < sinks) and i not in hidden]
    G, D = q.shape
    if not t:
        return np.zeros((G, D)), np.full(G, -np.inf), np.zeros(G)
    k, v = k[t], v[t]
    a = scale * (q @ k.T)
    m = a.max(1, keepdims=True)
    p = np.exp(a - m)
    l = p.sum(1, keepdims=True)
    return (p @ v) / l, (m + np.log(l))[:, 0], (np.abs(q) @ np.abs(k).T).max(1)


def score_row(x, tok, topk):
    """(logprob, entropy, indices, log probabilities) of one row, float64."""
    x = np.asarray(x, np.float64)
    order = sorted(range(len(x)), key=lambda i: (-np.inf if np.isnan(x[i]) else x[i], -i),
                   reverse=True)[:topk]
    if np.isnan(x).any() or np.isposinf(x).any():
        nan = float("nan")
        return (0.0 if tok == -1 else nan), nan, order, [nan] * topk
    m = x.max()
    if m == -np.inf:
        return (0.0 if tok == -1 else -np.inf), 0.0, order, [-np.inf] * topk
    e = np.exp(x - m)
    z = m + np.log(e.sum())
    p = np.exp(x - z)
    ent = float(-(p[p > 0] * (x[p > 0] - z)).sum())
    return (0.0 if tok == -1 else float(x[tok] - z)), ent, order, [float(x[i] - z) for i in order]


def fork(P, pages, max_pages, parent, grow, held, table, length):
    """pi_cache_fork on lists.  Returns a dict of its outputs (pairs a list),
    and whether a capacity error is reported."""
    S = len(parent)
    ref = list(held) if held is not None else [0] * pages
    out = [[-1] * max_pages for _ in range(S)]
    base = [length[p] if p >= 0 else 0 for p in parent]
    want = [max(0, b + g) for b, g in zip(base, grow)]
    short = any(w > max_pages * P for w in want)
    want = [min(w, max_pages * P) for w in want]
    keep = [min(b, w) for b, w in zip(base, want)]
    for s in range(S):
        for j in range(keep[s] // P):
            out[s][j] = table[parent[s]][j]
            ref[out[s][j]] += 1
    full = list(ref)
    first, src = [k // P for k in keep], [-1] * S
    for s in range(S):
        if keep[s] % P:
            p = table[parent[s]][keep[s] // P]
            lower = any(keep[u] % P and table[parent[u]][keep[u] // P] == p for u in range(s))
            if full[p] == 0 and not lower:
                out[s][first[s]] = p
                ref[p] = 1
                first[s] += 1
            else:
                src[s] = p
    free = [p for p in range(pages) if ref[p] == 0]
    pairs, new_len = [], list(want)
    for s in range(S):
        for j in range(first[s], -(-want[s] // P)):
            if not free:
                short = True
                new_len[s] = min(new_len[s], j * P)
                break
            p = free.pop(0)
            out[s][j] = p
            ref[p] = 1
            if j == first[s] and src[s] >= 0:
                pairs.append((src[s], p))
    return dict(table=out, len=new_len, ref=ref, pairs=pairs,
                live=sum(r > 0 for r in ref)), short


def compact(P, pages, max_pages, held, table, length):
    """pi_cache_compact on lists."""
    ref = list(held) if held is not None else [0] * pages
    for row, n in zip(table, length):
        for j in range(-(-n // P)):
            ref[row[j]] += 1
    live = [p for p in range(pages) if ref[p] > 0]
    c = len(live)
    holes = [p for p in range(c) if ref[p] == 0]
    movers = [p for p in live if p >= c]
    where = [-1] * pages
    for p in live:
        where[p] = p
    for p, to in zip(movers, holes):
        where[p] = to
    new_ref = [0] * pages
    for p in live:
        new_ref[where[p]] = ref[p]
    out = [[where[row[j]] if j < -(-n // P) else -1 for j in range(max_pages)]
           for row, n in zip(table, length)]
    return dict(table=out, ref=new_ref, map=where, pairs=list(zip(movers, holes)), live=c)
