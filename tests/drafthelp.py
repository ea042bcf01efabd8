"""Plain 64-bit forms of the operators of include/pi_draft.h for the tests: numpy
loops written from the definitions, none of the library's code."""
from __future__ import annotations

import math

import numpy as np


def path_of(parent, i):
    """The drafts from the root of draft i's tree down to it."""
    path = [i]
    while parent[path[0]] >= 0:
        path.insert(0, parent[path[0]])
    return path


def visible(base, parent, i, window, sinks, hidden=()):
    """Token numbers that draft i sees; `hidden` ones left out."""
    path = path_of(parent, i)
    here = base + len(path) - 1
    at = [(t, t) for t in range(base)] + [(base + j, base + d) for d, j in enumerate(path)]
    return [t for t, p in at
            if (window == 0 or p > here - window or p < sinks) and t not in hidden]


def attention(q, k, v, seen, scale):
    """q [G][D], k, v [tokens][D] float64; (y [G][D], lse [G], the largest |q| . |k| of a seen
    token per head, the largest |v|).  Infinite operands by the definition."""
    G, D = q.shape
    if not seen:
        return np.zeros((G, D)), np.full(G, -np.inf), np.zeros(G), 0.0
    k, v = k[seen], v[seen]
    with np.errstate(invalid="ignore", over="ignore"):
        a = scale * (q @ k.T)
        m = a.max(1, keepdims=True)
        p = np.exp(a - np.where(np.isneginf(m), 0.0, m))
        l = p.sum(1, keepdims=True)
        y = (p @ v) / np.where(l == 0, 1.0, l)
        lse = (m + np.log(l))[:, 0]
        mag = (np.abs(q) @ np.abs(k).T).max(1)
    return y, lse, mag, np.abs(v).max()


def accept(parent, tokens, choice):
    """Drafts taken of one slot, and the token chosen at the last (lists of count entries)."""
    if not len(tokens):
        return [], -1
    path = [0]
    while True:
        c = choice[path[-1]]
        fits = [i for i in range(len(tokens)) if parent[i] == path[-1] and tokens[i] == c and c >= 0]
        if not fits:
            return path, c
        path.append(fits[0])


def sample_row(x, temperature, top_k, top_p, min_p, u):
    """(token, logprob, margin) of one row; margin: how far the draw and the ends of the kept
    part are from where they would change, relative to the sums they are compared with."""
    x = np.asarray(x, np.float64)
    if np.isnan(x).any() or np.isposinf(x).any() or np.isneginf(x).all():
        return -1, math.nan, 1.0
    if not (0 <= temperature < math.inf and 0 <= u < 1 and top_p >= 0 and 0 <= min_p <= 1):
        return -1, math.nan, 1.0
    order = sorted(range(len(x)), key=lambda i: (-x[i], i))
    if temperature == 0:
        return order[0], 0.0, 1.0
    with np.errstate(under="ignore"):
        w = [math.exp((x[i] - x[order[0]]) / temperature) if x[i] > -math.inf else 0.0 for i in order]
    n = sum(1 for v in w if v > 0 and v >= min_p)
    margin = min([1.0] + [abs(v / min_p - 1) for v in w if v > 0 and min_p > 0 and min_p < 1])
    if top_k > 0:
        n = min(n, top_k)
    sums = [0.0]
    for v in w[:n]:
        sums.append(sums[-1] + v)
    if top_p < 1:
        goal = top_p * sums[n]
        m = next(i for i in range(1, n + 1) if sums[i] >= goal)
        margin = min(margin, min(abs(s - goal) for s in sums[max(m - 1, 1):m + 1]) / sums[n])
        n = m
    goal = u * sums[n]
    at = next(i for i in range(n) if sums[i + 1] > goal)
    near = [sums[i] for i in (at, at + 1) if 0 < i < n]
    margin = min([margin] + [abs(s - goal) / sums[n] for s in near])
    return order[at], math.log(w[at] / sums[n]), margin
