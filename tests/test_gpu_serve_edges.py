"""The serving operators at operands and sizes where 16-bit parts, split sums
or 32-bit counts could fail, against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import activation_sparse_decode_rank_gb300 as pi
from test_gpu_serve import DEV, TD, U, Cache, i32, new_status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    pi.build()


# ------------------------------------------------------------------ page numbers
@pytest.mark.parametrize("P", [16, 8, 5])
@pytest.mark.parametrize("bad", [-2, -3, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("append", [False, True])
def test_attention_reports_every_bad_page_number(P, bad, append):
    # a page in the middle, the first one, the new token's
    for s, j in ((0, 40 // P), (1, 0), (2, 44 // P)):
        c = Cache("f16", 8, 2, 64, P, [100, 60, 45], append=append)
        tab = c.np_table.copy()
        tab[s, j] = bad
        y, lse = c.run(table=i32(tab))
        c.check(y, lse, {s: set(range(j * P, j * P + P))})
        assert int(c.status[0]) == pi.PI_ERR_INDEX
        if append and s == 2:  # not stored anywhere
            pg = int(c.np_table[s, j])
            assert torch.isnan(c.pool[0, pg, :, :, 44 % P]).all()


# ------------------------------------------------------------------ large scores
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("qscale", [1e7, 1e8, 1e12, 1e20])
@pytest.mark.parametrize("shape,lens", [((8, 2, 128, 16), [1, 40, 300, 2]), ((4, 1, 64, 5), [70, 900]),
                                        ((16, 2, 256, 8), [7001, 33])])
def test_attention_of_large_finite_scores(dtype, sign, qscale, shape, lens):
    # Scores are off by da = scale |q|.|k| (2^-21 + D u); where the largest lies
    # more than 2 da + 40 above the second, the others weigh under e^-40 2^13
    # together, and y is the largest one's value (kept to 22 bits), lse its score.
    c = Cache(dtype, *shape, lens, qscale=qscale)
    c.scale *= sign
    y, lse = c.run()
    torch.cuda.synchronize()
    assert torch.isfinite(y).all() and torch.isfinite(lse[:-1]).all()
    y, lse = y.double().cpu().numpy(), lse.double().cpu().numpy()
    seen, G = 0, c.heads // c.kv
    for s, n in enumerate(lens):
        for h in range(c.heads):
            q, k = c.q[s, h].astype(np.float64), c.rows[0, s, :n, h // G]
            a = c.scale * (k @ q)
            da = abs(c.scale) * (np.abs(k) @ np.abs(q)).max() * (2.0 ** -21 + c.D * U)
            top = int(a.argmax())
            if n > 1 and a[top] - np.partition(a, -2)[-2] <= 2 * da + 40:
                continue
            seen += 1
            want = c.rows[1, s, top, h // G]
            assert np.abs(y[s, h] - want).max() <= 2.0 ** -20 * np.abs(want).max(), (s, h)
            assert abs(lse[s, h] - a[top]) <= da + 8 * U * abs(a[top]), (s, h)
    assert seen >= len(lens) * c.heads // 2


# ------------------------------------------------------------------ infinities
def plain_special(q, k, v, n, scale, window, sinks):
    """One slot and kv head as in servehelp.attention, with infinite and NaN
    operands: products and sums follow IEEE rules (0 x infinity is NaN).  A NaN
    or +infinity score makes y and lse NaN; a score of -infinity has weight 0; a
    finite score's weight is positive, however small."""
    G, D = q.shape
    t = [i for i in range(n) if window == 0 or i >= n - window or i < sinks]
    y, lse, mag = np.zeros((G, D)), np.full(G, -np.inf), np.zeros(G)
    if not t:
        return y, lse, mag
    k, v = k[t], v[t]
    with np.errstate(all="ignore"):
        a = scale * (q[:, None, :] * k[None]).sum(-1)
        for g in range(G):
            if np.isnan(a[g]).any() or np.isposinf(a[g]).any():
                y[g], lse[g] = np.nan, np.nan
                continue
            f = np.isfinite(a[g])
            w = np.zeros(len(t))
            if f.any():
                m = a[g][f].max()
                w[f] = np.exp(a[g][f] - m)
                lse[g] = m + np.log(w.sum())
                mag[g] = (np.abs(q[g]) @ np.abs(k[f]).T).max()
            finite = np.isfinite(v)
            y[g] = w @ np.where(finite, v, 0.0) / (w.sum() or 1.0)
            for d in np.flatnonzero(~finite.all(0)):
                odd = np.flatnonzero(~finite[:, d])
                signs = {float(v[i, d]) if f[i] else math.nan for i in odd}
                y[g, d] = signs.pop() if len(signs) == 1 else math.nan
    return y, lse, mag


def poke(c, kind, s, t, h, d, value):
    """Sets element d of the key (0) or value (1) of token t of slot s."""
    new = (c.knew, c.vnew)[kind] if c.append and t == c.lens[s] - 1 else None
    if new is not None:
        new[s, h, d] = value
    else:
        c.pool[c.layer, int(c.np_table[s, t // c.P]), kind, h, t % c.P, d] = value
    c.rows[kind, s, t, h, d] = float(torch.tensor(value).to(TD[c.dtype]))


def check_special(c, y, lse):
    torch.cuda.synchronize()
    y, lse = y.double().cpu().numpy(), lse.double().cpu().numpy()
    G, odd = c.heads // c.kv, 0
    for s, n in enumerate(c.lens):
        for h in range(c.kv):
            r = slice(h * G, (h + 1) * G)
            yo, lo, mag = plain_special(c.q[s, r].astype(np.float64), c.rows[0, s, :, h],
                                        c.rows[1, s, :, h], n, c.scale, c.window, c.sinks)
            e = (abs(c.scale) * mag * (2.0 ** -21 + c.D * U) + 2.0 ** -20 + n * U)[:, None]
            vis = c.rows[1, s, :max(n, 1), h]
            vmax = np.abs(vis[np.isfinite(vis)]).max()
            for got, want, tol in ((y[s, r], yo, 3 * e * vmax),
                                   (lse[s, r], lo, 2 * e[:, 0] + 4 * U * np.abs(lo))):
                f = np.isfinite(want)
                odd += (~f).sum()
                assert (np.isnan(got) == np.isnan(want)).all(), (s, h)
                assert (got[np.isinf(want)] == want[np.isinf(want)]).all(), (s, h)
                assert (np.abs(got[f] - want[f]) <= np.broadcast_to(tol, want.shape)[f]).all(), (s, h)
    assert odd > 0 and int(c.status[0]) == 0


INF = float("inf")
SPECIAL_SHAPES = [((8, 2, 64, 16), [1, 16, 90, 333]), ((12, 1, 128, 8), [2, 700]),
                  ((3, 3, 80, 24), [33, 500]), ((6, 2, 256, 16), [5, 300]),
                  ((4, 1, 40, 7), [19, 64]), ((8, 1, 128, 32), [9000])]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("q", [-1.0, 1.0, -1.2345678])
@pytest.mark.parametrize("append", [False, True])
def test_attention_of_one_token_with_an_infinite_key(dtype, q, append):
    for shape in ((4, 2, 64, 16), (4, 4, 128, 8), (9, 1, 200, 5)):
        c = Cache(dtype, *shape, [1], append=append)
        c.q[:] = q
        c.qd.fill_(q)
        for h in range(c.kv):
            poke(c, 0, 0, 0, h, 7, INF)
        y, lse = c.run()
        check_special(c, y, lse)
        if q < 0:
            assert (y[0] == 0).all() and torch.isneginf(lse[0]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape,lens", SPECIAL_SHAPES)
@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("exact_q", [False, True])
def test_attention_of_infinite_keys(dtype, shape, lens, append, exact_q):
    # heads of both signs: scores of -infinity and of +infinity, one or several
    # per slot; queries with and without low parts
    g = np.random.default_rng(sum(shape))
    for several in (1, 5):
        c = Cache(dtype, *shape, lens, append=append)
        if exact_q:
            c.q = np.round(c.q * 4).astype(np.float32) / 4
            c.q[c.q == 0] = 0.25
            c.qd.copy_(torch.from_numpy(c.q))
        d = int(g.integers(0, c.D))
        for s, n in enumerate(lens):
            for t in {n - 1, *g.integers(0, n, several).tolist()}:
                for h in range(c.kv):
                    poke(c, 0, s, t, h, d, INF)
        check_special(c, *c.run())
        assert not append or c.check_stored() is None


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape,lens", SPECIAL_SHAPES)
def test_attention_of_scores_that_are_all_minus_infinity(dtype, shape, lens):
    c = Cache(dtype, *shape, lens)
    c.q = -np.abs(c.q) - np.float32(1e-30)  # one of them tiny beside the others
    c.q[..., 3] = -1e-25
    c.qd.copy_(torch.from_numpy(c.q))
    for s, n in enumerate(lens):
        for t in range(n):
            for h in range(c.kv):
                poke(c, 0, s, t, h, 3, INF)
    y, lse = c.run()
    check_special(c, y, lse)
    S = len(lens)
    assert (y[:S] == 0).all() and torch.isneginf(lse[:S]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_of_nan_keys_mixed_signs_and_infinite_queries(dtype):
    # -infinity - infinity and 0 x infinity are NaN, for the heads they concern
    c = Cache(dtype, 8, 2, 64, 16, [50, 70, 90, 40])
    poke(c, 0, 0, 20, 0, 5, float("nan"))
    poke(c, 0, 1, 33, 1, 5, INF)
    poke(c, 0, 1, 33, 1, 6, -INF)
    c.q[1, 4, 5], c.q[1, 4, 6] = -2.0, 3.0   # both products -infinity
    c.q[1, 5, 5], c.q[1, 5, 6] = -2.0, 0.0   # 0 x infinity
    c.q[2, 3, 9] = -INF                       # keys of both signs: NaN
    c.q[3, 0, 9] = -INF
    for t in range(40):
        poke(c, 0, 3, t, 0, 9, 0.5 + t / 64)  # all scores -infinity
    c.qd.copy_(torch.from_numpy(c.q))
    check_special(c, *c.run())


def test_attention_of_new_rows_beyond_the_half_type():
    # 1e6 is rounded to infinity when it is stored
    c = Cache("f16", 4, 4, 64, 16, [40, 17], append=True)
    for h in range(4):
        poke(c, 0, 0, 39, h, h, 1e6)
        poke(c, 0, 1, 16, h, h, -1e6)
    check_special(c, *c.run())
    c.check_stored()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape,lens", SPECIAL_SHAPES)
@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (31, 4)])
def test_attention_of_infinite_values(dtype, shape, lens, append, window, sinks):
    # a column with one sign, one with both, one with NaN, one of the first
    # token's, one of the last's; hidden rows hold them too
    g = np.random.default_rng(sum(shape) + append)
    c = Cache(dtype, *shape, lens, window, sinks, append=append)
    for s, n in enumerate(lens):
        seen = [t for t in range(n) if not window or t >= n - window or t < sinks]
        for h in range(c.kv):
            pick = lambda: int(g.choice(seen))  # noqa: E731
            for t in {pick(), pick(), pick()}:
                poke(c, 1, s, t, h, 1, -INF)
            poke(c, 1, s, pick(), h, 8, INF)
            poke(c, 1, s, pick(), h, 8, -INF)
            poke(c, 1, s, pick(), h, 17, float("nan"))
            poke(c, 1, s, pick(), h, 17, INF)
            poke(c, 1, s, 0, h, c.D - 1, INF) if 0 in seen else None
            poke(c, 1, s, n - 1, h, c.D - 2, -INF)
            if len(seen) < n:
                poke(c, 1, s, seen[-1] - window, h, 20, INF)
    check_special(c, *c.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_of_infinite_values_of_any_weight(dtype):
    # weights from 1 down to far below fp32's smallest, in a unit that several
    # blocks share; a score of -infinity has no weight to multiply
    n = 6000
    for lens in ([n], [300, 40]):
        c = Cache(dtype, 4, 1, 128, 16, lens, qscale=0.0)
        for s in range(len(lens)):
            c.q[s, :, 0] = (0.01, 1.0, 4.0, -4.0)
            for i, t in enumerate(np.linspace(0, lens[s] - 1, 12).astype(int)):
                poke(c, 0, s, int(t), 0, 0, -100.0 * i)
                poke(c, 1, s, int(t), 0, 3 * i, INF if i % 2 else -INF)
            poke(c, 0, s, lens[s] - 3, 0, 5, INF)   # scores 0 x infinity: NaN but for head 2
        c.q[:, 2, 5] = -1.0
        c.qd.copy_(torch.from_numpy(c.q))
        for s in range(len(lens)):
            poke(c, 1, s, lens[s] - 3, 0, 70, INF)
        check_special(c, *c.run())
        # ... and without it
        for s in range(len(lens)):
            poke(c, 0, s, lens[s] - 3, 0, 5, 0.0)
        check_special(c, *c.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_of_infinite_keys_and_values(dtype):
    c = Cache(dtype, 16, 1, 64, 16, [200, 3000])
    for s, t in ((0, 7), (0, 100), (1, 10), (1, 2500)):
        poke(c, 0, s, t, 0, 4, INF if t != 100 else -INF)
        poke(c, 1, s, t + 1, 0, 9, INF)
        poke(c, 1, s, t, 0, 10, -INF)
    c.q[0, :8, 4] = 0.25
    c.qd.copy_(torch.from_numpy(c.q))
    check_special(c, *c.run())


# ------------------------------------------------------------------ page counts past 2^31
def test_fork_wants_more_pages_than_32_bits_count():
    # 1024 slots that each want 2^21 pages of one token (2^31 in all, tables of
    # 8 GB), 1000 pages to be had: the first slot takes them
    S, mp, pages = 1024, 1 << 21, 1000
    desc = pi.make_cache_desc(1, pages, 1, 8, 1, "f16")
    tables = [torch.empty((S, mp), dtype=torch.int32, device=DEV) for _ in range(2)]
    length, ref, pairs = i32([7] * S), i32([7] * pages), i32([[7, 7]] * S)
    counts, st, ws = i32([7] * 4), new_status(), pi.cache_workspace(desc, S, 0, DEV)
    pi.check(pi.pi_cache_fork(desc, S, mp, i32([-1] * S), i32([mp] * S), None, tables[0], i32([0] * S),
                              tables[1], length, ref, None, pairs, counts, st, ws))
    torch.cuda.synchronize()
    assert int(st[0]) == pi.PI_ERR_CAPACITY
    assert length.tolist() == [pages] + [0] * (S - 1) and ref.tolist() == [1] * pages
    assert counts.tolist() == [0, pages, 7, 7]
    assert tables[1][0, :pages].tolist() == list(range(pages))
    tables[1][0, :pages] = -1
    assert int(tables[1].max()) == -1 and int(tables[1].min()) == -1


@pytest.mark.parametrize("mp", [2 ** 31 - 1, 2 ** 31 - 4])
def test_tables_that_end_at_the_largest_index(mp):
    # one slot, pages of one token, a row of 8 GB read one entry or four at a time
    pages = 9
    desc = pi.make_cache_desc(1, pages, 1, 8, 1, "f16")
    tables = [torch.empty((1, mp), dtype=torch.int32, device=DEV) for _ in range(2)]
    tables[0][0, :3] = i32([8, 2, 5])
    length, ref, where, pairs = i32([0]), i32([7] * pages), i32([7] * pages), i32([[7, 7]] * pages)
    counts, st, ws = i32([7] * 4), new_status(), pi.cache_workspace(desc, 1, 0, DEV)
    pi.check(pi.pi_cache_fork(desc, 1, mp, i32([0]), i32([2]), None, tables[0], i32([3]), tables[1], length,
                              ref, None, pairs, counts, st, ws))
    torch.cuda.synchronize()
    del tables[0]
    t = tables[0]
    assert int(st[0]) == 0 and length.tolist() == [5] and counts.tolist() == [0, 5, 7, 7]
    assert t[0, :5].tolist() == [8, 2, 5, 0, 1] and ref.tolist() == [1, 1, 1, 0, 0, 1, 0, 0, 1]
    pi.check(pi.pi_cache_compact(desc, 1, mp, None, t, length, t, ref, where, None, pairs, counts, st, ws))
    torch.cuda.synchronize()
    assert int(st[0]) == 0 and counts.tolist()[:2] == [2, 5]
    assert t[0, :5].tolist() == [4, 2, 3, 0, 1] and ref.tolist() == [1, 1, 1, 1, 1, 0, 0, 0, 0]
    t[0, :5] = -1
    for part in t[0].split(1 << 28):
        assert int(part.max()) == -1 and int(part.min()) == -1


# ------------------------------------------------------------------ sums that are split
def indicate(c):
    """Values that are 1 in one element and 0 in the others, the element chosen
    by the token's tile of 16: y is then each class's share of the weights."""
    for s, n in enumerate(c.lens):
        t = np.arange(n)
        v = (t[:, None] // 16 % c.D == np.arange(c.D)[None, :]).astype(np.float64)
        c.rows[1, s, :n] = v[:, None, :]
        for j in range(-(-n // c.P)):
            t0, t1 = j * c.P, min(n, (j + 1) * c.P)
            blk = torch.from_numpy(v[t0:t1]).to(TD[c.dtype]).to(DEV)
            c.pool[c.layer, int(c.np_table[s, j]), 1, :, :t1 - t0] = blk[None]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape,lens", [
    ((8, 1, 128, 64), [20011]), ((16, 1, 64, 32), [9000, 0, 3]), ((4, 2, 256, 8), [1, 7003]),
    ((3, 3, 96, 7), [5000, 4100]), ((12, 1, 128, 24), [2500, 11000, 640]),
    ((40, 40, 128, 16), [700, 1300, 61]), ((8, 8, 64, 16), [333] * 30), ((6, 2, 40, 16), [1000, 257])])
def test_attention_loses_and_doubles_no_part(dtype, shape, lens):
    # All terms are positive, so an element of y has a relative error: the
    # weights' e = |da| + 2^-20 in numerator and denominator, 2^-22 of the
    # weights' parts, 2^-19 for the 16 products of a tile, and U for each sum of
    # tiles, warps and parts that it passes (under 2^10 of them at these sizes:
    # a warp's tiles, 4 warps, groups, parts).  A tile that is lost or counted
    # twice moves its element by one over the tiles of its class: a 40th at least.
    c = Cache(dtype, *shape, lens, qscale=0.05)
    indicate(c)
    y, lse = c.run()
    torch.cuda.synchronize()
    y, lse = y.double().cpu().numpy(), lse.double().cpu().numpy()
    G = c.heads // c.kv
    for s, n in enumerate(lens):
        for h in range(c.heads):
            if n == 0:
                assert (y[s, h] == 0).all()
                continue
            q, k = c.q[s, h].astype(np.float64), c.rows[0, s, :n, h // G]
            a = c.scale * (k @ q)
            p = np.exp(a - a.max())
            want = p @ c.rows[1, s, :n, h // G] / p.sum()
            da = c.scale * (np.abs(k) @ np.abs(q)).max() * (2.0 ** -21 + c.D * U)
            tol = 2 * (da + 2.0 ** -20 + 2.0 ** -22 + 2.0 ** -19 + 2 ** 10 * U)
            assert tol < 1 / 1000
            assert (np.abs(y[s, h] - want) <= tol * want).all(), (s, h)
            z = a.max() + math.log(p.sum())
            assert abs(lse[s, h] - z) <= tol + 4 * U * abs(z), (s, h)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,topk", [(1, 50273, 8), (2, 200001, 32), (7, 50273, 0), (1, 131072, 1),
                                             (300, 33000, 4), (1700, 9001, 3)])
def test_scores_lose_and_double_no_part(dtype, rows, vocab, topk):
    # A sum passes 32 terms of a thread's batch, at most vocab / 4096 batches (128
    # threads a row, 32 elements a batch), 5 + 8 warp sums and 64 parts: under 256
    # roundings, so its relative error is e = 2^-20 + 2^8 U.  The entropy's
    # t / s has terms of one sign but for the largest's, of mean |d| under the
    # entropy's own size: |d entropy| <= 2 e (1 + log n) + 4 U R.  Every part's
    # share of either sum is a 64th or more: logits rise and fall slowly over
    # the row, so that no part is like another.
    g = np.random.default_rng(vocab)
    x = g.standard_normal((rows, vocab)) + 2 * np.sin(np.arange(vocab) * (7.0 / vocab))
    tok = g.integers(0, vocab, rows)
    xd = torch.from_numpy(x).to(TD[dtype]).to(DEV)
    x = xd.double().cpu().numpy()
    lp, ent = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    idx, top = i32(np.zeros((rows, max(1, topk)))), torch.empty((rows, max(1, topk)), device=DEV)
    st = new_status()
    pi.check(pi.pi_token_logprobs(xd, dtype, rows, vocab, vocab, i32(tok), topk, lp, ent, idx, top, st,
                                  pi.logprob_workspace(rows, vocab, topk, DEV)))
    torch.cuda.synchronize()
    m = x.max(1, keepdims=True)
    z = m + np.log(np.exp(x - m).sum(1, keepdims=True))
    p = np.exp(x - z)
    want_ent, want_lp = -(p * (x - z)).sum(1), x[np.arange(rows), tok] - z[:, 0]
    e, R = 2.0 ** -20 + 2.0 ** 8 * U, float(x.max() - x.min())
    got_ent, got_lp = ent.double().cpu().numpy(), lp.double().cpu().numpy()
    assert (np.abs(got_ent - want_ent) <= 2 * e * (1 + math.log(vocab)) + 4 * U * R).all()
    assert (np.abs(got_lp - want_lp) <= 2 * e + 4 * U * (np.abs(want_lp) + R)).all()
    assert int(st[0]) == 0


# ------------------------------------------------------------------ scales, workspaces, threads
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.125, -3.0, 1e-30])
def test_attention_scales(dtype, scale):
    c = Cache(dtype, 8, 2, 64, 16, [0, 1, 40, 300, 1000])
    c.scale = scale
    y, lse = c.run()
    torch.cuda.synchronize()
    y, lse = y.double().cpu().numpy(), lse.double().cpu().numpy()
    for s, n in enumerate(c.lens):
        for h in range(c.heads if n else 0):
            q, k = c.q[s, h].astype(np.float64), c.rows[0, s, :n, h // 4]
            a = scale * (k @ q)
            p = np.exp(a - a.max())
            want, z = p @ c.rows[1, s, :n, h // 4] / p.sum(), a.max() + math.log(p.sum())
            e = abs(scale) * (np.abs(k) @ np.abs(q)).max() * (2.0 ** -21 + c.D * U) + 2.0 ** -20 + n * U
            assert (np.abs(y[s, h] - want) <= 3 * e * np.abs(c.rows[1, s, :n]).max()).all()
            assert abs(lse[s, h] - z) <= 2 * e + 4 * U * abs(z)


def test_one_workspace_serves_caches_of_several_shapes():
    # attention joined across blocks, forks and compactions of other pools in
    # between, on one workspace: each call's results are those on its own
    a = Cache("f16", 8, 1, 128, 16, [9000, 70])
    b = Cache("bf16", 12, 3, 256, 8, [3000, 0, 17], seed=2)
    small, large = (9, 4, 7, 40), (600, 16, 90, 70_001)
    sizes = [pi.pi_cache_workspace_size(c.desc, len(c.lens), c.heads) for c in (a, b)]
    for S, P, mp, pages in (small, large):
        sizes.append(pi.pi_cache_workspace_size(pi.make_cache_desc(1, pages, 1, 8, P, "f16"), S, 0))
    ws = torch.zeros(max(sizes), dtype=torch.uint8, device=DEV)
    want = [c.run() for c in (a, b)]
    a.ws = b.ws = ws

    def pages_calls(S, P, mp, pages):
        desc = pi.make_cache_desc(1, pages, 1, 8, P, "f16")
        table, length, st = i32(np.full((S, mp), -1)), i32([0] * S), new_status()
        t2, l2, ref, where = i32(np.full((S, mp), -1)), i32([0] * S), i32([0] * pages), i32([0] * pages)
        pairs, counts = i32(np.zeros((pages, 2))), i32([0] * 4)
        need = P * (pages // (2 * S))
        pi.check(pi.pi_cache_fork(desc, S, mp, i32([-1] * S), i32([need] * S), None, table, length, t2, l2,
                                  ref, None, pairs, counts, st, ws))
        assert l2.tolist() == [need] * S and int(counts[1]) == S * (need // P) and int(st[0]) == 0
        pi.check(pi.pi_cache_compact(desc, S, mp, None, t2, l2, t2, ref, where, None, pairs, counts, st, ws))
        assert int(counts[1]) == S * (need // P) and int(st[0]) == 0

    for _ in range(2):
        for c, (y, lse) in zip((a, b), want):
            y1, l1 = c.run()
            assert torch.equal(y, y1) and torch.equal(lse, l1)
            pages_calls(*small)
            y1, l1 = c.run()
            assert torch.equal(y, y1) and torch.equal(lse, l1)
            pages_calls(*large)


def test_two_threads_on_two_streams():
    # each with its own workspace; what one call looks up once is shared
    import threading
    torch.cuda.synchronize()
    work, failed = [], []
    for i in range(2):
        c = Cache(("f16", "bf16")[i], 8, 2, (128, 96)[i], 16, [3000, 1, 200], seed=i)
        x = torch.randn((5, 30011), device=DEV)
        work.append((c, x, torch.cuda.Stream(), c.run()))
    torch.cuda.synchronize()

    def go(c, x, stream, want):
        try:
            with torch.cuda.stream(stream):
                ent, top = torch.empty(5, device=DEV), torch.empty((5, 3), device=DEV)
                idx = torch.empty((5, 3), dtype=torch.int32, device=DEV)
                st, ws = new_status(), pi.logprob_workspace(5, 30011, 3, DEV)
                best = torch.topk(x, 3).indices.int()
                for _ in range(20):
                    y, lse = c.run()
                    pi.check(pi.pi_token_logprobs(x, "f32", 5, 30011, 30011, None, 3, None, ent, idx, top,
                                                  st, ws))
                    stream.synchronize()
                    assert torch.equal(y, want[0]) and torch.equal(lse, want[1])
                    assert torch.equal(idx, best) and int(st[0]) == 0
        except Exception as e:  # reported by the test's own thread
            failed.append(e)

    threads = [threading.Thread(target=go, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
