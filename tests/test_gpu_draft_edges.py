"""The operators of include/pi_draft.h where operands, numbers or the way they are
called could make them fail, against plain 64-bit forms."""
import math
import os
import sys
import threading

import numpy as np
import pytest
import torch

import activation_sparse_decode_rank_gb300 as pi
import drafthelp as plain
from test_gpu_draft import (DEV, TD, U, Accept, Tree, draw_rows, f32, i32, new_status, rounded,
                            run_sample)

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# few and many query rows per kv head: the two forms of the kernel
FEW, MANY = (8, 2, 128, 16), (32, 1, 64, 16)


@pytest.fixture(scope="module", autouse=True)
def _built():
    pi.build()


def compare(t, y, lse, seen=None):
    """Like Tree.check, with infinite operands: NaN and infinities where the definition has them."""
    torch.cuda.synchronize()
    y, lse = y.double().cpu().numpy(), lse.double().cpu().numpy()
    G = t.heads // t.kv
    for s in range(t.S):
        for i in range(t.count[s]):
            for h in range(t.kv):
                hs = slice(h * G, (h + 1) * G)
                vis = (seen or t.seen)[s][i]
                q = t.q[s, i, hs].astype(np.float64)
                k, v = t.rows[0, s, :, h], t.rows[1, s, :, h]
                yo, lo, _, _ = plain.attention(q, k, v, vis, t.scale)
                kf, vf = np.where(np.isfinite(k), k, 0.0), np.where(np.isfinite(v), v, 0.0)
                mag = (np.abs(q) @ np.abs(kf[vis]).T).max()
                e = t.scale * mag * (2.0 ** -21 + t.D * U) + 2.0 ** -20 + 2.0 ** -22 + len(vis) * U
                for g in range(G):
                    got, want = y[s, i, h * G + g], yo[g]
                    assert (np.isnan(got) == np.isnan(want)).all(), (s, i, h, g)
                    assert (got[np.isinf(want)] == want[np.isinf(want)]).all()
                    ok = np.isfinite(want)
                    assert (np.abs(got[ok] - want[ok]) <= 3 * e * np.abs(vf[vis]).max()).all()
                a, b = lse[s, i, hs], lo
                assert (np.isnan(a) == np.isnan(b)).all()
                ok = np.isfinite(b)
                assert (np.abs(a[ok] - b[ok]) <= 2 * e + 4 * U * np.abs(b[ok])).all()


def put(t, kind, s, tok, d, value):
    """Sets an element of a token's key (0) or value (1) in the pool, the new rows and the plain rows."""
    t.rows[kind, s, tok, :, d] = value
    page = int(t.np_table[s, tok // t.P])
    t.pool[t.layer, page, kind, :, tok % t.P, d] = value
    if t.append and tok >= t.base[s]:
        (t.knew, t.vnew)[kind][s, tok - t.base[s], :, d] = value


# ------------------------------------------------------------------ infinite operands
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", [FEW, MANY, (4, 1, 256, 8), (4, 2, 64, 5)])
@pytest.mark.parametrize("append", [False, True])
def test_infinite_values(dtype, shape, append):
    inf, nan = math.inf, math.nan
    t = Tree(dtype, *shape, [200, 20, 700], [6, 6, 3], 6, append=append, qscale=0.3, seed=1)
    put(t, 1, 0, 7, 3, inf)          # seen by all drafts of slot 0
    put(t, 1, 0, 150, 3, -inf)       # both signs: NaN
    put(t, 1, 0, 150, 11, -inf)
    put(t, 1, 1, 20 + 2, 5, inf)     # a draft's: seen by itself and those below it
    put(t, 1, 1, 20 + 4, 9, nan)
    put(t, 1, 2, 690, shape[2] - 1, nan)
    compare(t, *t.run())
    assert int(t.status[0]) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", [FEW, MANY, (4, 1, 256, 8)])
@pytest.mark.parametrize("append", [False, True])
def test_infinite_keys(dtype, shape, append):
    inf, nan = math.inf, math.nan
    t = Tree(dtype, *shape, [200, 20, 5], [6, 6, 3], 6, append=append, qscale=0.3, seed=2)
    put(t, 0, 0, 7, 3, inf)          # +-infinity by the sign of q: weight 0, or NaN
    put(t, 0, 1, 20 + 2, 5, -inf)
    put(t, 0, 1, 20 + 4, 9, nan)
    put(t, 0, 2, 0, 1, inf)
    put(t, 0, 2, 0, 2, -inf)
    compare(t, *t.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", [FEW, MANY])
def test_queries_that_are_not_finite(dtype, shape):
    t = Tree(dtype, *shape, [100, 20], None, 4, seed=3)
    t.q[0, 1, 0, 5], t.q[1, 2, 1, 0] = np.nan, np.inf
    t.qd = torch.from_numpy(t.q).to(DEV)
    y, lse = t.run()
    torch.cuda.synchronize()
    assert torch.isnan(y[0, 1, 0]).all() and torch.isnan(lse[0, 1, 0])
    assert torch.isnan(y[1, 2, 1]).all() and torch.isnan(lse[1, 2, 1])
    bad = torch.isnan(lse[:2])
    assert int(bad.sum()) == 2  # the other heads and drafts are as ever
    t.q[0, 1, 0, 5] = t.q[1, 2, 1, 0] = 0.25
    keep = y.clone(), lse.clone()
    t.qd = torch.from_numpy(t.q).to(DEV)
    y, lse = t.run()
    for a, b in zip((y[:2], lse[:2]), keep):
        assert torch.equal(a[~bad], b[:2][~bad])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("qscale", [1e8, 1e20])
@pytest.mark.parametrize("shape", [FEW, MANY])
def test_large_scores_stay_finite(dtype, qscale, shape):
    t = Tree(dtype, *shape, [300, 1], None, 5, qscale=qscale, seed=4)
    y, lse = t.run()
    torch.cuda.synchronize()
    assert torch.isfinite(y).all() and torch.isfinite(lse).all()
    # a mean of values lies between them
    for s in range(2):
        v = np.abs(t.rows[1, s]).max()
        assert float(y[s].abs().max()) <= v * (1 + 2.0 ** -18)


# ------------------------------------------------------------------ numbers out of range
@pytest.mark.parametrize("shape", [(8, 2, 64, 16), (64, 2, 64, 16), (4, 2, 64, 5), (4, 2, 128, 64), (2, 1, 256, 16)])
@pytest.mark.parametrize("append", [False, True])
def test_bad_page_numbers(shape, append):
    P = shape[3]
    for s, j, bad in ((0, 40 // P, -2), (1, 0, 10 ** 9), (2, 46 // P, 2 ** 31 - 1)):
        t = Tree("f16", *shape, [100, 60, 45], None, 4, append=append, seed=5)
        tab = t.np_table.copy()
        tab[s, j] = bad
        y, lse = t.run(table=i32(tab))
        hidden = set(range(j * P, j * P + P))
        if append:  # new rows are seen, though not stored
            hidden -= set(range(t.base[s], t.lens[s]))
        seen = [[[k for k in v if r != s or k not in hidden] for v in t.seen[r]] for r in range(3)]
        assert int(t.status[0]) == pi.PI_ERR_INDEX
        t.status.zero_()
        if append:
            t.append = False  # its rows are not all stored
        t.check(y, lse, seen)


def test_bad_parents_lengths_and_counts():
    t = Tree("f16", 4, 2, 64, 16, [50, 20, 30, 9], [5, 5, 5, 5], 5, seed=6)
    t.parent[0] = [-1, 3, 1, 2, 0]      # draft 1's parent is no earlier draft
    t.parent[1] = [-5, 0, 1, 2, 3]
    par = i32(t.parent)
    length = i32([t.lens[0], t.lens[1], t.mp * 16 + 1, t.lens[3]])
    count = i32([5, 5, 5, 6])
    y, lse = t.run(parent=par, len=length, count=count)
    assert int(t.status[0]) == pi.PI_ERR_INDEX
    t.status.zero_()
    t.parent[0][1], t.parent[1][0] = -1, -1
    t.seen = [[plain.visible(t.base[s], t.parent[s], i, 0, 0) for i in range(5)] for s in range(4)]
    t.count = [5, 5, 0, 0]
    t.check(y, lse)
    # a count past the length
    y, lse = t.run(len=i32([3, 4, 0, 5]), count=i32([5, 5, 1, 5]))
    torch.cuda.synchronize()
    assert int(t.status[0]) == pi.PI_ERR_INDEX
    assert (y[:3] == 77.0).all() and not (y[3] == 77.0).any()


# ------------------------------------------------------------------ how it is called
@pytest.mark.parametrize("shape,N", [(FEW, 4), (MANY, 4), ((16, 1, 128, 16), 64)])
def test_same_bits_every_time(shape, N):
    t = Tree("bf16", *shape, [3000, 5, 777, 1], None, N, append=True, seed=7)
    first = [x.clone() for x in t.run()]
    for _ in range(5):
        for a, b in zip(first, t.run()):
            assert torch.equal(a, b)


def test_streams_and_graphs():
    a = Tree("f16", 8, 2, 128, 16, [500, 40], None, 6, append=True, seed=8)
    b = Tree("bf16", 32, 2, 64, 16, [90, 700], None, 3, seed=9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ya = a.run(stream=side)
    yb = b.run()
    torch.cuda.synchronize()
    a.check(*ya)
    b.check(*yb)
    # two graphs, one workspace, in turn; what they read changes between replays
    ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    outs, graphs = [], []
    for t in (a, b):
        y = torch.full((t.S + 1, t.drafts, t.heads, t.D), 77.0, device=DEV)
        lse = torch.full((t.S + 1, t.drafts, t.heads), 77.0, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            t.run(y=y, lse=lse, ws=ws)
        outs.append((y, lse))
        graphs.append(g)
    for _ in range(2):
        for t, (y, lse), g in zip((a, b), outs, graphs):
            y.fill_(77.0)
            lse.fill_(77.0)
            g.replay()
            t.check(y, lse)
    b.qd.copy_(-b.qd)
    b.q = -b.q
    b.len.copy_(i32([90, 700]))  # three tokens fewer
    b.lens, b.base = [90, 700], [87, 697]
    b.seen = [[plain.visible(b.base[s], b.parent[s], i, 0, 0) for i in range(3)] for s in range(2)]
    outs[1][0].fill_(77.0)
    outs[1][1].fill_(77.0)
    graphs[1].replay()
    b.check(*outs[1])


def test_two_threads():
    ts = [Tree("f16", 8, 2, 64, 16, [300 + 40 * k, 9], None, 5, append=True, seed=10 + k) for k in range(2)]
    got = [None, None]

    def work(k):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                got[k] = ts[k].run(stream=s)
            s.synchronize()
    torch.cuda.synchronize()
    th = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    [x.start() for x in th]
    [x.join() for x in th]
    for k in range(2):
        ts[k].check(*got[k])


def test_offsets_past_31_bits():
    t = Tree("f16", 4, 1, 128, 16, [40, 3], None, 5, append=True, seed=12, pages=600000)
    assert t.pool.numel() > 2 ** 31
    t.check(*t.run())


@pytest.mark.parametrize("shape", [(8, 2, 128, 112), (32, 1, 64, 112), (4, 1, 256, 112), (8, 2, 32, 126),
                                   (32, 1, 64, 126)])
@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("short", [0, 5])
@pytest.mark.parametrize("infinite", [False, True])
def test_lengths_next_to_the_largest(shape, append, short, infinite):
    """Tokens up to 2^31: the numbers of the last tile's columns pass 31 bits."""
    P = shape[3]
    most = (2 ** 31 - 1) // P
    base = 10 * P - 16 - short
    t = Tree("f16", *shape, [base], None, 16, window=300, sinks=37, append=append, seed=14)
    if infinite:  # the rows once more in fp32
        put(t, 1, 0, base - 3, 2, math.inf)
    # the sinks' page stays, the window's pages go to the row's end; none in between is valid
    tab = torch.full((1, most), -7, dtype=torch.int32, device=DEV)
    tab[0, 0] = int(t.np_table[0, 0])
    tab[0, most - 9:] = i32(t.np_table[0, 1:10])
    t.mp = most
    y, lse = t.run(table=tab, len=i32([most * P - short]))
    if infinite:
        compare(t, y, lse)
        assert int(t.status[0]) == 0
    else:
        t.check(y, lse)


@pytest.mark.parametrize("args", [("f16", 8, 2, 64, 16), ("bf16", 64, 2, 128, 16), ("f16", 2, 1, 256, 8)])
def test_lost_copy_times_out(args):
    t = Tree(*args, [300, 40], None, 4, shape="chain", seed=13)
    y = torch.empty((2, 4, t.heads, t.D), device=DEV)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    pi.check(pi.pi_selftest_tree_timeout(t.desc, 2, t.heads, t.mp, 4, t.qd, t.table, t.len, t.pool, y, t.status,
                                         t.ws, 2_000_000), "pi_selftest_tree_timeout")
    end.record()
    torch.cuda.synchronize()
    assert int(t.status[0]) == pi.PI_ERR_TIMEOUT and start.elapsed_time(end) < 6000
    t.status.zero_()
    t.check(*t.run())  # the next call is as ever


# ------------------------------------------------------------------ sampling
def expected(x, T, top_k, top_p, u):
    """Vectorised plain form of one row for large vocabularies, with its margin."""
    order = np.lexsort((np.arange(len(x)), -x))
    w = np.exp((x[order] - x[order[0]]) / T)
    n = int((w > 0).sum())
    n = min(n, top_k) if top_k > 0 else n
    c, margin = np.cumsum(w[:n]), 1.0
    if top_p < 1:
        goal = top_p * c[-1]
        m = int(np.searchsorted(c, goal)) + 1
        margin = np.abs(c[max(m - 2, 0):m] - goal).min() / c[-1]
        c = c[:m]
    goal = u * c[-1]
    at = int(np.searchsorted(c, goal, side="right"))
    near = [v for v in (c[at - 1] if at else None, c[at] if at + 1 < len(c) else None) if v is not None]
    margin = min([margin] + [abs(v - goal) / c[-1] for v in near])
    return order[at], math.log(w[at] / c[-1]), margin


@pytest.mark.parametrize("dtype,V", [("f32", 700001), ("f32", 250001), ("bf16", 2000003),
                                     ("f16", 300000)])
def test_sample_large_vocabularies(dtype, V):
    g = np.random.default_rng(V)
    for R in (1, 5):
        x = (g.standard_normal((R, V)) * 2).astype(np.float32)
        u = g.random(R).astype(np.float32)
        top_k = [0, 0, 40, 900, 5000][:R]
        top_p = np.float32([1.0, 0.9, 1.0, 0.8, 0.97][:R])
        tok, lp, status = run_sample(x, dtype, [0.9] * R, top_k, top_p, None, u, pad=3)
        xr = rounded(x, dtype)
        for r in range(R):
            want = expected(xr[r], float(np.float32(0.9)), top_k[r], float(top_p[r]), float(u[r]))
            assert want[2] >= 2.0 ** -30 and tok[r] == want[0]
            assert abs(lp[r] - want[1]) <= 4 * U * (1 + abs(want[1]))
        assert status == 0


def test_sample_graph_stream_and_repeats():
    g = np.random.default_rng(3)
    rows = draw_rows(g, 16, 5000, "f32")
    x = f32(np.stack([r[0] for r in rows]))
    T, k, p, m, u = (f(c) for f, c in zip((f32, i32, f32, f32, f32), zip(*(r[1] for r in rows))))
    tok, lp, status = torch.zeros(16, dtype=torch.int32, device=DEV), torch.zeros(16, device=DEV), new_status()
    ws = pi.sample_workspace(16, 5000, DEV)

    def call(stream=None):
        pi.check(pi.pi_token_sample(x, "f32", 16, 5000, 5000, T, k, p, m, u, tok, lp, status, ws, stream=stream),
                 "pi_token_sample")
    want = [r[2] for r in rows]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.synchronize()
    assert tok.tolist() == want
    first = lp.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        tok.zero_()
        lp.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert tok.tolist() == want and torch.equal(lp, first)
    x.copy_(x.flip(0))
    for a in (T, k, p, m, u):
        a.copy_(a.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert tok.tolist() == want[::-1] and int(status[0]) == 0


def test_sample_more_rows_than_blocks():
    g = np.random.default_rng(4)
    R, V = 5000, 60
    x = g.standard_normal((R, V)).astype(np.float32)
    u = g.random(R).astype(np.float32)
    tok, lp, _ = run_sample(x, "f32", None, None, None, None, u)
    for r in range(0, R, 7):
        want = plain.sample_row(x[r], 1.0, 0, 1.0, 0.0, float(u[r]))
        assert want[2] < 2.0 ** -30 or tok[r] == want[0]


# ------------------------------------------------------------------ acceptance
def test_accept_in_a_graph():
    a = Accept(6, 9, 16, 40, 2, 2, 64, "f16", seed=8, wide=1)
    arg = dict(parent=i32(a.parent), count=i32(a.count), tokens=i32(a.tokens), choice=i32(a.choice),
               table=i32(a.tab), len=i32(a.lens), pool=a.pool)
    before = a.pool.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pi.check(pi.pi_tree_accept(a.desc, 6, a.mp, 9, *arg.values(), *a.out, a.status), "pi_tree_accept")
    a.pool.copy_(before)
    graph.replay()
    torch.cuda.synchronize()
    a.check(before)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("slots,temperature", [(1, 0.7), (3, 0.5), (4, 0.0)])
def test_draft_decode(slots, temperature):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import draft_decode as ex
    model = ex.Decoder(seed=3)
    prompts = torch.randint(0, ex.VOCAB, (slots, 37), generator=torch.Generator().manual_seed(slots))
    dec = ex.DraftDecoder(model, slots, 37 + 30 + ex.DRAFTS, temperature)
    out, steps = dec.run(prompts, 30)
    assert int(dec.status[0]) == 0 and int(model.status[0]) == 0
    assert steps <= 30
    u = dec.u.double().cpu().numpy()
    for s, t in enumerate(out):
        assert len(t) >= 67
        # every token is the one that its position's number draws from a pass without a cache
        logits, _ = model.prompt(torch.tensor(t[:-1], device=DEV))
        x = logits.double().cpu().numpy()
        for p in range(37, len(t)):
            want = plain.sample_row(x[p - 1], float(np.float32(temperature)), 50, float(np.float32(0.95)), 0.0,
                                    float(u[s, p]))
            second = np.sort(x[p - 1])[-2:]
            near = want[2] < 1e-3 or (temperature == 0 and second[1] - second[0] < 1e-3)
            assert near or t[p] == want[0], (s, p)
