"""The operators of include/pi_draft.h on the GPU against plain 64-bit forms
(drafthelp.py).

Tolerances, from the arithmetic the headers promise (u = 2^-24):
  * a score a = scale q . k: q keeps at least 22 bits and a sum of D products
    rounds D times at most, so |da| <= scale |q|.|k| (2^-21 + D u); an
    exponential adds 2^-20 relative, a weight's parts 2^-22; a sum of n terms n u
    at most.  With e = |da| + 2^-20 + 2^-22 + n u the weights are off by e
    relative (numerator and denominator), so |dy| <= 3 e max|v| and
    |dlse| <= 2 e + 4 u |lse|.
  * a drawn token is the plain form's where the draw and the ends of the kept part
    are 2^-30 or more from where they would change (sums are exact to 2^-35 of each
    weight, so the sums themselves to 2^-35, and the plain form's to n 2^-53); where they
    are nearer the row is drawn anew.  Its log probability is off by at most 4 u
    (1 + |logprob|): a rounding each of w / sum, the logarithm's argument and its result.
  * whole numbers and stored 16-bit values are equal.
"""
import math

import numpy as np
import pytest
import torch

import activation_sparse_decode_rank_gb300 as pi
import drafthelp as plain

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
TD = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    pi.build()


def i32(a):
    return torch.tensor(np.ascontiguousarray(a), dtype=torch.int32, device=DEV)


def f32(a):
    return torch.tensor(np.ascontiguousarray(a), dtype=torch.float32, device=DEV)


def new_status():
    return torch.zeros(4, dtype=torch.int32, device=DEV)


def random_parents(g, drafts):
    """A forest: mostly one tree, some drafts without a parent."""
    p = [-1]
    for i in range(1, drafts):
        p.append(-1 if g.random() < 0.1 else int(g.integers(max(0, i - 5), i)))
    return p


class Tree:
    """A one-call problem: every row of the pool that no draft may see is NaN."""

    def __init__(self, dtype, heads, kv, D, page, base, count, drafts, shape="tree", window=0, sinks=0,
                 append=False, layers=1, layer=0, qscale=1.5, seed=0, pages=None):
        g = np.random.default_rng(seed)
        S = len(base)
        self.__dict__.update(dtype=dtype, heads=heads, kv=kv, D=D, P=page, base=list(base), S=S,
                             drafts=drafts, window=window, sinks=sinks, append=append, layer=layer,
                             shape=shape)
        self.count = list(count) if count is not None else [drafts] * S
        self.lens = [b + c for b, c in zip(self.base, self.count)]
        self.parent = [list(range(-1, drafts - 1)) if shape == "chain" else random_parents(g, drafts)
                       for _ in range(S)]
        need = [-(-n // page) for n in self.lens]
        self.mp = max(1, max(need)) + 1
        self.pages = pages or sum(need) + 2
        order = self.pages - 1 - g.permutation(sum(need)) if pages else g.permutation(self.pages)
        tab = np.full((S, self.mp), -7, np.int64)
        at = 0
        for s in range(S):
            tab[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
        self.np_table = tab
        self.pool = torch.empty((layers, self.pages, 2, kv, page, D), dtype=TD[dtype], device=DEV)
        if not pages:
            self.pool.fill_(float("nan"))
        rows = g.standard_normal((2, S, max(self.lens + [1]), kv, D)).astype(np.float32)
        new = np.zeros((2, S, drafts, kv, D), np.float32)
        for s in range(S):
            new[:, s, :self.count[s]] = rows[:, s, self.base[s]:self.lens[s]]
        self.knew, self.vnew = (torch.from_numpy(new[i]).to(DEV) if append else None for i in (0, 1))
        self.rows = torch.from_numpy(rows).to(TD[dtype]).to(torch.float64).numpy()
        self.seen = [[plain.visible(self.base[s], self.parent[s], i, window, sinks)
                      for i in range(self.count[s])] for s in range(S)]
        for s in range(S):
            some = set(t for v in self.seen[s] for t in v)
            blk = torch.from_numpy(self.rows[:, s, :self.lens[s]]).to(TD[dtype])
            for t in range(self.lens[s]):
                if t not in some or (append and t >= self.base[s]):
                    blk[:, t] = float("nan")
            blk = blk.to(DEV)
            for j in range(need[s]):
                t0, t1 = j * page, min(self.lens[s], (j + 1) * page)
                self.pool[layer, int(tab[s, j])][:, :, :t1 - t0] = blk[:, t0:t1].permute(0, 2, 1, 3)
        self.q = g.standard_normal((S, drafts, heads, D)).astype(np.float32) * np.float32(qscale)
        self.qd = torch.from_numpy(self.q).to(DEV)
        self.table, self.len = i32(tab), i32(self.lens)
        self.scale = D ** -0.5
        self.desc = pi.make_cache_desc(layers, self.pages, kv, D, page, dtype)
        self.ws = pi.tree_workspace(self.desc, S, heads, drafts, DEV)
        self.par = None if shape == "chain" else i32(self.parent)
        self.cnt = None if count is None else i32(self.count)
        self.status = new_status()

    def run(self, want_lse=True, stream=None, **kw):
        a = dict(parent=self.par, count=self.cnt, q=self.qd, k_new=self.knew, v_new=self.vnew,
                 table=self.table, len=self.len, pool=self.pool, scale=self.scale, window=self.window,
                 sinks=self.sinks)
        y = kw.pop("y", None)
        if y is None:
            y = torch.full((self.S + 1, self.drafts, self.heads, self.D), 77.0, device=DEV)
        lse = kw.pop("lse", None)
        if lse is None and want_lse:
            lse = torch.full((self.S + 1, self.drafts, self.heads), 77.0, device=DEV)
        ws = kw.pop("ws", self.ws)
        a.update(kw)
        pi.check(pi.pi_tree_attention(self.desc, self.layer, self.S, self.heads, self.mp, self.drafts,
                                      *a.values(), y, lse, self.status, ws, stream=stream),
                 "pi_tree_attention")
        return y, lse

    def check(self, y, lse, seen=None):
        torch.cuda.synchronize()
        y = y.double().cpu().numpy()
        lse = lse.double().cpu().numpy() if lse is not None else None
        G = self.heads // self.kv
        assert (y[self.S] == 77.0).all()
        for s in range(self.S):
            assert (y[s, self.count[s]:] == 77.0).all()  # rows behind the last draft
            assert lse is None or (lse[s, self.count[s]:] == 77.0).all()
            for i in range(self.count[s]):
                for h in range(self.kv):
                    hs = slice(h * G, (h + 1) * G)
                    vis = (seen or self.seen)[s][i]
                    yo, lo, mag, vmax = plain.attention(self.q[s, i, hs].astype(np.float64),
                                                        self.rows[0, s, :, h], self.rows[1, s, :, h],
                                                        vis, self.scale)
                    e = self.scale * mag * (2.0 ** -21 + self.D * U) + 2.0 ** -20 + 2.0 ** -22 + len(vis) * U
                    err = np.abs(y[s, i, hs] - yo).max(1)
                    assert (err <= 3 * e * vmax + 1e-30).all(), (s, i, h, err, 3 * e * vmax)
                    if lse is not None and vis:
                        d = np.abs(lse[s, i, hs] - lo)
                        assert (d <= 2 * e + 4 * U * np.abs(lo)).all(), (s, i, h, d, e)
                    elif lse is not None:
                        assert np.isneginf(lse[s, i, hs]).all()
        if self.append:
            pool = self.pool[self.layer].double().cpu().numpy()
            for s in range(self.S):
                for t in range(self.base[s], self.lens[s]):
                    got = pool[self.np_table[s, t // self.P], :, :, t % self.P]
                    assert (got == self.rows[:, s, t]).all(), (s, t)
        assert int(self.status[0]) == 0


SHAPES = [
    # heads, kv, D, page, base, count, drafts
    (4, 4, 64, 16, [40], None, 5),
    (1, 1, 8, 1, [0, 3, 1], [1, 2, 0], 2),
    (8, 2, 128, 16, [0, 17, 255, 129, 128], [3, 13, 0, 7, 13], 13),
    (6, 3, 80, 24, [100, 131, 5], None, 9),
    (4, 1, 96, 8, [300, 1, 64], [6, 1, 3], 6),
    (2, 2, 256, 32, [70, 200, 129], None, 4),
    (3, 1, 192, 64, [200, 63, 64], None, 33),
    (16, 1, 64, 16, [260, 31], None, 17),
    (16, 2, 128, 128, [1000, 513], [64, 50], 64),
    (64, 4, 32, 16, [90], None, 64),
    (5, 5, 40, 7, [50, 0, 20], [8, 2, 5], 8),
    (2, 1, 72, 16, [33, 150], None, 3),
    (8, 8, 248, 256, [300], None, 2),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", SHAPES)
@pytest.mark.parametrize("shape,append", [("tree", False), ("chain", True), ("tree", True)])
def test_tree_attention(case, dtype, shape, append):
    t = Tree(dtype, *case, shape=shape, append=append, layers=2, layer=1, seed=len(case[4]))
    t.check(*t.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 0), (16, 1), (100, 4), (129, 130), (300, 7), (5, 1000)])
@pytest.mark.parametrize("shape", ["tree", "chain"])
def test_tree_window(dtype, window, sinks, shape):
    t = Tree(dtype, 4, 2, 64, 16, [0, 5, 130, 290, 127], [20, 7, 20, 20, 1], 20, shape=shape, window=window,
             sinks=sinks, append=True, seed=3)
    t.check(*t.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_tree_long(dtype):
    # units that many blocks share, and ragged neighbours
    t = Tree(dtype, 8, 2, 128, 16, [9001, 3, 700], None, 3, seed=5)
    t.check(*t.run())
    t = Tree(dtype, 32, 2, 64, 32, [5000], None, 20, append=True, seed=6)
    t.check(*t.run())


def test_no_lse_and_scales():
    t = Tree("f16", 4, 2, 64, 16, [70], None, 4, seed=7)
    y, _ = t.run()
    z, none = t.run(want_lse=False)
    torch.cuda.synchronize()
    assert none is None and torch.equal(y, z)
    for scale in (-0.3, 0.0):
        t.scale = scale
        yy, lse = t.run()
        t.scale = abs(scale)  # the tolerance's
        t.q = -t.q if scale < 0 else t.q
        t.check(yy, lse)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("qscale", [1e-30, 1e-6, 300.0, 1e6])
def test_query_scales(dtype, qscale):
    t = Tree(dtype, 4, 2, 64, 16, [150], None, 6, qscale=qscale, seed=8)
    t.check(*t.run())


# ------------------------------------------------------------------ sampling
def run_sample(x, dtype="f32", temperature=None, top_k=None, top_p=None, min_p=None, u=None, logprob=True,
               pad=0, ws=None, stream=None):
    """x [rows][vocab] numpy; (tokens, logprobs, status)."""
    R, V = x.shape
    full = torch.full((R, V + pad), float("nan"), device=DEV, dtype=TD[dtype])
    full[:, :V] = torch.from_numpy(np.ascontiguousarray(x)).to(DEV).to(TD[dtype])
    tok = torch.full((R + 1,), 77, dtype=torch.int32, device=DEV)
    lp = torch.full((R + 1,), 77.0, device=DEV) if logprob else None
    status = new_status()
    arg = [None if a is None else f(a) for a, f in ((temperature, f32), (top_k, i32), (top_p, f32),
                                                    (min_p, f32), (u, f32))]
    if ws is None:
        ws = pi.sample_workspace(R, V, DEV)
    pi.check(pi.pi_token_sample(full, dtype, R, V, V + pad, *arg, tok, lp, status, ws, stream=stream),
             "pi_token_sample")
    torch.cuda.synchronize()
    assert int(tok[R]) == 77 and (lp is None or float(lp[R]) == 77.0)
    return tok[:R].cpu().numpy(), None if lp is None else lp[:R].double().cpu().numpy(), int(status[0])


def rounded(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(TD[dtype]).double().numpy()


def draw_rows(g, R, V, dtype, banned=0.0, spread=3.0):
    """Rows with settings of their own whose draws are not on a border."""
    rows = []
    while len(rows) < R:
        x = (g.standard_normal(V) * spread).astype(np.float32)
        x[g.random(V) < banned] = -np.inf
        x[int(g.integers(V))] = spread
        xr = rounded(x[None], dtype)[0]
        s = (np.float32(g.choice([0.0, 0.3, 0.7, 1.0, 1.9])), int(g.choice([-1, 0, 1, 2, 20, 300, 10 ** 6])),
             np.float32(g.choice([0.0, 0.2, 0.5, 0.9, 0.99, 1.0, 1.5])),
             np.float32(g.choice([0.0, 0.0, 0.02, 0.3, 1.0])), np.float32(g.random()))
        tok, lp, margin = plain.sample_row(xr, *(float(v) if i != 1 else v for i, v in enumerate(s)))
        if margin >= 2.0 ** -30:
            rows.append((x, s, tok, lp))
    return rows


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("R,V,pad,banned", [(1, 1, 0, 0.0), (7, 2, 3, 0.0), (64, 100, 0, 0.1), (40, 1001, 1, 0.5),
                                            (24, 8191, 0, 0.0), (6, 50273, 64, 0.0), (3, 128257, 5, 0.01)])
def test_sample(dtype, R, V, pad, banned):
    g = np.random.default_rng(R + V)
    rows = draw_rows(g, R, V, dtype, banned)
    x = np.stack([r[0] for r in rows])
    st = list(zip(*(r[1] for r in rows)))
    tok, lp, status = run_sample(x, dtype, *st, pad=pad)
    assert status == 0
    assert (tok == [r[2] for r in rows]).all()
    want = np.array([r[3] for r in rows])
    assert (np.abs(lp - want) <= 4 * U * (1 + np.abs(want))).all()
    tok2, none, _ = run_sample(x, dtype, *st, logprob=False)
    assert none is None and (tok2 == tok).all()


def test_sample_defaults_off():
    g = np.random.default_rng(2)
    x = g.standard_normal((5, 333)).astype(np.float32)
    u = g.random(5).astype(np.float32)
    tok, lp, status = run_sample(x, u=u)
    for r in range(5):
        want = plain.sample_row(x[r].astype(np.float64), 1.0, 0, 1.0, 0.0, float(u[r]))
        assert want[2] >= 2.0 ** -30 and tok[r] == want[0]
        assert abs(lp[r] - want[1]) <= 4 * U * (1 + abs(want[1]))
    assert status == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("V", [4, 1000, 4096, 70000])
def test_sample_ties(dtype, V):
    # equal logits: token i takes u in [i / n, (i + 1) / n), n what is kept; exact in any order
    n = V // 4 * 4
    for top_k, top_p, keep in [(0, 1.0, V), (n // 2, 1.0, n // 2), (0, 0.5, -(-V // 2)), (n // 2, 0.25, n // 8 if n % 8 == 0 else -(-n // 8)),
                               (0, 0.0, 1), (1, 0.9, 1)]:
        at = sorted({0, keep // 3, keep - 1})
        u = [np.float32((a + 0.5) / keep) for a in at]
        x = np.full((len(at), V), -2.5, np.float32)
        tok, lp, status = run_sample(x, dtype, None, [top_k] * len(at), [top_p] * len(at), None, u)
        assert status == 0 and list(tok) == at, (top_k, top_p)
        assert (np.abs(lp + math.log(keep)) <= 4 * U * (1 + math.log(keep))).all()


def test_sample_many_near_equal():
    # more logits in one bin than are ordered at once, all different and partly equal
    g = np.random.default_rng(9)
    for V, step in [(30000, 2.0 ** -22), (30000, 2.0 ** -16), (200000, 2.0 ** -23)]:
        x = 1.0 + (g.integers(0, 5000, V) * step).astype(np.float32)
        u = [np.float32(0.123), np.float32(0.5), np.float32(0.987), np.float32(0.7)]
        top_k, top_p = [0, V // 3, 0, 7777], [1.0, 0.9, 0.33, 1.0]
        tok, lp, status = run_sample(np.tile(x.astype(np.float32), (4, 1)), "f32", None, top_k, top_p, None, u)
        for r in range(4):
            want = plain.sample_row(x.astype(np.float32).astype(np.float64), 1.0, top_k[r],
                                    float(np.float32(top_p[r])), 0.0, float(u[r]))
            assert want[2] >= 2.0 ** -30 and tok[r] == want[0], (V, r)
        assert status == 0


def test_sample_refused_rows():
    nan, inf = math.nan, math.inf
    x = np.tile(np.float32([0.5, 1.0, -inf, 0.25]), (12, 1))
    x[0, 3], x[1, 0], x[2] = nan, inf, -inf
    T, p, m, u = [1.0] * 12, [1.0] * 12, [0.0] * 12, [0.5] * 12
    T[3], T[4], T[5], u[6], u[7], p[8], p[9], m[10] = -1.0, nan, inf, 1.0, -0.1, nan, -0.5, 1.5
    tok, lp, status = run_sample(x, "f32", T, None, p, m, u)
    assert status == pi.PI_ERR_RANGE
    assert (tok[:11] == -1).all() and np.isnan(lp[:11]).all()
    assert tok[11] == plain.sample_row([0.5, 1.0, -inf, 0.25], 1.0, 0, 1.0, 0.0, 0.5)[0]


def test_sample_extremes():
    inf = math.inf
    big = float(np.float32(3e38))
    x = np.float32([[big, -big, 0.0, 1.0], [-big, -inf, -big, -big], [1e-40, 0.0, -1e-40, -0.0],
                    [5.0, 5.0 - 1e-6, -inf, 4.0]])
    tok, lp, status = run_sample(x, "f32", [1.0, 1.0, 1.0, 1e-38], None, None, None, [0.99, 0.5, 0.6, 0.99])
    assert status == 0 and list(tok) == [0, 2, 3, 0]
    # row 2's order: 1e-40, then 0.0 and -0.0 (equal, by index), -1e-40
    assert np.allclose(lp, [0.0, -math.log(3), -math.log(4), 0.0], atol=1e-6)


def test_sample_frequencies():
    # u on an even grid draws each token as often as its probability says, to one
    V, R = 12, 4096
    x = np.linspace(-1, 2, V).astype(np.float32)
    u = (np.arange(R) / R).astype(np.float32)
    tok, _, _ = run_sample(np.tile(x, (R, 1)), "f32", [0.8] * R, None, None, None, u)
    p = np.exp(x.astype(np.float64) / np.float32(0.8))
    assert (np.abs(np.bincount(tok, minlength=V) - R * p / p.sum()) <= 1.0).all()


# ------------------------------------------------------------------ acceptance
class Accept:
    def __init__(self, S, N, page, longest, layers, kv, D, dtype, seed=0, ragged=True, wide=3):
        g = np.random.default_rng(seed)
        self.S, self.N, self.P = S, N, page
        self.base = g.integers(0, longest + 1, S)
        self.count = g.integers(0, N + 1, S) if ragged else np.full(S, N)
        self.lens = self.base + self.count
        self.parent = [random_parents(g, N) for _ in range(S)]
        for p in self.parent:
            p[1:] = [max(v, 0) if g.random() < 0.9 else v for v in p[1:]]
        self.tokens = g.integers(0, wide, (S, N))
        self.choice = g.integers(-1, wide, (S, N))
        need = -(-self.lens // page)
        self.mp = max(1, int(need.max()))
        pages = int(need.sum()) + 1
        tab = np.full((S, self.mp), -1)
        order = g.permutation(pages)
        at = 0
        for s in range(S):
            tab[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
        self.tab = tab
        self.pool = torch.randn((layers, pages, 2, kv, page, D), device=DEV).to(TD[dtype])
        self.desc = pi.make_cache_desc(layers, pages, kv, D, page, dtype)

        def ints(*shape):
            return torch.full(shape, 77, dtype=torch.int32, device=DEV)
        self.out = [ints(S + 1), ints(S + 1, N), ints(S + 1), ints(S + 1)]
        self.status = new_status()

    def run(self, pool=True, **kw):
        a = dict(parent=i32(self.parent), count=i32(self.count), tokens=i32(self.tokens),
                 choice=i32(self.choice), table=i32(self.tab), len=i32(self.lens),
                 pool=self.pool if pool else None)
        a.update(kw)
        pi.check(pi.pi_tree_accept(self.desc, self.S, self.mp, self.N, *a.values(), *self.out,
                                   self.status), "pi_tree_accept")
        torch.cuda.synchronize()

    def check(self, before, parent=None, count=None):
        ln, path, acc, nxt = (o.cpu().numpy() for o in self.out)
        want = before.clone()
        count = self.count if count is None else count
        for s in range(self.S):
            n = int(count[s])
            par = (parent or self.parent)[s]
            way, c = plain.accept(par, self.tokens[s][:n], self.choice[s])
            base = int(self.lens[s]) - n
            assert list(path[s]) == way + [-1] * (self.N - len(way))
            assert (ln[s], acc[s], nxt[s]) == (base + len(way), len(way), c)
            for j, i in enumerate(way):
                f, t = base + i, base + j
                want[:, self.tab[s, t // self.P], :, :, t % self.P] = \
                    before[:, self.tab[s, f // self.P], :, :, f % self.P]
        assert all((o[self.S] == 77).all() for o in (ln, path, acc, nxt))
        assert torch.equal(self.pool, want)


@pytest.mark.parametrize("args", [(1, 1, 16, 20, 1, 1, 8, "f16"), (5, 13, 16, 40, 3, 2, 64, "bf16"),
                                  (70, 64, 7, 30, 2, 3, 72, "f16"), (3, 33, 1, 9, 2, 1, 256, "bf16"),
                                  (1024, 3, 8, 5, 1, 1, 16, "f16")])
def test_accept(args):
    for seed, wide in ((1, 3), (2, 1)):
        a = Accept(*args, seed=seed, wide=wide)
        before = a.pool.clone()
        a.run()
        a.check(before)
        assert int(a.status[0]) == 0


def test_accept_without_pool_and_defaults():
    a = Accept(4, 9, 16, 40, 2, 2, 64, "f16", seed=3, ragged=False, wide=1)
    before = a.pool.clone()
    a.run(pool=False, parent=None, count=None)
    assert torch.equal(a.pool, before)
    ln, path, acc, nxt = (o.cpu().numpy() for o in a.out)
    for s in range(4):
        way, c = plain.accept(list(range(-1, 8)), a.tokens[s], a.choice[s])
        assert list(path[s][:len(way)]) == way and acc[s] == len(way) and nxt[s] == c


def test_accept_reports_bad_input():
    a = Accept(4, 6, 16, 40, 2, 2, 64, "f16", seed=4, ragged=False, wide=1)
    a.choice[:] = 0
    a.parent = [[-1, 0, 1, 2, 3, 4], [-1, 0, 5, 1, 3, 4], [-1, 0, 0, 0, 0, 0], [-1, 0, 0, 2, 2, 4]]
    a.lens[2] = a.mp * 16 + 1
    before = a.pool.clone()
    tab = a.tab.copy()
    tab[3, (a.lens[3] - 6 + 4) // 16] = 10 ** 6  # draft 4's page, perhaps the whole path's
    a.run(table=i32(tab))
    assert int(a.status[0]) == pi.PI_ERR_INDEX
    ln, path, acc, nxt = (o.cpu().numpy() for o in a.out)
    assert list(path[0]) == [0, 1, 2, 3, 4, 5]
    assert list(path[1]) == [0, 1, 3, 4, 5, -1]  # draft 2's parent counts as -1
    assert (ln[2], acc[2], nxt[2]) == (0, 0, -1) and (path[2] == -1).all()
    assert list(path[3]) == [0, 1, -1, -1, -1, -1]
    for s in (0, 3):  # these paths stay where they are
        for t in range(int(a.lens[s])):
            pg = a.tab[s, t // 16]
            assert torch.equal(a.pool[:, pg], before[:, pg])
