"""The serving operators on the GPU against plain 64-bit forms (servehelp.py).

Tolerances, from the arithmetic the header promises (u = 2^-24):
  * a score a = scale q . k: q keeps at least 22 bits and the sum of D
    products rounds D times, so |da| <= scale |q|.|k| (2^-21 + D u); an
    exponential adds 2^-20 relative; a sum of n terms n u at most.  With
    e = |da| + 2^-20 + n u the weights are off by e relative (numerator and
    denominator), so |dy| <= 3 e max|v| and |dlse| <= 2 e + 4 u |lse|.
  * logits: s = sum exp(x - m) has relative error e = 2^-20 + n u (n u
    bounds any order of summation; terms are positive), and x - m rounds by
    u |x - m|; so a log probability is off by at most 2 e + 4 u (|lp| + R)
    with R = max - min of the finite logits, the entropy by 4 e (1 + log n).
  * whole numbers (tables, lengths, references, pairs, indices) and stored
    16-bit values are equal.
"""
import math

import numpy as np
import pytest
import torch

import activation_sparse_decode_rank_gb300 as pi
import servehelp as plain

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
TD = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    pi.build()


def i32(a):
    return torch.tensor(np.ascontiguousarray(a), dtype=torch.int32, device=DEV)


def new_status():
    return torch.zeros(4, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ attention
class Cache:
    """A one-call attention problem: random pool, every row no slot may see NaN."""

    def __init__(self, dtype, heads, kv_heads, D, page, lens, window=0, sinks=0, append=False,
                 layers=1, layer=0, qscale=1.5, seed=0, pages=None, spare=2):
        g = np.random.default_rng(seed)
        self.__dict__.update(dtype=dtype, heads=heads, kv=kv_heads, D=D, P=page, lens=list(lens),
                             window=window, sinks=sinks, append=append, layer=layer)
        S = len(lens)
        need = [-(-n // page) for n in lens]
        self.mp = max(1, max(need)) + 1
        self.pages = pages or sum(need) + spare
        order = self.pages - 1 - g.permutation(sum(need)) if pages else g.permutation(self.pages)
        tab = np.full((S, self.mp), -7, np.int64)
        at = 0
        for s in range(S):
            tab[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
        self.np_table = tab
        self.pool = torch.empty((layers, self.pages, 2, kv_heads, page, D), dtype=TD[dtype],
                                device=DEV)
        if not pages:
            self.pool.fill_(float("nan"))
        rows = g.standard_normal((2, S, max(list(lens) + [1]), kv_heads, D)).astype(np.float32)
        self.rows = torch.from_numpy(rows).to(TD[dtype]).to(torch.float64).numpy()
        for s, n in enumerate(lens):
            for j in range(need[s]):
                t0, t1 = j * page, min(n, (j + 1) * page)
                blk = torch.from_numpy(self.rows[:, s, t0:t1]).to(TD[dtype]).to(DEV)
                pg = self.pool[layer, int(tab[s, j])]
                pg[:, :, :t1 - t0] = blk.permute(0, 2, 1, 3)
                if window:
                    for t in range(t0, t1):
                        if not (t >= n - window or t < sinks):
                            pg[:, :, t - t0] = float("nan")
        self.q = g.standard_normal((S, heads, D)).astype(np.float32) * np.float32(qscale)
        self.knew = self.vnew = None
        if append:
            new = g.standard_normal((2, S, kv_heads, D)).astype(np.float32)
            self.knew, self.vnew = (torch.from_numpy(new[i]).to(DEV) for i in (0, 1))
            r16 = torch.from_numpy(new).to(TD[dtype]).to(torch.float64).numpy()
            for s, n in enumerate(lens):
                if n:
                    self.rows[:, s, n - 1] = r16[:, s]
                    pg = self.pool[layer, int(tab[s, (n - 1) // page])]
                    pg[:, :, (n - 1) % page] = float("nan")  # not written yet
        self.table, self.len = i32(tab), i32(lens)
        self.scale = D ** -0.5
        self.desc = pi.make_cache_desc(layers, self.pages, kv_heads, D, page, dtype)
        self.ws = pi.cache_workspace(self.desc, S, heads, DEV)
        self.status = new_status()
        self.qd = torch.from_numpy(self.q).to(DEV)

    def run(self, want_lse=True, stream=None, table=None, length=None):
        S = len(self.lens)
        y = torch.full((S + 1, self.heads, self.D), 77.0, device=DEV)
        lse = torch.full((S + 1, self.heads), 77.0, device=DEV) if want_lse else None
        rc = pi.pi_paged_attention(
            self.desc, self.layer, S, self.heads, self.mp, self.qd, self.knew, self.vnew,
            self.table if table is None else table, self.len if length is None else length,
            self.pool, self.scale, self.window, self.sinks, y, lse, self.status, self.ws,
            stream=stream)
        pi.check(rc, "pi_paged_attention")
        return y, lse

    def check(self, y, lse, hidden=None, lens=None):
        torch.cuda.synchronize()
        y = y.double().cpu().numpy()
        lse = lse.double().cpu().numpy() if lse is not None else None
        assert (y[len(self.lens)] == 77.0).all()  # nothing past the end
        G = self.heads // self.kv
        for s, n in enumerate(lens or self.lens):
            for h in range(self.kv):
                q = self.q[s, h * G:(h + 1) * G].astype(np.float64)
                yo, lo, mag = plain.attention(q, self.rows[0, s, :, h], self.rows[1, s, :, h], n,
                                              self.scale, self.window, self.sinks,
                                              (hidden or {}).get(s, ()))
                got = y[s, h * G:(h + 1) * G]
                e = (self.scale * mag * (2.0 ** -21 + self.D * U) + 2.0 ** -20 + n * U)[:, None]
                vmax = np.nanmax(np.abs(self.rows[1, s, :max(n, 1), h]))
                assert np.isfinite(got).all(), (s, h)
                assert (np.abs(got - yo) <= 3 * e * vmax).all(), (s, h, np.abs(got - yo).max())
                if lse is None:
                    continue
                gl = lse[s, h * G:(h + 1) * G]
                assert (np.isneginf(gl) == np.isneginf(lo)).all()
                f = np.isfinite(lo)
                assert (np.abs(gl[f] - lo[f]) <= 2 * e[f, 0] + 4 * U * np.abs(lo[f])).all()

    def check_stored(self):
        """The new rows are in the cache, rounded to its type."""
        for s, n in enumerate(self.lens):
            if n:
                pg = self.pool[self.layer, int(self.np_table[s, (n - 1) // self.P])]
                for kind, src in ((0, self.knew), (1, self.vnew)):
                    assert torch.equal(pg[kind, :, (n - 1) % self.P], src[s].to(TD[self.dtype]))


SHAPES = [  # heads, kv_heads, head_dim, page
    (4, 4, 64, 16), (8, 1, 128, 16), (6, 2, 80, 24), (32, 2, 128, 32), (5, 5, 96, 7),
    (3, 1, 256, 128), (12, 1, 8, 1), (40, 2, 72, 16), (14, 2, 200, 8), (2, 1, 136, 16),
    (4, 2, 96, 48), (18, 2, 112, 64), (64, 4, 256, 16), (33, 1, 64, 32), (4, 2, 40, 16),
    (8, 8, 128, 24), (4, 4, 64, 8), (4, 1, 256, 40), (2, 2, 192, 8),
]
LENS = [0, 1, 15, 16, 17, 33, 64, 100, 257]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("append", [False, True])
def test_attention_matches_64_bits(dtype, shape, append):
    c = Cache(dtype, *shape, LENS, append=append, seed=sum(shape))
    c.check(*c.run())
    assert int(c.status[0]) == 0
    if append:
        c.check_stored()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (33, 3), (100, 40), (300, 9),
                                          (50, 2000000000), (2147483647, 2147483647)])
@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("page", [16, 24, 7])
def test_attention_window_and_first_tokens(dtype, window, sinks, append, page):
    c = Cache(dtype, 8, 2, 64, page, [0, 1, 16, 34, 99, 100, 101, 333], window, sinks, append)
    c.check(*c.run())
    assert int(c.status[0]) == 0


@pytest.mark.parametrize("lens", [[5000], [1, 4099], [3000, 0, 17, 2049, 1]])
@pytest.mark.parametrize("shape", [(1, 1, 64, 16), (8, 1, 128, 64), (16, 2, 128, 48),
                                   (7, 7, 32, 256)])
def test_attention_long_and_ragged(shape, lens):
    for dtype in ("f16", "bf16"):
        c = Cache(dtype, *shape, lens, seed=len(lens))
        c.check(*c.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", [(16, 1, 128, 16), (20, 2, 128, 24), (32, 2, 80, 8), (48, 2, 64, 8),
                                   (71, 1, 64, 16), (128, 8, 64, 16), (24, 2, 96, 7), (18, 2, 32, 16)])
def test_attention_many_heads_per_kv_head(dtype, shape):
    # more than eight query heads per kv head: short, long (joined across
    # blocks) and windowed
    for lens, window, sinks in ((LENS, 0, 0), ([2900, 1, 0, 803, 16], 0, 0), ([2000, 40, 133], 90, 5)):
        c = Cache(dtype, *shape, lens, window, sinks, append=True)
        c.check(*c.run())
        c.check_stored()
        assert int(c.status[0]) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape,lens", [((8, 1, 128, 16), [20011]), ((16, 1, 64, 32), [9000, 0, 3]),
                                        ((4, 2, 256, 8), [1, 7003]), ((3, 3, 96, 7), [5000, 4100]),
                                        ((12, 1, 128, 24), [2500, 11000, 640]), ((2, 2, 8, 16), [12000])])
def test_attention_units_of_many_blocks(dtype, shape, lens):
    # joined in two steps; the counters are left as they were found
    c = Cache(dtype, *shape, lens, seed=9)
    y, lse = c.run()
    c.check(y, lse)
    for _ in range(3):
        y1, l1 = c.run()
        assert torch.equal(y, y1) and torch.equal(lse, l1)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape,window,sinks", [((32, 32, 96, 8), 0, 0), ((64, 32, 128, 16), 0, 0), ((40, 40, 64, 5), 30, 3)])
def test_attention_many_short_units(dtype, shape, window, sinks):
    # more units than blocks, no more than warps, none longer than 64 tokens
    g = np.random.default_rng(6)
    lens = g.integers(1, 64 if not window else 2000, 24).tolist()
    lens[0], lens[7], lens[23] = 0, 1, 63
    c = Cache(dtype, *shape, lens, window, sinks, append=True)
    c.check(*c.run())
    c.check_stored()


def test_attention_many_slots():
    g = np.random.default_rng(4)
    c = Cache("f16", 4, 2, 64, 16, g.integers(0, 40, 1024).tolist())
    c.check(*c.run())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("qscale", [0.0, 1e-30, 1e-6, 200.0, 3e6])
def test_attention_extreme_queries(dtype, qscale):
    # uniform weights, and one weight that takes all; no overflow in the parts
    c = Cache(dtype, 8, 2, 128, 16, [1, 40, 300], qscale=qscale)
    y, lse = c.run()
    if qscale <= 200.0:
        return c.check(y, lse)
    torch.cuda.synchronize()
    # scores differ by far more than their rounding: the largest one's value
    for s, n in enumerate(c.lens):
        for h in range(8):
            a = c.q[s, h].astype(np.float64) @ c.rows[0, s, :n, h // 4].T
            want = c.rows[1, s, int(a.argmax()), h // 4]
            assert np.abs(y[s, h].cpu().numpy() - want).max() <= 2.0 ** -20 * np.abs(want).max()


def test_attention_without_lse_is_the_same_and_repeats_bit_for_bit():
    c = Cache("bf16", 32, 4, 128, 16, [0, 3, 700, 2500, 64])
    y0, l0 = c.run()
    for _ in range(3):
        y1, l1 = c.run()
        assert torch.equal(y0, y1) and torch.equal(l0, l1)
    assert torch.equal(c.run(want_lse=False)[0], y0)


def test_attention_slots_share_pages():
    c = Cache("f16", 8, 2, 64, 16, [100, 100, 100])
    tab = c.np_table.copy()
    tab[1, :5] = tab[0, :5]
    c.rows[:, 1, :80] = c.rows[:, 0, :80]
    c.check(*c.run(table=i32(tab)))


@pytest.mark.parametrize("layer", [0, 2])
def test_attention_reads_its_layer(layer):
    c = Cache("f16", 4, 4, 64, 16, [20, 50], layers=3, layer=layer, append=True)
    c.check(*c.run())
    c.check_stored()
    for other in range(3):
        if other != layer:
            assert torch.isnan(c.pool[other]).all()


@pytest.mark.parametrize("P", [16, 8, 5])
def test_attention_reports_bad_pages_and_lengths(P):
    c = Cache("f16", 8, 2, 64, P, [100, 60, 45])
    tab = c.np_table.copy()
    tab[0, 2], tab[0, 99 // P], tab[2, 0] = c.pages, -1, 2 ** 30
    y, lse = c.run(table=i32(tab), length=i32([100, c.mp * P + 1, 45]))
    hidden = {0: set(range(2 * P, 3 * P)) | set(range(99 // P * P, 100)), 2: set(range(P))}
    c.check(y, lse, hidden, [100, 0, 45])
    assert int(c.status[0]) == pi.PI_ERR_INDEX
    # the workspace is ready for a good call
    c.status.zero_()
    c.check(*c.run())
    assert int(c.status[0]) == 0
    c.status.zero_()
    y, lse = c.run(length=i32([-1, 60, 45]))
    c.check(y, lse, None, [0, 60, 45])
    assert int(c.status[0]) == pi.PI_ERR_INDEX


def test_attention_append_skips_a_bad_page():
    c = Cache("f16", 4, 2, 64, 16, [20, 30], append=True)
    tab = c.np_table.copy()
    tab[0, 1] = -1
    before = c.pool.clone()
    y, lse = c.run(table=i32(tab))
    c.check(y, lse, {0: set(range(16, 20))})
    assert int(c.status[0]) == pi.PI_ERR_INDEX
    pg = int(c.np_table[0, 1])
    assert torch.equal(c.pool[0, pg].isnan(), before[0, pg].isnan())


def test_attention_past_32_bit_offsets():
    # 5.4e9 elements: the pages used are the pool's last ones
    c = Cache("f16", 8, 8, 128, 64, [129, 64, 7], pages=41000, append=True)
    c.check(*c.run())
    c.check_stored()


def test_attention_past_31_bit_rows():
    # 2.15e9 rows: gathered with 64-bit offsets (34 GB, only its last pages touched)
    c = Cache("f16", 256, 256, 8, 256, [300, 5], pages=16_400)
    c.check(*c.run())


def test_attention_wait_times_out_and_returns():
    # a flag that nothing sets: the copy of the first tile is never ordered
    import time
    c = Cache("f16", 4, 4, 64, 16, [200, 100])
    y = torch.zeros((2, 4, 64), device=DEV)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    pi.check(pi.pi_selftest_attention_timeout(c.desc, 2, 4, c.mp, c.qd, c.table, c.len, c.pool, y,
                                              c.status, c.ws, 2_000_000))
    torch.cuda.synchronize()
    assert int(c.status[0]) == pi.PI_ERR_TIMEOUT
    assert time.perf_counter() - t0 < 6.0  # the limit, and the 2 s that copies get to land
    c.status.zero_()
    c.ws.zero_()
    c.check(*c.run())
    assert int(c.status[0]) == 0


def test_all_operators_in_one_graph():
    # captured on a side stream, replayed on changed inputs: as direct calls
    S, H, kv, D, P, mp, V, k = 4, 8, 2, 64, 16, 6, 3000, 5
    pages = 40
    g = np.random.default_rng(8)
    desc = pi.make_cache_desc(1, pages, kv, D, P, "bf16")
    ws, lws = pi.cache_workspace(desc, S, H, DEV), pi.logprob_workspace(S, V, k, DEV)

    def buffers(seed):
        r = np.random.default_rng(seed)
        t = np.full((S, mp), -1)
        length = r.integers(20, 64, S)
        order = iter(r.permutation(pages))
        for s in range(S):
            for j in range(-(-int(length[s]) // P)):
                t[s, j] = next(order)
        f = lambda *sh: torch.from_numpy(r.standard_normal(sh).astype(np.float32)).to(DEV)  # noqa: E731
        return dict(table=i32(t), len=i32(length), parent=i32(r.integers(0, S, S)),
                    q=f(S, H, D), k=f(S, kv, D), v=f(S, kv, D), x=f(S, V) * 3,
                    pool=f(1, pages, 2, kv, P, D).bfloat16(), slot=i32(range(S)), pos=i32([0] * S),
                    tok=i32(r.integers(0, V, S)))

    one = i32([1] * S)
    o = dict(t2=i32(np.zeros((S, mp))), l2=i32([0] * S), ref=i32([0] * pages),
             pairs=i32(np.zeros((pages, 2))), counts=i32([0] * 4), map=i32([0] * pages),
             y=torch.zeros((S, H, D), device=DEV), lse=torch.zeros((S, H), device=DEV),
             lp=torch.zeros(S, device=DEV), ent=torch.zeros(S, device=DEV),
             idx=i32(np.zeros((S, k))), top=torch.zeros((S, k), device=DEV), st=new_status())

    def step(b):
        pi.check(pi.pi_cache_append(desc, 0, S, mp, S, b["slot"], b["pos"], b["v"], b["k"],
                                    b["table"], b["pool"], o["st"]))
        pi.check(pi.pi_cache_fork(desc, S, mp, b["parent"], one, None, b["table"], b["len"], o["t2"],
                                  o["l2"], o["ref"], b["pool"], o["pairs"], o["counts"], o["st"], ws))
        pi.check(pi.pi_paged_attention(desc, 0, S, H, mp, b["q"], b["k"], b["v"], o["t2"], o["l2"],
                                       b["pool"], 0.125, 30, 2, o["y"], o["lse"], o["st"], ws))
        pi.check(pi.pi_cache_compact(desc, S, mp, None, o["t2"], o["l2"], o["t2"], o["ref"], o["map"],
                                     b["pool"], o["pairs"], o["counts"], o["st"], ws))
        pi.check(pi.pi_token_logprobs(b["x"], "f32", S, V, V, b["tok"], k, o["lp"], o["ent"],
                                      o["idx"], o["top"], o["st"], lws))

    live = buffers(1)
    step(live)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(live)
    for seed in (2, 3):
        b = buffers(seed)
        for name, t in b.items():
            live[name].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in o.items()}
        step(b)
        torch.cuda.synchronize()
        assert int(o["st"][0]) == 0
        for n, t in o.items():
            if n == "pairs":
                t, got[n] = t[: int(o["counts"][0])], got[n][: int(o["counts"][0])]
            assert torch.equal(t, got[n]), n
        assert torch.equal(b["pool"], live["pool"])


def test_attention_on_another_stream_and_in_a_graph():
    c = Cache("f16", 8, 2, 64, 16, [200, 0, 31])
    want, _ = c.run()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got, _ = c.run(stream=st)
    st.synchronize()
    assert torch.equal(want, got)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, lse = c.run()
    y.zero_()
    c.len.copy_(i32([150, 5, 31]))  # lengths are read on the device
    c.rows[:, 1, :5] = np.nan_to_num(c.rows[:, 1, :5])
    c.table[1, 0] = int(c.np_table[0, 0])
    g.replay()
    torch.cuda.synchronize()
    c.rows[:, 1, :16] = c.rows[:, 0, :16]
    y[-1] = 77.0
    c.check(y, None, None, [150, 5, 31])


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kv,D,P", [(1, 8, 1), (3, 80, 7), (8, 128, 16), (2, 256, 256)])
@pytest.mark.parametrize("tokens", [0, 1, 37])
def test_append_stores_rounded_rows(dtype, kv, D, P, tokens):
    g = np.random.default_rng(tokens + D)
    S, mp, layers = 3, 2 + 64 // P, 2
    desc = pi.make_cache_desc(layers, S * mp + 1, kv, D, P, dtype)
    pool = torch.full((layers, S * mp + 1, 2, kv, P, D), 3.0, dtype=TD[dtype], device=DEV)
    table = g.permutation(S * mp).reshape(S, mp)
    where = g.permutation(S * mp * P)[:tokens]
    slot, pos = where // (mp * P), where % (mp * P)
    k, v = (torch.randn((tokens, kv, D), device=DEV) * 100 for _ in range(2))
    want = pool.clone()
    for i in range(tokens):
        if i == 5:
            slot[i] = -1
            continue
        pg = int(table[slot[i], pos[i] // P])
        want[1, pg, 0, :, pos[i] % P] = k[i].to(TD[dtype])
        want[1, pg, 1, :, pos[i] % P] = v[i].to(TD[dtype])
    st = new_status()
    args = (i32(slot), i32(pos), k, v) if tokens else (None,) * 4
    pi.check(pi.pi_cache_append(desc, 1, S, mp, tokens, *args, i32(table), pool, st))
    assert torch.equal(pool, want) and int(st[0]) == 0


def test_append_skips_what_is_out_of_range():
    desc = pi.make_cache_desc(1, 8, 2, 16, 4, "f16")
    pool = torch.zeros((1, 8, 2, 2, 4, 16), dtype=torch.float16, device=DEV)
    table = i32([[0, 1, 8], [2, -1, 3]])
    for slot, pos in [(2, 0), (-2, 0), (0, 12), (0, -1), (0, 8), (1, 5)]:
        st = new_status()
        one = torch.ones((1, 2, 16), device=DEV)
        pi.check(pi.pi_cache_append(desc, 0, 2, 3, 1, i32([slot]), i32([pos]), one, one, table,
                                    pool, st))
        assert int(st[0]) == pi.PI_ERR_INDEX
        assert float(pool.abs().sum()) == 0.0


# ------------------------------------------------------------------ pages
def run_fork(P, pages, mp, parent, grow, held, table, length, layers=2, kv=1, D=8, pool=True):
    S = len(parent)
    desc = pi.make_cache_desc(layers, pages, kv, D, P, "f16")
    data = torch.randn((layers, pages, 2, kv, P, D), device=DEV).half() if pool else None
    before = data.clone() if pool else None
    o = dict(table=torch.full((S + 1, mp), 55, dtype=torch.int32, device=DEV),
             len=i32([55] * (S + 1)), ref=i32([55] * (pages + 1)), pairs=i32([[-9, -9]] * (S + 1)),
             counts=i32([-9] * 4))
    st = new_status()
    ws = pi.cache_workspace(desc, S, 0, DEV)
    for _ in range(2):  # the second run finds the workspace as the first left it
        if pool:
            data.copy_(before)
        pi.check(pi.pi_cache_fork(desc, S, mp, i32(parent), i32(grow),
                                  None if held is None else i32(held), i32(table), i32(length),
                                  o["table"], o["len"], o["ref"], data, o["pairs"], o["counts"],
                                  st, ws))
    torch.cuda.synchronize()
    got = {k: v.cpu().tolist() for k, v in o.items()}
    assert got["table"][S] == [55] * mp and got["len"][S] == 55 and got["ref"][pages] == 55
    n = got["counts"][0]
    assert got["counts"][2:] == [-9, -9] and all(p == [-9, -9] for p in got["pairs"][n:])
    if pool:
        for a, b in got["pairs"][:n]:
            before[:, b] = before[:, a]
        assert torch.equal(before, data)
    return dict(table=got["table"][:S], len=got["len"][:S], ref=got["ref"][:pages],
                pairs=[tuple(p) for p in got["pairs"][:n]], live=got["counts"][1]), int(st[0])


def random_tables(g, S, P, pages, mp, share=True):
    """Tables with shared full pages (and shared partly filled ones)."""
    length = g.integers(0, mp * P + 1, S)
    length[g.integers(0, S)] = 0
    numbers = list(g.permutation(pages))
    table = np.full((S, mp), -1, np.int64)
    for s in range(S):
        n = -(-int(length[s]) // P)
        if share and s and g.random() < 0.5:
            u = int(g.integers(0, s))
            m = min(n, -(-int(length[u]) // P))
            table[s, :m] = table[u, :m]
        else:
            m = 0
        for j in range(m, n):
            if not numbers:
                length[s] = j * P
                break
            table[s, j] = numbers.pop()
    return table, length


@pytest.mark.parametrize("seed", range(12))
def test_fork_matches_the_plain_form(seed):
    g = np.random.default_rng(seed)
    S = int(g.choice([1, 3, 8, 40, 200]))
    P = int(g.choice([1, 4, 7, 16]))
    mp = int(g.choice([1, 5, 33, 130]))
    pages = int(S * mp * g.choice([0.5, 0.8, 2.0])) + 2
    table, length = random_tables(g, S, P, pages, mp)
    parent = g.integers(-1, S, S)
    if seed % 3 == 0:
        parent = np.arange(S)
    grow = g.integers(-2 * P, 2 * P + 1, S)
    if seed % 4 == 1:
        grow[:] = 1
    held = None
    if seed % 2:
        held = np.zeros(pages, np.int64)
        held[g.integers(0, pages, 3)] = 2
    want, short = plain.fork(P, pages, mp, parent.tolist(), grow.tolist(),
                             None if held is None else held.tolist(), table.tolist(),
                             length.tolist())
    got, st = run_fork(P, pages, mp, parent, grow, held, table, length, pool=seed % 5 != 4)
    assert got == want
    assert st == (pi.PI_ERR_CAPACITY if short else 0)


def test_fork_large_pool_and_many_slots():
    g = np.random.default_rng(99)
    S, P, mp, pages = 1024, 16, 70, 100_003
    table, length = random_tables(g, S, P, pages, mp)
    parent, grow = g.integers(-1, S, S), g.integers(-3, 40, S)
    held = (g.random(pages) < 0.3).astype(np.int64)
    held[np.unique(table[table >= 0])] = 0
    want, short = plain.fork(P, pages, mp, parent.tolist(), grow.tolist(), held.tolist(),
                             table.tolist(), length.tolist())
    got, st = run_fork(P, pages, mp, parent, grow, held, table, length, layers=1)
    assert got == want and st == (pi.PI_ERR_CAPACITY if short else 0)


def test_fork_steps_of_a_beam():
    # parents of a beam: two children of slot 0, one of slot 2, slot 1 freed;
    # worked by hand
    table = [[4, 1, -1], [0, 2, -1], [4, 5, -1]]
    got, st = run_fork(4, 8, 3, [0, 0, 2], [1, 1, 1], None, table, [6, 7, 8])
    assert st == 0
    assert got["table"] == [[4, 1, -1], [4, 0, -1], [4, 5, 2]]
    assert got["len"] == [7, 7, 9] and got["pairs"] == [(1, 0)]
    assert got["ref"] == [1, 1, 1, 0, 3, 1, 0, 0] and got["live"] == 5


def test_fork_begins_trims_and_frees():
    table = [[3, 0], [1, 2]]
    # slot 0 begins anew with 5 tokens, slot 1 is slot 1 cut to 4 of 8 tokens
    got, st = run_fork(4, 6, 2, [-1, 1], [5, -4], None, table, [8, 8])
    assert st == 0 and got["len"] == [5, 4] and got["table"] == [[0, 2], [1, -1]]
    # everything ends
    got, st = run_fork(4, 6, 2, [-1, -1], [0, -3], None, table, [8, 8])
    assert st == 0 and got["len"] == [0, 0] and got["live"] == 0 and got["ref"] == [0] * 6


def test_fork_runs_out_of_pages():
    # three pages are free: slot 0 takes two, slot 1 one of the two it wants,
    # slot 2 none
    got, st = run_fork(4, 4, 4, [0, -1, -1], [8, 8, 1], None, [[3, -1, -1, -1]] * 3, [4, 0, 0])
    assert st == pi.PI_ERR_CAPACITY
    assert got["table"] == [[3, 0, 1, -1], [2, -1, -1, -1], [-1] * 4]
    assert got["len"] == [12, 4, 0] and got["live"] == 4
    # a slot cannot pass its table's end
    got, st = run_fork(4, 9, 2, [0], [7], None, [[3, -1]], [4])
    assert st == pi.PI_ERR_CAPACITY and got["len"] == [8] and got["table"] == [[3, 0]]


def test_fork_reports_what_is_out_of_range():
    for parent, table, length, keep in [
            ([2, 1], [[0, -1], [1, -1]], [4, 4], [0, 4]),       # no such parent
            ([-2, 1], [[0, -1], [1, -1]], [4, 4], [0, 4]),
            ([0, 1], [[0, -1], [1, -1]], [9, 4], [0, 4]),       # no such length
            ([0, 1], [[0, -1], [1, -1]], [-1, 4], [0, 4])]:
        got, st = run_fork(4, 4, 2, parent, [0, 0], None, table, length)
        assert st == pi.PI_ERR_INDEX and got["len"] == keep and got["table"][1] == [1, -1]
    got, st = run_fork(4, 4, 2, [0, 1], [0, 0], None, [[4, 0], [1, -1]], [8, 4])
    assert st == pi.PI_ERR_INDEX and got["table"] == [[-1, 0], [1, -1]]
    assert got["ref"] == [1, 1, 0, 0]


def run_compact(P, pages, mp, held, table, length, in_place=False, pool=True):
    S, layers = len(length), 2
    desc = pi.make_cache_desc(layers, pages, 1, 8, P, "bf16")
    data = torch.randn((layers, pages, 2, 1, P, 8), device=DEV).bfloat16() if pool else None
    before = data.clone() if pool else None
    tin = i32(table)
    tout = tin if in_place else torch.full((S, mp), 55, dtype=torch.int32, device=DEV)
    ref, where = i32([55] * (pages + 1)), i32([55] * (pages + 1))
    pairs, counts, st = i32([[-9, -9]] * (pages // 2 + 1)), i32([-9] * 4), new_status()
    ws = pi.cache_workspace(desc, S, 0, DEV)
    for r in range(1 if in_place else 2):
        if pool:
            data.copy_(before)
        pi.check(pi.pi_cache_compact(desc, S, mp, None if held is None else i32(held), tin,
                                     i32(length), tout, ref, where, data, pairs, counts, st, ws))
    torch.cuda.synchronize()
    c, ref, where = counts.tolist(), ref.tolist(), where.tolist()
    assert c[2:] == [-9, -9] and ref[pages] == 55 and where[pages] == 55
    pl = [tuple(p) for p in pairs.tolist()]
    assert all(p == (-9, -9) for p in pl[c[0]:])
    if pool:
        for a, b in pl[:c[0]]:
            before[:, b] = before[:, a]
        assert torch.equal(before, data)
    return dict(table=tout.tolist(), ref=ref[:pages], map=where[:pages], pairs=pl[:c[0]],
                live=c[1]), int(st[0])


@pytest.mark.parametrize("seed", range(10))
def test_compact_matches_the_plain_form(seed):
    g = np.random.default_rng(100 + seed)
    S = int(g.choice([1, 2, 9, 64]))
    P, mp = int(g.choice([1, 5, 16])), int(g.choice([1, 6, 60]))
    pages = int(S * mp * g.choice([0.6, 1.0, 4.0])) + 1
    table, length = random_tables(g, S, P, pages, mp)
    held = (g.random(pages) < 0.1).astype(np.int64) * 3 if seed % 2 else None
    want = plain.compact(P, pages, mp, None if held is None else held.tolist(), table.tolist(),
                         length.tolist())
    got, st = run_compact(P, pages, mp, held, table, length, in_place=seed % 3 == 2,
                          pool=seed % 4 != 3)
    assert got == want and st == 0


def test_compact_large_pool():
    g = np.random.default_rng(7)
    S, P, mp, pages = 300, 16, 90, 70_001
    table, length = random_tables(g, S, P, pages, mp)
    want = plain.compact(P, pages, mp, None, table.tolist(), length.tolist())
    got, st = run_compact(P, pages, mp, None, table, length)
    assert got == want and st == 0


def test_compact_nothing_live_and_nothing_to_move():
    got, st = run_compact(4, 6, 2, None, [[5, 3]], [0])
    assert st == 0 and got["live"] == 0 and got["table"] == [[-1, -1]] and got["map"] == [-1] * 6
    got, st = run_compact(4, 6, 2, None, [[1, 0]], [8])
    assert st == 0 and got["pairs"] == [] and got["table"] == [[1, 0]] and got["live"] == 2
    got, st = run_compact(4, 6, 2, None, [[6, 5], [-1, 4]], [8, 4])
    assert st == pi.PI_ERR_INDEX and got["table"] == [[-1, 0], [-1, -1]] and got["live"] == 1


def test_copy_pairs():
    desc = pi.make_cache_desc(3, 10, 2, 24, 5, "f16")
    pool = torch.randn((3, 10, 2, 2, 5, 24), device=DEV).half()
    want = pool.clone()
    for a, b in [(0, 9), (3, 4), (3, 5)]:
        want[:, b] = want[:, a]
    st = new_status()
    pairs = i32([[0, 9], [3, 4], [3, 5], [1, 2]])
    pi.check(pi.pi_cache_copy(desc, pairs, i32([3]), 4, pool, st))
    assert torch.equal(pool, want) and int(st[0]) == 0
    pi.check(pi.pi_cache_copy(desc, pairs, i32([4]), 3, pool, st))
    assert torch.equal(pool, want) and int(st[0]) == pi.PI_ERR_CAPACITY
    st.zero_()
    pi.check(pi.pi_cache_copy(desc, i32([[10, 1], [1, -1]]), i32([2]), 2, pool, st))
    assert torch.equal(pool, want) and int(st[0]) == pi.PI_ERR_INDEX


# ------------------------------------------------------------------ scoring
def run_score(x, dtype, tokens, topk, pad=0, want_entropy=True):
    R, V = x.shape
    full = torch.full((R, V + pad), 9e4 if dtype != "f16" else 6e4, dtype=TD[dtype], device=DEV)
    full[:, :V] = torch.from_numpy(x).to(TD[dtype])
    lp = torch.full((R + 1,), 77.0, device=DEV) if tokens is not None else None
    ent = torch.full((R + 1,), 77.0, device=DEV) if want_entropy else None
    idx = i32([[77] * topk] * (R + 1)) if topk else None
    top = torch.full((R + 1, topk), 77.0, device=DEV) if topk else None
    st = new_status()
    ws = pi.logprob_workspace(R, V, topk, DEV)
    outs = []
    for _ in range(2):
        pi.check(pi.pi_token_logprobs(full, dtype, R, V, V + pad,
                                      None if tokens is None else i32(tokens), topk, lp, ent, idx,
                                      top, st, ws))
        torch.cuda.synchronize()
        outs.append([None if t is None else t.clone() for t in (lp, ent, idx, top)])
    for a, b in zip(*outs):  # bit for bit
        assert a is None or torch.equal(a.view(torch.int32), b.view(torch.int32))
    for t in (lp, ent, idx, top):
        assert t is None or (t[R] == 77).all()
    return [None if t is None else t[:R].double().cpu().numpy() for t in (lp, ent, idx, top)], \
        int(st[0])


def check_score(x, dtype, tokens, topk, pad=0):
    x16 = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(TD[dtype]).double().numpy()
    (lp, ent, idx, top), st = run_score(np.ascontiguousarray(x, np.float32), dtype, tokens, topk,
                                        pad)
    n = x.shape[1]
    e = 2.0 ** -20 + n * U
    for r in range(x.shape[0]):
        wl, we, wi, wt = plain.score_row(x16[r], -1 if tokens is None else tokens[r], topk)
        fin = x16[r][np.isfinite(x16[r])]
        R = fin.max() - fin.min() if fin.size else 0.0

        def near(got, want, tol):
            if math.isnan(want):
                return math.isnan(got)
            return got == want if math.isinf(want) else abs(got - want) <= tol
        if tokens is not None:
            assert near(lp[r], wl, 2 * e + 4 * U * (abs(wl) + R) if np.isfinite(wl) else 0), r
        assert near(ent[r], we, 4 * e * (1 + math.log(n)) + 4 * U * R), (r, ent[r], we)
        if topk:
            assert idx[r].astype(int).tolist() == wi, r
            for a, b in zip(top[r], wt):
                assert near(a, b, 2 * e + 4 * U * (abs(b) + R) if np.isfinite(b) else 0)
    return st


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,pad,topk", [
    (1, 1, 0, 1), (3, 2, 1, 2), (5, 31, 0, 5), (2, 32, 0, 32), (9, 1000, 3, 20), (4, 4099, 0, 32),
    (1, 50273, 5, 20), (40, 513, 0, 0), (300, 777, 0, 8), (2, 200001, 0, 32), (1, 1, 0, 0),
    (600, 2500, 1, 3)])
def test_scores_match_64_bits(dtype, rows, vocab, pad, topk):
    g = np.random.default_rng(rows + vocab)
    x = g.standard_normal((rows, vocab)) * 3
    tok = g.integers(0, vocab, rows)
    tok[rows // 2] = -1
    assert check_score(x, dtype, tok.tolist(), topk, pad) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 200])
def test_scores_of_ties_sorted_rows_and_banned_tokens(dtype, rows):
    V, k = 9001, 32
    g = np.random.default_rng(5)
    same = np.zeros((rows, V))
    up = np.tile(np.arange(V) / 64.0, (rows, 1))
    few = g.integers(0, 3, (rows, V)).astype(float)
    blocky = np.where(np.arange(V)[None, :] % 512 < 16, 5.0, -5.0) + np.zeros((rows, 1))
    signed_zero = np.where(g.random((rows, V)) < 0.5, 0.0, -0.0)
    banned = g.standard_normal((rows, V))
    banned[:, g.random(V) < 0.999] = -np.inf
    for x in (same, up, up[:, ::-1], few, blocky, signed_zero, banned):
        assert check_score(x, dtype, [V // 3] * rows, k) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab,pad,topk", [(701, 0, 20), (5003, 5, 32), (33_000, 0, 7)])
def test_scores_of_many_rows(dtype, vocab, pad, topk):
    # more rows than the GPU holds blocks: random, rising, tied and banned rows
    # in turn; every 37th is compared
    R, g = 2100, np.random.default_rng(vocab)
    x = g.standard_normal((R, vocab)).astype(np.float32) * 3
    x[1::5] = np.arange(vocab) / 64.0
    x[2::5] = np.round(x[2::5])
    x[3::5, g.random(vocab) < 0.98] = -np.inf
    tok = g.integers(0, vocab, R)
    (lp, ent, idx, top), st = run_score(x, dtype, tok.tolist(), topk, pad)
    assert st == 0
    e = 2.0 ** -20 + vocab * U
    for r in range(0, R, 37):
        x16 = torch.from_numpy(x[r]).to(TD[dtype]).double().numpy()
        wl, we, wi, wt = plain.score_row(x16, int(tok[r]), topk)
        f = x16[np.isfinite(x16)]
        tol = 2 * e + 8 * U * (f.max() - f.min() + 20)
        assert idx[r].astype(int).tolist() == wi, r
        assert lp[r] == wl or abs(lp[r] - wl) <= tol
        assert abs(ent[r] - we) <= 4 * e * (1 + math.log(vocab)) + 4 * U * (f.max() - f.min())
        for a, b in zip(top[r], wt):
            assert a == b or abs(a - b) <= tol


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_scores_of_odd_rows(dtype):
    V = 3001
    g = np.random.default_rng(6)
    x = g.standard_normal((7, V))
    x[0] = -np.inf                       # nothing is left
    x[1] = -np.inf
    x[1, 2999] = 4.0                     # one token is left
    x[2, 77] = np.nan
    x[3, 5] = np.inf
    x[4] *= 1e4                          # one token takes all
    x[5] = -6e4
    x[6, 1500:] = np.nan
    assert check_score(x, dtype, [3, 2999, 77, 5, 9, 0, 1], 20, pad=2) == 0


def test_scores_report_tokens_out_of_range():
    x = np.random.default_rng(1).standard_normal((3, 100)).astype(np.float32)
    (lp, ent, _, _), st = run_score(x, "f32", [100, 5, -2], 0)
    assert st == pi.PI_ERR_INDEX and math.isnan(lp[0]) and math.isnan(lp[2])
    assert abs(lp[1] - plain.score_row(x[1], 5, 0)[0]) < 1e-4 and np.isfinite(ent).all()


def test_scores_without_some_outputs():
    x = np.random.default_rng(2).standard_normal((4, 500)).astype(np.float32)
    (lp, ent, idx, top), _ = run_score(x, "f32", [1, 2, 3, 4], 6)
    (l2, e2, i2, t2), _ = run_score(x, "f32", None, 6, want_entropy=False)
    assert l2 is None and e2 is None and (i2 == idx).all() and (t2 == top).all()
    (l3, e3, _, _), _ = run_score(x, "f32", [1, 2, 3, 4], 0)
    assert (l3 == lp).all() and (e3 == ent).all()


def test_scores_past_32_bit_offsets():
    R, V = 35_000, 128_000  # 4.48e9 elements
    x = torch.zeros((R, V), dtype=torch.bfloat16, device=DEV)
    x[-1, 127_999] = 9.0
    x[-2, 64_000] = 8.0
    tok = torch.full((R,), 127_999, dtype=torch.int32, device=DEV)
    lp, ent = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
    idx = torch.empty((R, 1), dtype=torch.int32, device=DEV)
    top = torch.empty((R, 1), device=DEV)
    st = new_status()
    pi.check(pi.pi_token_logprobs(x, "bf16", R, V, V, tok, 1, lp, ent, idx, top, st,
                                  pi.logprob_workspace(R, V, 1, DEV)))
    assert idx[-1, 0] == 127_999 and idx[-2, 0] == 64_000 and idx[0, 0] == 0
    z = math.log(V - 1 + math.exp(9.0))
    assert abs(float(lp[-1]) - (9.0 - z)) < 1e-3 and abs(float(lp[0]) + math.log(V)) < 1e-3


def test_empty_batches():
    st = new_status()
    ws = pi.logprob_workspace(0, 10, 0, DEV)
    assert pi.pi_token_logprobs(None, "f32", 0, 10, 10, None, 0, None, None, None, None, st,
                                ws) == 0


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("beams,window,sinks", [(1, 0, 0), (4, 0, 0), (5, 17, 3)])
def test_beam_search_scores_hold_without_a_cache(beams, window, sinks):
    # The example's beams: each sequence's log probability, summed step by step
    # over forked caches, is that of one pass over the whole sequence.  Both
    # sides use the same projections and FFN calls; keys, values and scores
    # differ by fp32 rounding (2^-23 of sums of some hundred terms, three
    # layers), but a neuron whose predictor logit lies within that of zero may
    # switch, which moves a logit by its contribution (under 1e-2 here).
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                    "examples"))
    import beam_decode as ex
    model = ex.Decoder(seed=3)
    prompt = torch.randint(0, ex.VOCAB, (37,), generator=torch.Generator().manual_seed(beams))
    search = ex.BeamSearch(model, beams, 37 + 30, window, sinks)
    tokens, score = search.run(prompt, 30)
    assert int(search.status[0]) == 0 and int(model.status[0]) == 0
    assert (score[:-1] >= score[1:]).all() and len({tuple(t) for t in tokens.tolist()}) == beams
    for b in range(beams):
        assert abs(float(score[b]) - ex.rescore(model, tokens[b], 37, window, sinks)) <= 5e-2
    # after compaction the slots read what they read before
    before = [search.pool[:, search.table[search.now][b, :5].long()].clone() for b in range(beams)]
    n = int(search.length[search.now][0])
    assert n == 66
    live = search.compact()
    t = search.table[search.now]
    assert live == len(set(t.flatten().tolist()) - {-1}) and int(t.max()) < live
    for b in range(beams):
        after = search.pool[:, t[b, :5].long()]
        full = after.permute(0, 1, 4, 2, 3, 5).reshape(ex.LAYERS, -1, 2, 2, 32)[:, :n]
        was = before[b].permute(0, 1, 4, 2, 3, 5).reshape(ex.LAYERS, -1, 2, 2, 32)[:, :n]
        assert torch.equal(full, was)
