"""The operators of include/pi_draft.h at the ends of what their header allows:
waits that run out, extreme temperatures and queries, sums that have to be exact,
shared workspaces, more rows than a launch has blocks."""
import math

import numpy as np
import pytest
import torch

import activation_sparse_decode_rank_gb300 as pi
import drafthelp as plain
from test_gpu_draft import DEV, U, Tree, f32, i32, new_status, rounded, run_sample
from test_gpu_serve import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    pi.build()


# ------------------------------------------------------------------ waits that run out
def lose_copy(t, limit_ns):
    """The self-test on t's problem: (status, milliseconds)."""
    y = torch.empty((t.S, t.drafts, t.heads, t.D), device=DEV)
    status = new_status()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    pi.check(pi.pi_selftest_tree_timeout(t.desc, t.S, t.heads, t.mp, t.drafts, t.qd, t.table, t.len, t.pool, y,
                                         status, t.ws, limit_ns), "pi_selftest_tree_timeout")
    end.record()
    torch.cuda.synchronize()
    return int(status[0]), start.elapsed_time(end)


@pytest.mark.parametrize("args,drafts", [(("f16", 8, 2, 128, 16), 4), (("bf16", 64, 2, 128, 16), 16),
                                         (("f16", 64, 2, 64, 32), 40), (("bf16", 4, 1, 256, 8), 16)])
def test_waits_run_out_at_once(args, drafts):
    # a limit of a microsecond: the block leaves while copies and products are under way
    t = Tree(*args, [300, 200], None, drafts, shape="chain", seed=21)
    got, ms = lose_copy(t, 1000)
    assert got == pi.PI_ERR_TIMEOUT and ms < 6000
    t.check(*t.run())  # the next call is as ever


@pytest.mark.parametrize("args,lens,drafts", [
    (("f16", 1, 1, 64, 16), [2047], 1),                 # a block's share may be a fixed cost alone
    (("bf16", 8, 2, 128, 16), [5000, 7], 4),
    (("f16", 64, 2, 128, 64), [4000, 0, 900], 32),
    (("bf16", 4, 1, 256, 8), [3000, 1], 16)])
def test_lost_copy_of_a_shared_unit(args, lens, drafts):
    t = Tree(*args, lens, None, drafts, shape="chain", seed=24)
    got, ms = lose_copy(t, 2_000_000)
    assert got == pi.PI_ERR_TIMEOUT and ms < 6000
    t.check(*t.run())  # the next call is as ever


# ------------------------------------------------------------------ queries
# (bf16 below 2^-110 keeps fewer bits by the header: its third part would lie below 2^-133)
@pytest.mark.parametrize("shape", [(8, 2, 128, 16), (32, 1, 64, 16), (4, 1, 256, 8)])
@pytest.mark.parametrize("dtype,log2", [("f16", -121), ("f16", -105), ("f16", 108), ("f16", 119), ("bf16", -105),
                                        ("bf16", 108), ("bf16", 119)])
def test_small_and_large_queries_with_a_scale_to_match(dtype, shape, log2):
    # the scores are of the size of any others
    qscale = 2.0 ** log2
    t = Tree(dtype, *shape, [200, 20], None, 6, qscale=qscale, seed=29)
    t.scale = float(np.float32(1 / qscale / shape[2] ** 0.5))
    t.check(*t.run())


# ------------------------------------------------------------------ sampling
def test_sample_more_rows_than_a_grid():
    # past 2^20 rows a block takes several; each row has settings of its own
    R, V = (1 << 20) + 777, 3
    g = np.random.default_rng(22)
    x = g.integers(-1, 2, (R, V)).astype(np.float32)
    u = g.random(R).astype(np.float32)
    T = g.choice(np.float32([0.0, 1.0]), R)
    tok, lp, status = run_sample(x, "f32", T, None, None, None, u)
    order = np.argsort(-x, axis=1, kind="stable")
    w = np.exp(np.take_along_axis(x, order, 1).astype(np.float64))
    w[T == 0, 1:] = 0.0
    sums = np.cumsum(w, 1)
    goal = u.astype(np.float64)[:, None] * sums[:, -1:]
    at = (sums <= goal).sum(1)
    clear = (np.abs(sums - goal) > 2.0 ** -30 * sums[:, -1:]).all(1)
    assert status == 0 and clear.sum() > R - 10
    want = np.take_along_axis(order, at[:, None], 1)[:, 0]
    assert (tok == want)[clear].all()
    wl = np.log(np.take_along_axis(w, at[:, None], 1)[:, 0] / sums[:, -1])
    assert (np.abs(lp - wl) <= 4 * 2.0 ** -24 * (1 + np.abs(wl)))[clear].all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sample_large_temperatures(dtype):
    # finite logits further apart than the largest float, temperatures as large
    g = np.random.default_rng(23)
    R, V = 48, 64
    x = np.zeros((R, V), np.float32)
    T = np.zeros(R, np.float32)
    for r in range(R):
        x[r] = g.uniform(-3.3e38, 3.3e38, V)
        x[r, :2] = 3e38, -3e38
        T[r] = g.choice([2.0 ** 60, 2.0 ** 64, 2.0 ** 65, 1e30, 1e36, 1e37, 1e38, 3e38, 3.4028235e38])
        if T[r] < 1e36:
            x[r] = x[r] / np.float32(3e38) * T[r] * 5
    x[0], x[1], x[2] = -1e38, -1e38, -1e38
    x[:3, 7], x[:3, 9] = 3e38, -3e38
    T[:3] = 1e38, 3e38, 3e38
    k = g.choice([0, 0, 5, 40], R)
    p = g.choice(np.float32([1.0, 1.0, 0.8]), R)
    m = g.choice(np.float32([0.0, 0.0, 0.1, 0.2]), R)
    u = g.random(R).astype(np.float32)
    u[:3], k[:3], p[:3], m[:3] = 0.99999, 0, 1.0, [0.0, 0.1, 0.2]
    tok, lp, status = run_sample(x, dtype, T, k, p, m, u)
    xr = rounded(x, dtype)
    checked = 0
    for r in range(R):
        want = plain.sample_row(xr[r], float(T[r]), int(k[r]), float(p[r]), float(m[r]), float(u[r]))
        if want[2] >= 2.0 ** -30:
            checked += 1
            assert tok[r] == want[0], (r, T[r])
            assert abs(lp[r] - want[1]) <= 4 * U * (1 + abs(want[1]))
    assert status == 0 and checked >= 40


def half_row(g, V):
    """Weights whose sum is 2 (1 + e), 2^-33.6 < e < 2^-32.9: the first logit weighs 1, the
    second about 0.95, one logit in every 32nd of an octave from 2^-10 down to 2^-62 the
    rest; what is not listed is -infinity.  A draw (or an end of top-p) of 0.5 lies e
    behind the first logit's end, so it takes the second, while sums that are 2^-32 short
    take the first."""
    while True:
        t = (10 + (np.arange(52 * 32) + g.random(52 * 32)) / 32) * -math.log(2.0)
        x = np.concatenate([[0.0, 0.0], t]).astype(np.float32)
        tail = np.exp(x[2:].astype(np.float64)).sum()
        x[1] = np.float32(math.log(1 - tail))
        e = (math.exp(float(x[1])) + tail - 1) / 2
        if 2.0 ** -33.6 < e < 2.0 ** -32.9:
            break
    where = g.permutation(V)[:len(x)]
    row = np.full(V, -np.inf, np.float32)
    row[where] = x
    return row, x, where


@pytest.mark.parametrize("V", [2500, 128256, 2000003, (1 << 24) - 3])
def test_sample_small_weights_count(V):
    # exact sums whatever the vocabulary: a border within 2^-33 of the draw, the tail's
    # weights down to 2^-62 of the largest
    g = np.random.default_rng(V)
    for top_p, u in ((1.0, 0.5), (0.5, 0.999)):
        row, x, where = half_row(g, V)
        want = plain.sample_row(x, 1.0, 0, top_p, 0.0, u)
        assert want[0] == 1 and want[2] > 2.0 ** -35
        tok, lp, status = run_sample(row[None], "f32", None, None, [top_p], None, [u])
        assert status == 0 and tok[0] == where[1]
        assert abs(lp[0] - want[1]) <= 4 * U * (1 + abs(want[1]))


@pytest.mark.parametrize("V", [2500, (1 << 24) - 3])
def test_sample_small_weights_count_in_a_list(V):
    # few logits kept: a list, whose weights are as exact; top-k keeps 1000 of 2^-10 and less
    g = np.random.default_rng(V + 1)
    while True:
        x = np.concatenate([[0.0, 0.0], -math.log(2.0) * (10 + np.arange(998) / 32 + g.random(998) / 32)])
        x = x.astype(np.float32)
        tail = np.exp(x[2:].astype(np.float64)).sum()
        x[1] = np.float32(math.log(1 - tail))
        e = (math.exp(float(x[1])) + tail - 1) / 2
        if 2.0 ** -33.6 < e < 2.0 ** -32.9:
            break
    row = np.full(V, -100.0, np.float32)  # not kept
    where = g.permutation(V)[:1000]
    row[where] = x
    for top_p, u in ((1.0, 0.5), (0.5, 0.999)):
        want = plain.sample_row(x, 1.0, 0, top_p, 0.0, u)
        assert want[0] == 1 and want[2] > 2.0 ** -35
        tok, lp, status = run_sample(row[None], "f32", None, [1000], [top_p], None, [u])
        assert status == 0 and tok[0] == where[1]
        assert abs(lp[0] - want[1]) <= 4 * U * (1 + abs(want[1]))


# ------------------------------------------------------------------ workspaces
@pytest.mark.parametrize("fill", [0, 1])
def test_one_workspace_for_every_call(fill):
    # tree attention between calls whose counters lie at the workspace's start
    tree = [Tree("f16", 8, 2, 128, 16, [9001, 3, 700], None, 3, seed=25),
            Tree("bf16", 32, 2, 64, 32, [5000], None, 20, append=True, seed=26)]
    cache = Cache("f16", 8, 2, 64, 16, [6000, 3, 40], seed=27)
    g = np.random.default_rng(28)
    V, S = 60000, 3
    x, tok = f32(g.standard_normal((2, V))), i32([5, V - 1])
    u = f32(g.random(2))
    own = [t.ws for t in tree] + [cache.ws, pi.logprob_workspace(2, V, 4, DEV)]
    ws = torch.zeros(max(w.numel() * w.element_size() for w in own), dtype=torch.uint8, device=DEV)
    if fill:  # beyond the counters it may hold anything
        ws[8192:] = 0xff

    def ints(*shape):
        return torch.full(shape, 77, dtype=torch.int32, device=DEV)

    def calls(shared):
        out = []
        for k, t in enumerate(tree + tree[:1]):
            out += t.run(ws=ws if shared else t.ws)
            cache.ws = ws if shared else own[2]
            out += cache.run()
            lp, ent, idx, top = (torch.zeros(2, device=DEV), torch.zeros(2, device=DEV), ints(2, 4),
                                 torch.zeros((2, 4), device=DEV))
            pi.check(pi.pi_token_logprobs(x, "f32", 2, V, V, tok, 4, lp, ent, idx, top, cache.status,
                                          ws if shared else own[3]), "pi_token_logprobs")
            drawn = ints(2)
            pi.check(pi.pi_token_sample(x, "f32", 2, V, V, None, None, None, None, u, drawn, lp, cache.status,
                                        ws if shared else own[3]), "pi_token_sample")
            table, length, ref, pairs, counts = (ints(S, cache.mp), ints(S), ints(cache.pages), ints(S, 2),
                                                 ints(4))
            pi.check(pi.pi_cache_fork(cache.desc, S, cache.mp, i32([0, 0, 2]), i32([-1, 0, 5]), None, cache.table,
                                      cache.len, table, length, ref, None, pairs, counts, cache.status,
                                      ws if shared else own[2]), "pi_cache_fork")
            out += [lp, ent, idx, top, drawn, table, length, ref, counts[:2]]
        torch.cuda.synchronize()
        return out
    want, got = calls(False), calls(True)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    tree[0].check(*got[:2])
    cache.check(*got[2:4])
    assert int(ws[:8192].sum()) == 0
