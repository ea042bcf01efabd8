"""The serving operators without a GPU: every entry point of
include/pi_serve.h is exported and bound, bad arguments are refused on the
host before any launch, and the plain forms the GPU tests compare with agree
with hand-worked and brute-force results."""
import os
import re

import numpy as np
import pytest

import activation_sparse_decode_rank_gb300 as pi
import servehelp as plain

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 40  # stand-in address: every call below is refused before a launch


@pytest.fixture(scope="module", autouse=True)
def _built():
    pi.build()


def test_exports_and_bindings():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "pi_serve.h")).read(),
                 flags=re.S)
    names = sorted(set(re.findall(r"\b(pi_[a-z_]+)\s*\(", src)))
    assert len(names) == 9
    for n in names:
        assert hasattr(pi.lib(), n) and n in pi.SIGNATURES and callable(getattr(pi, n))


BAD_CACHES = [dict(layers=0), dict(layers=257), dict(pages=0), dict(pages=(1 << 26) + 1),
              dict(kv_heads=0), dict(kv_heads=257), dict(head_dim=12), dict(head_dim=264),
              dict(head_dim=0), dict(page_tokens=0), dict(page_tokens=257)]


def cache(**kw):
    a = dict(layers=2, pages=100, kv_heads=4, head_dim=64, page_tokens=16, dtype="f16")
    a.update(kw)
    return pi.make_cache_desc(**a)


def test_workspace_sizes():
    c = cache()
    assert pi.pi_cache_workspace_size(c, 4, 8) % 256 == 0 and pi.pi_cache_workspace_size(c, 4, 8) > 0
    for bad in BAD_CACHES + [dict(dtype="f32")]:
        assert pi.pi_cache_workspace_size(cache(**bad), 4, 0) == 0
    for slots, heads in [(0, 8), (1025, 8), (4, 6), (4, -4), (4, 2048)]:
        assert pi.pi_cache_workspace_size(c, slots, heads) == 0
    assert pi.pi_logprob_workspace_size(4, 100, 5) > 0
    for bad in [(-1, 100, 5), (4, 0, 0), (4, 100, 33), (4, 100, -1), (4, 3, 4),
                (4, (1 << 24) + 1, 5)]:
        assert pi.pi_logprob_workspace_size(*bad) == 0
    with pytest.raises(pi.PiError):
        pi.cache_workspace(cache(pages=0), 4, 8)
    with pytest.raises(pi.PiError):
        pi.logprob_workspace(4, 0, 0)


def attention(c=None, **kw):
    a = dict(layer=0, slots=4, heads=8, max_pages=10, q=P, k_new=None, v_new=None, table=P, len=P,
             pool=P, scale=0.125, window=0, sinks=0, y=P, lse=P, dev_status=P, ws=P)
    a.update(kw)
    c = c or cache()
    return pi.pi_paged_attention(c, *a.values(), pi.pi_cache_workspace_size(c, 4, 8)
                                 if "wsb" not in kw else kw["wsb"], stream=0)


def refused(call, rows):
    for want, kw in rows:
        assert call(**kw) == want, kw


def test_attention_refusals():
    refused(attention, [
        (pi.PI_ERR_NULL, {k: None}) for k in ("q", "table", "len", "pool", "y", "dev_status", "ws")
    ] + [(pi.PI_ERR_ALIGN, {k: P + 4}) for k in ("q", "table", "len", "pool", "y", "lse", "ws",
                                                  "dev_status")]
        + [(pi.PI_ERR_SHAPE, kw) for kw in (
            dict(layer=-1), dict(layer=2), dict(slots=0), dict(slots=1025), dict(heads=0),
            dict(heads=6), dict(heads=2048), dict(max_pages=0), dict(max_pages=1 << 27),
            dict(window=-1), dict(sinks=-1))]
        + [(pi.PI_ERR_NULL, dict(k_new=P)), (pi.PI_ERR_NULL, dict(v_new=P)),
           (pi.PI_ERR_ALIGN, dict(k_new=P + 8, v_new=P))])
    for bad in BAD_CACHES:
        assert attention(cache(**bad)) == pi.PI_ERR_SHAPE
    assert attention(cache(dtype="f32")) == pi.PI_ERR_DTYPE
    c = cache()
    assert pi.pi_paged_attention(c, 0, 4, 8, 10, P, None, None, P, P, P, 1.0, 0, 0, P, None, P, P,
                                 pi.pi_cache_workspace_size(c, 4, 8) - 1,
                                 stream=0) == pi.PI_ERR_WORKSPACE


def test_attention_selftest_refusals():
    def f(c, limit, wsb=None):
        size = pi.pi_cache_workspace_size(c, 4, 8) if wsb is None else wsb
        return pi.pi_selftest_attention_timeout(c, 4, 8, 10, P, P, P, P, P, P, P, limit, size, stream=0)
    assert f(cache(), 10) == pi.PI_ERR_SHAPE and f(cache(), 6 * 10 ** 9) == pi.PI_ERR_SHAPE
    assert f(cache(), 10 ** 6, 0) == pi.PI_ERR_WORKSPACE
    for c in (cache(dtype="bf16"), cache(head_dim=128), cache(page_tokens=8)):
        assert f(c, 10 ** 6) == pi.PI_ERR_SHAPE


def append(c=None, **kw):
    a = dict(layer=0, slots=4, max_pages=10, tokens=3, slot=P, pos=P, k=P, v=P, table=P, pool=P,
             dev_status=P)
    a.update(kw)
    return pi.pi_cache_append(c or cache(), *a.values(), stream=0)


def test_append_refusals():
    refused(append, [(pi.PI_ERR_NULL, {k: None}) for k in ("slot", "pos", "k", "v", "table", "pool",
                                                           "dev_status")]
            + [(pi.PI_ERR_ALIGN, {k: P + 2}) for k in ("slot", "pos", "k", "v", "table", "pool")]
            + [(pi.PI_ERR_SHAPE, kw) for kw in (dict(layer=2), dict(tokens=-1), dict(slots=0),
                                                dict(max_pages=0))])
    assert append(tokens=0, slot=None, pos=None, k=None, v=None) == pi.PI_OK  # nothing to do
    for bad in BAD_CACHES:
        assert append(cache(**bad)) == pi.PI_ERR_SHAPE


def fork(c=None, wsb=None, **kw):
    a = dict(slots=4, max_pages=10, parent=P, grow=P, held=None, table_in=P, len_in=P,
             table=P + 4096, len=P + 8192, ref=P, pool=P, pairs=P, counts=P, dev_status=P, ws=P)
    a.update(kw)
    c = c or cache()
    return pi.pi_cache_fork(c, *a.values(), pi.pi_cache_workspace_size(c, 4, 0) if wsb is None
                            else wsb, stream=0)


def test_fork_refusals():
    names = ("parent", "grow", "table_in", "len_in", "table", "len", "ref", "pairs", "counts",
             "dev_status", "ws")
    refused(fork, [(pi.PI_ERR_NULL, {k: None}) for k in names]
            + [(pi.PI_ERR_ALIGN, {k: P + 4}) for k in names + ("pool", "held")]
            + [(pi.PI_ERR_SHAPE, kw) for kw in (
                dict(slots=0), dict(slots=1025), dict(max_pages=0), dict(table=P), dict(len=P),
                dict(held=P))]
            + [(pi.PI_ERR_WORKSPACE, dict(wsb=0))])
    for bad in BAD_CACHES:
        assert fork(cache(**bad)) == pi.PI_ERR_SHAPE


def compact(c=None, wsb=None, **kw):
    a = dict(slots=4, max_pages=10, held=None, table_in=P, len=P, table=P, ref=P, map=P, pool=P,
             pairs=P, counts=P, dev_status=P, ws=P)
    a.update(kw)
    c = c or cache()
    return pi.pi_cache_compact(c, *a.values(), pi.pi_cache_workspace_size(c, 4, 0) if wsb is None
                               else wsb, stream=0)


def test_compact_and_copy_refusals():
    names = ("table_in", "len", "table", "ref", "map", "pairs", "counts", "dev_status", "ws")
    refused(compact, [(pi.PI_ERR_NULL, {k: None}) for k in names]
            + [(pi.PI_ERR_ALIGN, {k: P + 4}) for k in names + ("pool", "held")]
            + [(pi.PI_ERR_SHAPE, kw) for kw in (dict(slots=0), dict(max_pages=0), dict(held=P))]
            + [(pi.PI_ERR_WORKSPACE, dict(wsb=64))])
    c = cache()
    assert pi.pi_cache_copy(c, P, P, -1, P, P, stream=0) == pi.PI_ERR_SHAPE
    assert pi.pi_cache_copy(c, None, P, 1, P, P, stream=0) == pi.PI_ERR_NULL
    assert pi.pi_cache_copy(c, P, P + 4, 1, P, P, stream=0) == pi.PI_ERR_ALIGN
    assert pi.pi_cache_copy(c, P, P, 1, P, None, stream=0) == pi.PI_ERR_NULL


def score(**kw):
    a = dict(logits=P, dtype="bf16", rows=4, vocab=100, stride=100, tokens=P, topk=5, logprob=P,
             entropy=P, top_idx=P, top_logprob=P, dev_status=P, ws=P)
    a.update(kw)
    wsb = a.pop("wsb", None)
    return pi.pi_token_logprobs(*a.values(), pi.pi_logprob_workspace_size(4, 100, 5) if wsb is None
                                else wsb, stream=0)


def test_score_refusals():
    refused(score, [(pi.PI_ERR_NULL, {k: None}) for k in (
        "logits", "tokens", "logprob", "top_idx", "top_logprob", "dev_status", "ws")]
        + [(pi.PI_ERR_ALIGN, {k: P + 4}) for k in ("logits", "tokens", "logprob", "entropy",
                                                    "top_idx", "top_logprob", "dev_status", "ws")]
        + [(pi.PI_ERR_SHAPE, kw) for kw in (
            dict(rows=-1), dict(vocab=0), dict(vocab=(1 << 24) + 1), dict(stride=99),
            dict(topk=33), dict(topk=-1), dict(vocab=4))]
        + [(pi.PI_ERR_DTYPE, dict(dtype=3)), (pi.PI_ERR_DTYPE, dict(dtype=-1)),
           (pi.PI_ERR_WORKSPACE, dict(wsb=0))])


# ------------------------------------------------------------------ plain forms
def test_plain_attention_by_hand():
    q = np.array([[1.0, 0.0]])
    k = np.array([[0.0, 5.0], [np.log(3.0), 0.0], [7.0, 7.0]])
    v = np.array([[4.0, 0.0], [8.0, 4.0], [100.0, 100.0]])
    y, lse, _ = plain.attention(q, k, v, 2, 1.0, 0, 0)
    np.testing.assert_allclose(y, [[7.0, 3.0]])
    np.testing.assert_allclose(lse, [np.log(4.0)])
    y, _, _ = plain.attention(q, k, v, 2, 1.0, 1, 0)   # the window hides token 0
    np.testing.assert_allclose(y, [[8.0, 4.0]])
    y, _, _ = plain.attention(q, k, v, 2, 1.0, 1, 1)   # token 0 stays visible
    np.testing.assert_allclose(y, [[7.0, 3.0]])
    y, lse, _ = plain.attention(q, k, v, 0, 1.0, 0, 0)
    assert (y == 0).all() and np.isneginf(lse).all()


def test_plain_score_by_hand():
    lp, ent, idx, top = plain.score_row([0.0, np.log(2.0), 0.0, -np.inf], 1, 3)
    assert lp == pytest.approx(np.log(0.5)) and idx == [1, 0, 2]
    assert ent == pytest.approx(0.5 * np.log(2) + 0.5 * np.log(4))
    assert top == pytest.approx([np.log(0.5), np.log(0.25), np.log(0.25)])


@pytest.mark.parametrize("seed", range(6))
def test_plain_fork_keeps_contents_and_counts(seed):
    # whatever the parents: each slot reads its parent's kept tokens, no page
    # that a slot will write is shared, the counts are those of the tables
    g = np.random.default_rng(seed)
    S, pt, mp, pages = 6, 4, 5, 200
    length = g.integers(0, mp * pt, S)
    perm = g.permutation(pages)
    table = [[int(perm[s * mp + j]) if j * pt < length[s] else -1 for j in range(mp)]
             for s in range(S)]
    parent, grow = g.integers(-1, S, S), g.integers(-5, 4, S)
    out, short = plain.fork(pt, pages, mp, parent, grow, None, table, length)
    content = {p: p for p in range(pages)}
    for a, b in out["pairs"]:
        content[b] = a
    count = [0] * pages
    for s in range(S):
        n = out["len"][s]
        for j in range(-(-n // pt)):
            count[out["table"][s][j]] += 1
        keep = min(n, length[parent[s]] if parent[s] >= 0 else 0)
        for t in range(keep):
            assert content[out["table"][s][t // pt]] == table[parent[s]][t // pt]
        for t in range(keep, n):  # to be written: the slot's alone
            p = out["table"][s][t // pt]
            assert sum(p in row for row in out["table"]) == 1
    assert count == out["ref"] and out["live"] == sum(c > 0 for c in count)


def test_plain_compact_by_hand():
    out = plain.compact(4, 7, 2, [0, 0, 0, 0, 1, 0, 0], [[6, 1], [6, 5]], [8, 6])
    assert out["map"] == [-1, 1, -1, -1, 0, 2, 3]
    assert out["table"] == [[3, 1], [3, 2]] and out["live"] == 4
    assert out["ref"] == [1, 1, 1, 2, 0, 0, 0] and out["pairs"] == [(4, 0), (5, 2), (6, 3)]
