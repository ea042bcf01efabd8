"""The operators of include/pi_draft.h without a GPU: every entry point is exported
and bound, bad arguments are refused on the host before any launch, and the plain
forms the GPU tests compare with agree with hand-worked results."""
import math
import os
import re

import numpy as np
import pytest

import activation_sparse_decode_rank_gb300 as pi
import drafthelp as plain

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 40  # stand-in address: every call below is refused before a launch


@pytest.fixture(scope="module", autouse=True)
def _built():
    pi.build()


def test_exports_and_bindings():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "pi_draft.h")).read(),
                 flags=re.S)
    names = sorted(set(re.findall(r"\b(pi_[a-z_]+)\s*\(", src)))
    assert {"pi_tree_attention", "pi_tree_accept", "pi_token_sample"} <= set(names)
    for n in names:
        assert hasattr(pi.lib(), n) and n in pi.SIGNATURES and callable(getattr(pi, n))


def cache(**kw):
    a = dict(layers=2, pages=100, kv_heads=4, head_dim=64, page_tokens=16, dtype="f16")
    a.update(kw)
    return pi.make_cache_desc(**a)


BAD_CACHES = [dict(layers=0), dict(layers=257), dict(pages=0), dict(pages=(1 << 26) + 1),
              dict(kv_heads=0), dict(kv_heads=257), dict(head_dim=12), dict(head_dim=264),
              dict(head_dim=0), dict(page_tokens=0), dict(page_tokens=257)]


def test_workspace_sizes():
    c = cache()
    assert pi.pi_tree_workspace_size(c, 4, 8, 5) > 0
    for bad in BAD_CACHES + [dict(dtype="f32")]:
        assert pi.pi_tree_workspace_size(cache(**bad), 4, 8, 5) == 0
    for bad in [(0, 8, 5), (1025, 8, 5), (4, 6, 5), (4, 0, 5), (4, 2048, 5), (4, 8, 0), (4, 8, 65)]:
        assert pi.pi_tree_workspace_size(c, *bad) == 0
    assert pi.pi_sample_workspace_size(4, 100) > 0 and pi.pi_sample_workspace_size(0, 1) > 0
    for bad in [(-1, 100), (4, 0), (4, (1 << 24) + 1)]:
        assert pi.pi_sample_workspace_size(*bad) == 0
    with pytest.raises(pi.PiError):
        pi.tree_workspace(c, 4, 8, 65)
    with pytest.raises(pi.PiError):
        pi.sample_workspace(4, 0)


def refused(call, rows):
    for want, kw in rows:
        assert call(**kw) == want, kw


def attention(c=None, wsb=None, **kw):
    a = dict(layer=0, slots=4, heads=8, max_pages=10, drafts=5, parent=P, count=P, q=P, k_new=None,
             v_new=None, table=P, len=P, pool=P, scale=0.125, window=0, sinks=0, y=P, lse=P,
             dev_status=P, ws=P)
    a.update(kw)
    c = c or cache()
    return pi.pi_tree_attention(c, *a.values(), pi.pi_tree_workspace_size(cache(), 4, 8, 5)
                                if wsb is None else wsb, stream=0)


def test_attention_refusals():
    refused(attention, [
        (pi.PI_ERR_NULL, {k: None}) for k in ("q", "table", "len", "pool", "y", "dev_status", "ws")
    ] + [(pi.PI_ERR_ALIGN, {k: P + 4}) for k in ("parent", "count", "q", "table", "len", "pool", "y",
                                                  "lse", "ws", "dev_status")]
        + [(pi.PI_ERR_SHAPE, kw) for kw in (
            dict(layer=-1), dict(layer=2), dict(slots=0), dict(slots=1025), dict(heads=0),
            dict(heads=6), dict(heads=2048), dict(max_pages=0), dict(max_pages=1 << 27),
            dict(drafts=0), dict(drafts=65), dict(drafts=-1), dict(window=-1), dict(sinks=-1))]
        + [(pi.PI_ERR_NULL, dict(k_new=P)), (pi.PI_ERR_NULL, dict(v_new=P)),
           (pi.PI_ERR_ALIGN, dict(k_new=P + 8, v_new=P)), (pi.PI_ERR_WORKSPACE, dict(wsb=0))])
    for bad in BAD_CACHES:
        assert attention(cache(**bad)) == pi.PI_ERR_SHAPE
    assert attention(cache(dtype="f32")) == pi.PI_ERR_DTYPE


def test_tree_selftest_refusals():
    def f(c, limit, wsb=None):
        size = pi.pi_tree_workspace_size(c, 4, 8, 5) if wsb is None else wsb
        return pi.pi_selftest_tree_timeout(c, 4, 8, 10, 5, P, P, P, P, P, P, P, limit, size, stream=0)
    assert f(cache(), 10) == pi.PI_ERR_SHAPE and f(cache(), 6 * 10 ** 9) == pi.PI_ERR_SHAPE
    assert f(cache(), 10 ** 6, 0) == pi.PI_ERR_WORKSPACE
    for c in (cache(head_dim=56), cache(page_tokens=7)):
        assert f(c, 10 ** 6) == pi.PI_ERR_SHAPE


def accept(c=None, **kw):
    a = dict(slots=4, max_pages=10, drafts=5, parent=P, count=P, tokens=P + 64, choice=P + 128,
             table=P + 4096, len=P + 256, pool=P + 65536, len_out=P + 8192, path=P + 8256,
             accepted=P + 8320, next=P + 8384, dev_status=P + 512)
    a.update(kw)
    return pi.pi_tree_accept(c or cache(), *a.values(), stream=0)


def test_accept_refusals():
    names = ("tokens", "choice", "table", "len", "len_out", "path", "accepted", "next", "dev_status")
    refused(accept, [(pi.PI_ERR_NULL, {k: None}) for k in names]
            + [(pi.PI_ERR_ALIGN, {k: P + 4}) for k in names + ("parent", "count", "pool")]
            + [(pi.PI_ERR_SHAPE, kw) for kw in (
                dict(slots=0), dict(slots=1025), dict(max_pages=0), dict(drafts=0), dict(drafts=65),
                dict(len_out=P + 256), dict(path=P), dict(next=P + 128), dict(accepted=P + 64))])
    for bad in BAD_CACHES:
        assert accept(cache(**bad)) == pi.PI_ERR_SHAPE
    assert accept(cache(dtype="f32")) == pi.PI_ERR_DTYPE


def sample(**kw):
    a = dict(logits=P, dtype="bf16", rows=4, vocab=100, stride=100, temperature=P, top_k=P, top_p=P,
             min_p=P, u=P, token=P, logprob=P, dev_status=P, ws=P)
    a.update(kw)
    wsb = a.pop("wsb", None)
    return pi.pi_token_sample(*a.values(), pi.pi_sample_workspace_size(4, 100) if wsb is None else wsb,
                              stream=0)


def test_sample_refusals():
    refused(sample, [(pi.PI_ERR_NULL, {k: None}) for k in ("logits", "u", "token", "dev_status", "ws")]
            + [(pi.PI_ERR_ALIGN, {k: P + 4}) for k in ("logits", "temperature", "top_k", "top_p", "min_p",
                                                       "u", "token", "logprob", "dev_status", "ws")]
            + [(pi.PI_ERR_SHAPE, kw) for kw in (dict(rows=-1), dict(vocab=0), dict(stride=99),
                                                dict(vocab=(1 << 24) + 1, stride=1 << 25))]
            + [(pi.PI_ERR_DTYPE, dict(dtype=3)), (pi.PI_ERR_DTYPE, dict(dtype=-1)),
               (pi.PI_ERR_WORKSPACE, dict(wsb=0))])
    assert sample(rows=0, logits=None, u=None, token=None) == pi.PI_OK  # nothing to do


# ------------------------------------------------------------------ plain forms
def test_plain_visible_by_hand():
    parent = [-1, 0, 0, 1, 2, -1]
    assert plain.path_of(parent, 3) == [0, 1, 3]
    assert plain.visible(2, parent, 4, 0, 0) == [0, 1, 2, 4, 6]
    assert plain.visible(2, parent, 5, 0, 0) == [0, 1, 7]
    # positions of 0, 1, root, 2, 4: 0 1 2 3 4; a window of 3 leaves 2, 3, 4
    assert plain.visible(2, parent, 4, 3, 0) == [2, 4, 6]
    assert plain.visible(2, parent, 4, 1, 1) == [0, 6]
    assert plain.visible(0, parent, 3, 2, 1) == [0, 1, 3]


def test_plain_accept_by_hand():
    parent, tokens = [-1, 0, 0, 0, 2, 2], [7, 5, 9, 9, 5, 6]
    assert plain.accept(parent, tokens, [9, 0, 6, 0, 0, 4]) == ([0, 2, 5], 4)
    assert plain.accept(parent, tokens, [8, 0, 6, 0, 0, 4]) == ([0], 8)
    assert plain.accept([], [], []) == ([], -1)


def test_plain_sample_by_hand():
    x = [math.log(2.0), math.log(4.0), math.log(2.0), -math.inf]  # weights 1/2, 1, 1/2: 1 0 2
    for u, tok in [(0.0, 1), (0.49, 1), (0.51, 0), (0.74, 0), (0.76, 2), (0.999, 2)]:
        t, lp, _ = plain.sample_row(x, 1.0, 0, 1.0, 0.0, u)
        assert t == tok and lp == pytest.approx(math.log(0.5 if tok == 1 else 0.25))
    assert plain.sample_row(x, 1.0, 2, 1.0, 0.0, 0.99)[0] == 0          # top-k
    assert plain.sample_row(x, 1.0, 0, 0.6, 0.0, 0.99)[0] == 0          # top-p: 1/2 + 1/4
    assert plain.sample_row(x, 1.0, 0, 1.0, 0.7, 0.99)[:2] == (1, 0.0)  # min-p
    assert plain.sample_row(x, 0.0, 0, 1.0, 0.0, 0.99)[:2] == (1, 0.0)
    t, lp, _ = plain.sample_row(x, 0.5, 0, 1.0, 0.0, 0.7)               # weights 1/4, 1, 1/4
    assert t == 0 and lp == pytest.approx(math.log(1 / 6))
    for bad in ([0.0, math.nan], [math.inf, 0.0], [-math.inf, -math.inf]):
        assert plain.sample_row(bad, 1.0, 0, 1.0, 0.0, 0.5)[0] == -1
    assert plain.sample_row(x, -1.0, 0, 1.0, 0.0, 0.5)[0] == -1
    assert plain.sample_row(x, 1.0, 0, 1.0, 0.0, 1.0)[0] == -1


def test_plain_attention_infinite_by_hand():
    q = np.array([[1.0, 0.0]])
    k = np.array([[0.0, 1.0], [-np.inf, 0.0]])
    v = np.array([[2.0, np.inf], [5.0, 1.0]])
    y, lse, _, _ = plain.attention(q, k[:1], v[:1], [0], 1.0)
    assert y[0, 0] == 2.0 and y[0, 1] == np.inf and lse[0] == 0.0
