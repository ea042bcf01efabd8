"""Performance cases of the operators for drafted tokens and for sampling.

A decode step may check several drafted continuations at once: the drafts of a
slot form a tree whose root is the token chosen last.

  tree     pi_tree_attention  the drafts' attention over the paged cache
  sample   pi_token_sample    tokens drawn by temperature, top-k, min-p, top-p
  accept   pi_tree_accept     the drafts that the drawn tokens confirm stay in
                              the cache, right behind the tokens before them

``run`` computes them in plain torch operations (32-bit arithmetic, 64-bit for
the sampling's sums) or, where ``own`` is true, through the library's entry
points.  Cache layout: pool [layers][pages][2 (K, V)][kv_heads][page_tokens]
[head_dim], 16-bit; table [slots][max_pages] int32 page numbers (-1: none); len
[slots] int32, drafts included.  Draft i of slot s, i < count[s], is stored as
token len[s] - count[s] + i and sees the tokens before the drafts, its
ancestors and itself.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest step: one short conversation, 1024 wide, a tree of five drafts (latency)
        dict(name="tree_1slot_16h64_5drafts_len200_f16", op="tree", slots=1, heads=16, kv_heads=16,
             head_dim=64, page=16, longest=200, drafts=5, shape="tree", ragged=False, window=0,
             sinks=0, dtype="f16", append=True),
        # an ordinary batch of the 13B shape (40 heads of 128), 13 drafts a slot
        dict(name="tree_32slots_40h128_13drafts_len2048_f16", op="tree", slots=32, heads=40,
             kv_heads=40, head_dim=128, page=16, longest=2048, drafts=13, shape="tree",
             ragged=True, window=0, sinks=0, dtype="f16", append=True),
        # shared heads, 26 drafts: about a hundred query rows per key-value head
        dict(name="tree_16slots_32h8x128_26drafts_len8001_bf16", op="tree", slots=16, heads=32,
             kv_heads=8, head_dim=128, page=64, longest=8001, drafts=26, shape="tree", ragged=True,
             window=0, sinks=0, dtype="bf16", append=False),
        # streaming chat: chains of drafts, last 1000 tokens and the first 4
        dict(name="tree_24slots_32h8x128_chain7_window1000_bf16", op="tree", slots=24, heads=32,
             kv_heads=8, head_dim=128, page=32, longest=16001, drafts=7, shape="chain",
             ragged=True, window=1000, sinks=4, dtype="bf16", append=True),
        # the largest: pieces of 64 prompt tokens behind long documents, eight heads a kv head
        dict(name="tree_8slots_64h8x128_chain64_len32768_f16", op="tree", slots=8, heads=64,
             kv_heads=8, head_dim=128, page=64, longest=32768, drafts=64, shape="chain",
             ragged=False, window=0, sinks=0, dtype="f16", append=True),
        # one conversation, odd vocabulary, fp32 logits (latency)
        dict(name="sample_1row_50273_f32", op="sample", rows=1, vocab=50273, pad=0, dtype="f32",
             banned=0.0, filters="top_p"),
        # a batch of requests with settings of their own
        dict(name="sample_64rows_128256_bf16", op="sample", rows=64, vocab=128256, pad=64,
             dtype="bf16", banned=0.01, filters="mixed"),
        # every draft of many slots, no filter but the temperature
        dict(name="sample_832rows_50272_f16", op="sample", rows=832, vocab=50272, pad=0,
             dtype="f16", banned=0.0, filters="none"),
        # the largest: a wide batch over a large vocabulary
        dict(name="sample_1024rows_128256_f32", op="sample", rows=1024, vocab=128256, pad=0,
             dtype="f32", banned=0.0, filters="mixed"),
        # one tree of five drafts, 24 layers 1024 wide (latency)
        dict(name="accept_1slot_24layers_5drafts_f16", op="accept", slots=1, drafts=5, width=3,
             longest=200, page=16, layers=24, kv_heads=16, head_dim=64, dtype="f16"),
        # the drafts of a batch in 48 layers of shared heads
        dict(name="accept_64slots_48layers_26drafts_bf16", op="accept", slots=64, drafts=26,
             width=5, longest=500, page=32, layers=48, kv_heads=8, head_dim=128, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "sample", "sample", "accept"])
    dtype = rng.choice(["f16", "bf16"])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "tree":
        kv_heads = rng.choice([1, 2, 4, 8, 16, 32, 40])
        group = rng.choice([1, 1, 2, 4, 5, 8, 16]) if kv_heads <= 8 else 1
        head_dim = rng.choice([64, 80, 96, 128, 128, 256])
        slots, drafts = _log_int(rng, 1, 64), _log_int(rng, 1, 64)
        rows = slots * kv_heads * group * drafts
        most = min(1.2e8 / (slots * kv_heads * head_dim), 1.5e8 / rows, 2.0e10 / (rows * head_dim))
        longest = _log_int(rng, 1, max(2, min(65536, int(most))))
        window = _log_int(rng, 16, 8192) if rng.random() < 0.4 else 0
        return dict(op=op, slots=slots, heads=kv_heads * group, kv_heads=kv_heads,
                    head_dim=head_dim, page=page, longest=longest, drafts=drafts,
                    shape=rng.choice(["tree", "tree", "chain"]), ragged=rng.random() < 0.5,
                    window=window, sinks=rng.choice([0, 1, 4, 7]) if window else 0, dtype=dtype,
                    append=rng.random() < 0.5)
    if op == "sample":
        vocab = _log_int(rng, 500, 200000)
        return dict(op=op, rows=_log_int(rng, 1, max(2, min(4096, int(6.0e7 / vocab)))),
                    vocab=vocab, pad=rng.choice([0, 0, 3, 64]),
                    dtype=rng.choice(["f16", "bf16", "f32"]), banned=rng.choice([0.0, 0.02, 0.5]),
                    filters=rng.choice(["none", "top_k", "top_p", "mixed", "mixed"]))
    slots, drafts, longest = _log_int(rng, 1, 64), _log_int(rng, 1, 64), _log_int(rng, 1, 500)
    kv_heads, head_dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 128, 256])
    most = 8.0e8 / (slots * (longest + drafts + page) * kv_heads * head_dim)
    return dict(op=op, slots=slots, drafts=drafts, width=rng.randint(1, 8), longest=longest,
                page=page, layers=min(_log_int(rng, 1, 48), max(1, int(most))),
                kv_heads=kv_heads, head_dim=head_dim, dtype=dtype)


# ------------------------------------------------------------------ inputs
def _base(c):
    """The slots' lengths before the drafts: spread evenly over (0, longest], the last one
    full, and one slot without any where there are eight or more."""
    i = np.arange(c["slots"])
    n = np.maximum(1, np.ceil(c["longest"] * np.modf((i + 1) * 0.6180339887)[0])).astype(np.int64)
    n[-1] = c["longest"]
    if c["slots"] >= 8:
        n[0] = 0
    return n


def _count(c):
    """Drafts per slot: all, or (ragged) spread over 0 .. drafts."""
    n = np.full(c["slots"], c["drafts"])
    if c.get("ragged"):
        i = np.arange(c["slots"])
        n = np.minimum(c["drafts"], np.ceil((c["drafts"] + 1) * np.modf((i + 2) * 0.7548776662)[0])).astype(np.int64)
        n[::5] = c["drafts"]
        if c["slots"] >= 8:
            n[1] = 0
    return n


def _parents(c, rng):
    """Random trees, parents before children and level by level, or chains."""
    i = np.arange(c["drafts"])
    if c["shape"] == "chain":
        return np.broadcast_to(i - 1, (c["slots"], c["drafts"]))
    back = np.sort((rng.random_sample((c["slots"], c["drafts"])) ** 0.5 * i).astype(np.int64), 1)
    back = np.minimum(back, np.maximum(i - 1, 0))
    back[:, 0] = -1
    return back


def _pages_of(n, page):
    return (n + page - 1) // page


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _cache(s, c, n, layers, rng, gen):
    """The pool, table and lengths of unshared slots of n tokens, pages in any order."""
    need = _pages_of(n, c["page"])
    pages, width = int(need.sum()) + 3, max(1, int(need.max()))
    t = np.full((len(n), width), -1, np.int64)
    t[np.arange(width)[None, :] < need[:, None]] = rng.permutation(pages)[: int(need.sum())]
    shape = (layers, pages, 2, c["kv_heads"], c["page"], c["head_dim"])
    s["pool"] = torch.empty(shape, dtype=_DTYPES[c["dtype"]], device="cuda").normal_(generator=gen)
    s["table"], s["len"] = _i32(t), _i32(n)


def _accept_tree(c, rng):
    """Trees of the accept cases, level by level: the root has `width` children, every
    level's first node has the next level's.  The tokens drawn confirm first children and
    then another child, at random, on at most `width` levels: so no confirmed draft's
    place is that of another, and a repeated pass finds the same rows."""
    S, N, w = c["slots"], c["drafts"], c["width"]
    i = np.arange(N)
    level = (i + w - 1) // w
    parent = np.where(i == 0, -1, np.where(level <= 1, 0, (level - 2) * w + 1))
    tokens = rng.randint(0, 50000, (S, N))
    # tokens of siblings differ: their last digit in base 8 is their place among them
    tokens = tokens // 8 * 8 + (i - 1) % w
    choice = rng.randint(50001, 60000, (S, N))
    heads = (level >= 1) & (level <= w) & ((i - 1) % w == 0)
    first = heads & (rng.random_sample((S, N)) < 0.8)
    row, col = np.nonzero(first)
    choice[row, parent[col]] = tokens[row, col]  # the first child goes on
    other = rng.randint(0, w, (S, N))  # or another child, whose path ends there
    last = heads & (rng.random_sample((S, N)) < 0.3) & (i[None, :] + other < N)
    row, col = np.nonzero(last)
    choice[row, parent[col]] = tokens[row, col + other[row, col]]
    return np.broadcast_to(parent, (S, N)), tokens, choice


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rng = np.random.RandomState(int(seed) % (1 << 32))
    s = {"case": c}
    op = c["op"]
    if op == "sample":
        R, V = c["rows"], c["vocab"]
        full = torch.empty((R, V + c["pad"]), dtype=_DTYPES[c["dtype"]], device="cuda")
        full.normal_(0.0, 3.0, generator=gen)
        if c["banned"]:
            ban = torch.rand(V, device="cuda", generator=gen) < c["banned"]
            full[:, :V].masked_fill_(ban, -math.inf)
        s["logits"] = full[:, :V]
        s["u"] = torch.rand(R, device="cuda", generator=gen)
        kind = c["filters"]
        temperature = rng.choice([0.0, 0.5, 0.7, 1.0, 1.3], R) if kind == "mixed" else np.full(R, 0.8)
        s["temperature"] = torch.from_numpy(temperature.astype(np.float32)).cuda()
        s["top_k"] = _i32(rng.choice([0, 1, 20, 50, 1000], R)) if kind in ("mixed", "top_k") else None
        s["top_p"] = s["min_p"] = None
        if kind in ("mixed", "top_p"):
            s["top_p"] = torch.from_numpy(rng.choice([0.5, 0.9, 0.95, 1.0], R).astype(np.float32)).cuda()
        if kind == "mixed":
            s["min_p"] = torch.from_numpy(rng.choice([0.0, 0.01, 0.1], R).astype(np.float32)).cuda()
        s["out"] = (torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, device="cuda"))
    elif op == "tree":
        S, N, H, D = c["slots"], c["drafts"], c["heads"], c["head_dim"]
        count = _count(c)
        _cache(s, c, _base(c) + count, 1, rng, gen)
        s["count"] = _i32(count) if c["ragged"] else None
        s["parent"] = _i32(_parents(c, rng)) if c["shape"] != "chain" else None
        s["q"] = torch.randn((S, N, H, D), device="cuda", generator=gen) * 2.0
        kv = (S, N, c["kv_heads"], D)
        s["k_new"] = torch.randn(kv, device="cuda", generator=gen) if c["append"] else None
        s["v_new"] = torch.randn(kv, device="cuda", generator=gen) if c["append"] else None
        s["out"] = (torch.zeros((S, N, H, D), device="cuda"), torch.zeros((S, N, H), device="cuda"))
    else:
        S, N = c["slots"], c["drafts"]
        parent, tokens, choice = _accept_tree(c, rng)
        _cache(s, c, _base(c) + N, c["layers"], rng, gen)
        s |= {"parent": _i32(parent), "tokens": _i32(tokens), "choice": _i32(choice)}
        ints = dict(dtype=torch.int32, device="cuda")
        s["out"] = {"len": torch.empty(S, **ints), "path": torch.empty((S, N), **ints),
                    "accepted": torch.empty(S, **ints), "next": torch.empty(S, **ints)}
    s["status"] = torch.zeros(4, dtype=torch.int32, device="cuda")
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The descriptor and the workspace that a program keeps between calls."""
    import activation_sparse_decode_rank_gb300 as pi
    c = s["case"]
    s["pi"] = pi
    if c["op"] == "sample":
        s["ws"] = pi.sample_workspace(c["rows"], c["vocab"])
        return
    pool = s["pool"]
    s["desc"] = pi.make_cache_desc(pool.shape[0], pool.shape[1], c["kv_heads"], c["head_dim"],
                                   c["page"], c["dtype"])
    if c["op"] == "tree":
        s["ws"] = pi.tree_workspace(s["desc"], c["slots"], c["heads"], c["drafts"])


# ------------------------------------------------------------------ one pass
def run(s):
    return _RUN_OWN[s["case"]["op"]](s) if own else _RUN_PLAIN[s["case"]["op"]](s)


def _own_tree(s):
    pi, c = s["pi"], s["case"]
    y, lse = s["out"]
    pi.check(pi.pi_tree_attention(
        s["desc"], 0, c["slots"], c["heads"], s["table"].shape[1], c["drafts"], s["parent"],
        s["count"], s["q"], s["k_new"], s["v_new"], s["table"], s["len"], s["pool"],
        c["head_dim"] ** -0.5, c["window"], c["sinks"], y, lse, s["status"], s["ws"]),
        "pi_tree_attention")
    return {"y": y, "lse": lse, "pool": s["pool"] if c["append"] else None}


def _own_sample(s):
    pi, c = s["pi"], s["case"]
    token, logprob = s["out"]
    pi.check(pi.pi_token_sample(
        s["logits"], c["dtype"], c["rows"], c["vocab"], s["logits"].stride(0), s["temperature"],
        s["top_k"], s["top_p"], s["min_p"], s["u"], token, logprob, s["status"], s["ws"]),
        "pi_token_sample")
    return {"token": token, "logprob": logprob}


def _own_accept(s):
    pi, c, o = s["pi"], s["case"], s["out"]
    pi.check(pi.pi_tree_accept(
        s["desc"], c["slots"], s["table"].shape[1], c["drafts"], s["parent"], None, s["tokens"],
        s["choice"], s["table"], s["len"], s["pool"], o["len"], o["path"], o["accepted"],
        o["next"], s["status"]), "pi_tree_accept")
    return dict(o, pool=s["pool"])


def _ancestors(parent):
    """[S][N][N] truth values: j is i or an ancestor of i.  Links of 1, 2, 4, .. steps."""
    N = parent.shape[1]
    i = torch.arange(N, device=parent.device)
    up = ((parent[:, :, None] == i) | (i[:, None] == i)).float()
    for _ in range(max(1, N.bit_length())):
        up = (torch.matmul(up, up) > 0).float()
    return up > 0


def _plain_tree(s):
    c, table, n = s["case"], s["table"], s["len"].long()
    S, H, Hk, D, P, N = c["slots"], c["heads"], c["kv_heads"], c["head_dim"], c["page"], c["drafts"]
    G, pool, dev = H // Hk, s["pool"][0], n.device
    i = torch.arange(N, device=dev)
    count = s["count"].long() if s["count"] is not None else torch.full((S,), N, device=dev)
    parent = s["parent"].long() if s["parent"] is not None else (i - 1).expand(S, N)
    base, live = n - count, i[None, :] < count[:, None]
    if c["append"]:
        slot, at = torch.nonzero(live, as_tuple=True)
        place = base[slot] + at
        page = table[slot, place // P].long()
        pool[page, 0, :, place % P] = s["k_new"][slot, at].to(pool.dtype)
        pool[page, 1, :, place % P] = s["v_new"][slot, at].to(pool.dtype)
    kv = pool[table.clamp(min=0).long()]                     # [S][pages][2][Hk][P][D]
    T = table.shape[1] * P
    k = kv[:, :, 0].permute(0, 2, 1, 3, 4).reshape(S, Hk, T, D).float()
    v = kv[:, :, 1].permute(0, 2, 1, 3, 4).reshape(S, Hk, T, D).float()
    del kv
    up = _ancestors(parent)
    depth = up.sum(2) - 1
    t = torch.arange(T, device=dev)
    before = t[None, :] < base[:, None]                      # [S][T]
    j = (t[None, :] - base[:, None]).clamp(0, N - 1)
    place = torch.where(before, t[None, :], base[:, None] + depth.gather(1, j))
    mine = (base[:, None] + depth)[:, :, None]               # positions of the drafts
    draft = (~before & (t[None, :] < n[:, None]))[:, None, :]
    seen = before[:, None, :] | (draft & up.gather(2, j[:, None, :].expand(S, N, T)))
    if c["window"]:
        seen &= (place[:, None, :] > mine - c["window"]) | (place[:, None, :] < c["sinks"])
    seen &= live[:, :, None]
    q = s["q"].view(S, N, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(S, Hk, N * G, D)
    score = torch.matmul(q, k.transpose(2, 3)).view(S, Hk, N, G, T) * D ** -0.5
    score.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    score -= torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = score.exp_()
    total = e.sum(-1, keepdim=True)
    y = torch.matmul(e.view(S, Hk, N * G, T), v).view(S, Hk, N, G, D)
    y /= torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total))[..., 0]
    y = torch.where(live[:, :, None, None], y.permute(0, 2, 1, 3, 4).reshape(S, N, H, D), 0.0)
    lse = torch.where(live[:, :, None], lse.permute(0, 2, 1, 3).reshape(S, N, H), 0.0)
    return {"y": y, "lse": lse, "pool": s["pool"] if c["append"] else None}


def _plain_sample(s):
    """In 64 bits: a token is a border between sums over the whole vocabulary."""
    x, T = s["logits"].float(), s["temperature"].double()
    R, V = x.shape
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    shift = (x.double() - x[:, :1].double()) / torch.where(T > 0, T, torch.ones_like(T))[:, None]
    rank = torch.arange(V, device=x.device)[None, :]
    keep = torch.where((T > 0)[:, None], torch.isfinite(shift), rank == 0)
    if s["top_k"] is not None:
        k = s["top_k"].long()
        keep &= rank < torch.where(k > 0, k, torch.full_like(k, V))[:, None]
    if s["min_p"] is not None:
        keep &= shift >= torch.log(s["min_p"].double())[:, None]
    w = torch.where(keep, shift.exp(), torch.zeros_like(shift))
    del shift
    sums = torch.cumsum(w, 1)
    if s["top_p"] is not None:
        keep &= (sums - w < s["top_p"].double()[:, None] * sums[:, -1:]) | (rank == 0)
    last = keep.sum(1, keepdim=True) - 1
    total = sums.gather(1, last)
    at = torch.minimum((sums <= s["u"].double()[:, None] * total).sum(1, keepdim=True), last)
    logprob = torch.log(w.gather(1, at) / total)
    return {"token": order.gather(1, at)[:, 0].int(), "logprob": logprob[:, 0].float()}


def _plain_accept(s):
    c, n, pool = s["case"], s["len"].long(), s["pool"]
    S, N, P, dev = c["slots"], c["drafts"], c["page"], s["len"].device
    parent, tokens, choice = s["parent"].long(), s["tokens"].long(), s["choice"].long()
    i = torch.arange(N, device=dev)
    fits = (parent >= 0) & (tokens == choice.gather(1, parent.clamp(min=0)))
    # of several children that fit, the first
    same = (parent[:, :, None] == parent[:, None, :]) & fits[:, None, :] & (i[None, :] < i[:, None])
    fits = (fits & ~same.any(2)) | (i == 0)
    taken = (~_ancestors(parent) | fits[:, None, :]).all(2)
    accepted = taken.sum(1)
    path = torch.sort(torch.where(taken, i, torch.full_like(parent, N)), 1).values
    base = n - N
    slot, j = torch.nonzero(path < N, as_tuple=True)
    frm, to = base[slot] + path[slot, j], base[slot] + j
    page, goal = s["table"][slot, frm // P].long(), s["table"][slot, to // P].long()
    pool[:, goal, :, :, to % P] = pool[:, page, :, :, frm % P]
    end = path.gather(1, (accepted - 1)[:, None])
    return {"len": (base + accepted).int(), "path": torch.where(path < N, path, -1).int(),
            "accepted": accepted.int(), "next": choice.gather(1, end)[:, 0].int(), "pool": pool}


_RUN_OWN = {"tree": _own_tree, "sample": _own_sample, "accept": _own_accept}
_RUN_PLAIN = {"tree": _plain_tree, "sample": _plain_sample, "accept": _plain_accept}


# ------------------------------------------------------------------ the least work
def work(case):
    """Bytes and operations that one pass cannot do without."""
    c, op = case, case["op"]
    if op == "sample":
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": c["rows"] * (c["vocab"] * size + 28), "flops": 6 * c["rows"] * c["vocab"]}
    row = 2 * c["kv_heads"] * c["head_dim"] * 2              # a token's K and V
    if op == "accept":
        # a level is reached by four of five paths of the one before; from the second
        # level on, confirmed drafts move
        levels = min(c["width"], -(-(c["drafts"] - 1) // c["width"]))
        moved = int(c["slots"] * sum(0.8 ** k for k in range(2, levels + 1)))
        return {"bytes": 2 * moved * row * c["layers"] + c["slots"] * (12 * c["drafts"] + 16),
                "flops": 0}
    base, count = _base(c), _count(c)
    live = count > 0
    reach = base
    if c["window"]:
        reach = np.minimum(base, c["window"] - 1) + np.minimum(
            c["sinks"], np.maximum(0, base - c["window"] + 1))
    tokens, drafts = int(reach[live].sum()), int(count.sum())
    pairs = int((reach * count)[live].sum()) + int((count * (count + 1) // 2).sum())
    io = drafts * c["heads"] * (8 * c["head_dim"] + 4)       # q, y, lse
    new = drafts * row * (3 if c["append"] else 1)
    return {"bytes": tokens * row + io + new + 4 * tokens // c["page"],
            "flops": 4 * pairs * c["heads"] * c["head_dim"]}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The operators' floating outputs from their definitions in 64 bits."""
    c = dict(case)
    s = prepare(c, seed)
    return {"tree": _exact_tree, "sample": _exact_sample}.get(c["op"], lambda c, s: None)(c, s)


def _exact_tree(c, s):
    S, H, Hk, D, P, N = c["slots"], c["heads"], c["kv_heads"], c["head_dim"], c["page"], c["drafts"]
    G, pool = H // Hk, s["pool"][0]
    n = s["len"].tolist()
    count = s["count"].tolist() if s["count"] is not None else [N] * S
    parent = s["parent"].tolist() if s["parent"] is not None else [list(range(-1, N - 1))] * S
    y = torch.zeros((S, N, H, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((S, N, H), dtype=torch.float64, device="cuda")
    for i in range(S):
        if not count[i]:
            continue
        base = n[i] - count[i]
        paths = []                                           # each draft's way from the root
        for d in range(count[i]):
            paths.append((paths[parent[i][d]] if parent[i][d] >= 0 else []) + [d])
        place = list(range(base)) + [base + len(p) - 1 for p in paths]
        place = torch.tensor(place, device="cuda")
        seen = torch.zeros((count[i], n[i]), dtype=torch.bool, device="cuda")
        seen[:, :base] = True
        for d, p in enumerate(paths):
            seen[d, [base + a for a in p]] = True
        if c["window"]:
            seen &= (place[None, :] > place[base:, None] - c["window"]) | (place < c["sinks"])[None, :]
        t = torch.arange(n[i], device="cuda")
        page = s["table"][i].long()[t // P]
        for h in range(Hk):
            k = pool[page, 0, h, t % P].double()
            v = pool[page, 1, h, t % P].double()
            if c["append"]:                                  # the cache holds them in its own type
                k[base:] = s["k_new"][i, :count[i], h].to(pool.dtype).double()
                v[base:] = s["v_new"][i, :count[i], h].to(pool.dtype).double()
            a = torch.einsum("dgx,tx->dgt", s["q"][i, :count[i], h * G:(h + 1) * G].double(), k)
            a = (a / math.sqrt(D)).masked_fill(~seen[:, None, :], -math.inf)
            z = torch.logsumexp(a, 2, keepdim=True)
            lse[i, :count[i], h * G:(h + 1) * G] = z[..., 0]
            y[i, :count[i], h * G:(h + 1) * G] = (a - z).exp() @ v
    return {"y": y, "lse": lse, "pool": None}


def _exact_sample(c, s):
    """Row by row: the probabilities by value, the token where their running sum passes u."""
    got = []
    T, u = s["temperature"].tolist(), s["u"].tolist()
    for r in range(c["rows"]):
        if T[r] == 0.0:
            got.append(0.0)
            continue
        p = torch.softmax(s["logits"][r].double() / T[r], 0)
        p = torch.sort(p, descending=True).values
        if s["min_p"] is not None:
            p = p[p >= s["min_p"][r].double() * p[0]]
        if s["top_k"] is not None and int(s["top_k"][r]) > 0:
            p = p[: int(s["top_k"][r])]
        p = p[p > 0]
        p = p / p.sum()
        if s["top_p"] is not None:
            p = p[: max(1, int((torch.cumsum(p, 0) - p < s["top_p"][r].double()).sum()))]
            p = p / p.sum()
        at = min(len(p) - 1, int((torch.cumsum(p, 0) <= u[r]).sum()))
        got.append(float(torch.log(p[at])))
    return {"token": None, "logprob": torch.tensor(got, dtype=torch.float64)}
