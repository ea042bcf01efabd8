"""Performance cases of the key-value cache and token-scoring operators.

The operators are what a decode loop runs around the activation-sparse FFN:

  attend    pi_paged_attention   one new token per slot over its paged cache
  append    pi_cache_append      new keys and values into their pages
  fork      pi_cache_fork        reorder / fork / free / trim / grow the slots
  compact   pi_cache_compact     live pages to the front of the pool
  logprobs  pi_token_logprobs    given tokens' log probabilities, entropy, top

``run`` computes them in plain torch operations (32-bit arithmetic) or, where
``own`` is true, through the library's entry points.  Cache layout:
pool [layers][pages][2 (K, V)][kv_heads][page_tokens][head_dim], 16-bit;
table [slots][max_pages] int32 page numbers (-1: none); len [slots] int32.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest decode step: one short conversation, 1024 wide (latency)
        dict(name="attend_1slot_16h64_len200_f16", op="attend", slots=1, heads=16, kv_heads=16,
             head_dim=64, page=16, longest=200, window=0, sinks=0, dtype="f16", append=True),
        # an ordinary batch of the 13B shape (40 heads of 128), lengths of every age
        dict(name="attend_32slots_40h128_len2048_f16", op="attend", slots=32, heads=40,
             kv_heads=40, head_dim=128, page=16, longest=2048, window=0, sinks=0, dtype="f16",
             append=False),
        # streaming chat: shared heads, last 1000 tokens and the first 4, new token appended
        dict(name="attend_24slots_32h8x128_window1000_bf16", op="attend", slots=24, heads=32,
             kv_heads=8, head_dim=128, page=32, longest=16001, window=1000, sinks=4,
             dtype="bf16", append=True),
        # the largest: long documents, eight query heads per key-value head
        dict(name="attend_8slots_64h8x128_len131072_bf16", op="attend", slots=8, heads=64,
             kv_heads=8, head_dim=128, page=64, longest=131072, window=0, sinks=0, dtype="bf16",
             append=False),
        # one decode step's keys and values of 32 slots
        dict(name="append_32tokens_40h128_f16", op="append", slots=32, tokens=32, kv_heads=40,
             head_dim=128, page=16, dtype="f16"),
        # prompts admitted together: 12001 tokens of four slots
        dict(name="append_12001tokens_32h128_bf16", op="append", slots=4, tokens=12001,
             kv_heads=32, head_dim=128, page=16, dtype="bf16"),
        # one beam of four after a scoring step, 24 layers 1024 wide (latency)
        dict(name="fork_4slots_24layers_f16", op="fork", slots=4, width=4, prompt=203, tail=52,
             page=16, max_pages=32, spare=64, layers=24, kv_heads=16, head_dim=64, dtype="f16"),
        # 128 groups of eight samples each on shared prompts, some ended and replaced
        dict(name="fork_1024slots_len12000_bf16", op="fork", slots=1024, width=8, prompt=12001,
             tail=333, page=16, max_pages=1024, spare=40000, layers=2, kv_heads=1, head_dim=128,
             dtype="bf16"),
        # a small pool after a few conversations ended
        dict(name="compact_8slots_24layers_f16", op="compact", slots=8, page=16, max_pages=32,
             longest=500, live=0.6, layers=24, kv_heads=16, head_dim=64, dtype="f16"),
        # a large pool before it is shrunk
        dict(name="compact_64slots_16layers_bf16", op="compact", slots=64, page=16, max_pages=128,
             longest=1003, live=0.7, layers=16, kv_heads=8, head_dim=128, dtype="bf16"),
        # a decode step's candidates of seven beams, odd vocabulary, fp32 logits
        dict(name="logprobs_7rows_50273_f32", op="logprobs", rows=7, vocab=50273, pad=0, topk=8,
             dtype="f32", banned=0.01),
        # scoring of prompts: one row per prompt token, 16-bit logits with ties
        dict(name="logprobs_4096rows_128256_bf16", op="logprobs", rows=4096, vocab=128256, pad=64,
             topk=20, dtype="bf16", banned=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "fork", "compact", "logprobs",
                     "logprobs"])
    dtype = rng.choice(["f16", "bf16"])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "attend":
        kv_heads = rng.choice([1, 2, 4, 8, 16, 32, 40])
        group = rng.choice([1, 1, 2, 4, 5, 8, 16]) if kv_heads <= 8 else 1
        head_dim = rng.choice([64, 80, 96, 128, 128, 256])
        slots = _log_int(rng, 1, 64)
        most = 4.0e8 / (slots * kv_heads * head_dim)  # elements of K
        longest = _log_int(rng, 1, max(2, min(131072, int(most))))
        window = _log_int(rng, 16, 8192) if rng.random() < 0.4 else 0
        return dict(op=op, slots=slots, heads=kv_heads * group, kv_heads=kv_heads,
                    head_dim=head_dim, page=page, longest=longest, window=window,
                    sinks=rng.choice([0, 1, 4, 7]) if window else 0, dtype=dtype,
                    append=rng.random() < 0.5)
    if op == "append":
        return dict(op=op, slots=_log_int(rng, 1, 64), tokens=_log_int(rng, 1, 16384),
                    kv_heads=rng.choice([1, 4, 8, 32, 40]), head_dim=rng.choice([64, 80, 128, 256]),
                    page=page, dtype=dtype)
    if op == "fork":
        width = rng.choice([1, 2, 4, 5, 8])
        slots = width * _log_int(rng, 1, 512 // width)
        prompt, tail = _log_int(rng, 1, 8192), _log_int(rng, 1, 400)
        return dict(op=op, slots=slots, width=width, prompt=prompt, tail=tail, page=page,
                    max_pages=(prompt + tail) // page + 4, spare=slots * (prompt // page // 8 + 4),
                    layers=rng.choice([1, 2, 3]), kv_heads=rng.choice([1, 2]),
                    head_dim=rng.choice([64, 80, 128]), dtype=dtype)
    if op == "compact":
        slots, longest = _log_int(rng, 1, 128), _log_int(rng, 1, 4096)
        return dict(op=op, slots=slots, page=page, max_pages=longest // page + 3, longest=longest,
                    live=rng.choice([0.3, 0.5, 0.8, 0.95]), layers=rng.choice([1, 3, 4]),
                    kv_heads=rng.choice([1, 2, 4]), head_dim=rng.choice([64, 80, 128]),
                    dtype=dtype)
    vocab = _log_int(rng, 500, 200000)
    return dict(op=op, rows=_log_int(rng, 1, max(2, min(8192, int(2.5e8 / vocab)))), vocab=vocab,
                pad=rng.choice([0, 0, 3, 64]), topk=rng.choice([0, 1, 5, 20, 32]),
                dtype=rng.choice(["f16", "bf16", "f32"]), banned=rng.choice([0.0, 0.02, 0.5]))


# ------------------------------------------------------------------ inputs
def _lengths(c):
    """The slots' lengths: spread evenly over (0, longest], the last one full, and one
    slot empty where there are eight or more."""
    i = np.arange(c["slots"])
    n = np.maximum(1, np.ceil(c["longest"] * np.modf((i + 1) * 0.6180339887)[0])).astype(np.int64)
    n[-1] = c["longest"]
    if c["slots"] >= 8:
        n[0] = 0
    return n


def _pages_of(n, page):
    return (n + page - 1) // page


def _tables(n, page, numbers, max_pages):
    """Tables of unshared slots of lengths n, filled from `numbers` in turn."""
    need = _pages_of(n, page)
    t = np.full((len(n), max_pages), -1, np.int64)
    t[np.arange(max_pages)[None, :] < need[:, None]] = numbers[: int(need.sum())]
    return t


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _pool(c, layers, pages, gen):
    shape = (layers, pages, 2, c["kv_heads"], c["page"], c["head_dim"])
    return torch.empty(shape, dtype=_DTYPES[c["dtype"]], device="cuda").normal_(generator=gen)


def _fork_plan(c):
    """Who is whose parent, what the slots hold and how many pages that is.  Groups of
    `width` slots share a prompt; the first half of each group's slots have two children
    each, the others end; every eighth group (of eight or more) ends and its slots begin
    anew with a prompt of their own."""
    S, w, P = c["slots"], c["width"], c["page"]
    s = np.arange(S)
    g, j = s // w, s % w
    length = np.full(S, c["prompt"] + c["tail"]) + g % 7  # groups are of several ages
    parent, grow = g * w + j // 2, np.ones(S, np.int64)
    new = g % 8 == 7
    parent[new] = -1
    grow[new] = c["prompt"] // 8 + 1
    length = np.minimum(length, c["max_pages"] * P - 1)
    shared = min(c["prompt"], int(length.min())) // P  # full prompt pages
    return parent, grow, length, shared


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rng = np.random.RandomState(int(seed) % (1 << 32))
    s = {"case": c}
    op = c["op"]
    if op == "logprobs":
        R, V = c["rows"], c["vocab"]
        full = torch.empty((R, V + c["pad"]), dtype=_DTYPES[c["dtype"]], device="cuda")
        full.normal_(0.0, 3.0, generator=gen)
        if c["banned"]:
            ban = torch.rand(V, device="cuda", generator=gen) < c["banned"]
            full[:, :V].masked_fill_(ban, -math.inf)
        s["logits"] = full[:, :V]
        tok = torch.randint(0, V, (R,), device="cuda", generator=gen, dtype=torch.int32)
        s["tokens"] = tok
        k = c["topk"]
        s["out"] = (torch.empty(R, device="cuda"), torch.empty(R, device="cuda"),
                    torch.empty((R, k), dtype=torch.int32, device="cuda"),
                    torch.empty((R, k), device="cuda"))
    elif op == "attend":
        n = _lengths(c)
        need = int(_pages_of(n, c["page"]).sum())
        pages, mp = need + 3, max(1, int(_pages_of(n, c["page"]).max()))
        s["table"] = _i32(_tables(n, c["page"], rng.permutation(pages), mp))
        s["len"] = _i32(n)
        s["pool"] = _pool(c, 1, pages, gen)
        S, H, D = c["slots"], c["heads"], c["head_dim"]
        s["q"] = torch.randn((S, H, D), device="cuda", generator=gen) * 2.0
        kv = (S, c["kv_heads"], D)
        s["k_new"] = torch.randn(kv, device="cuda", generator=gen) if c["append"] else None
        s["v_new"] = torch.randn(kv, device="cuda", generator=gen) if c["append"] else None
        s["out"] = (torch.empty((S, H, D), device="cuda"), torch.empty((S, H), device="cuda"))
    elif op == "append":
        # tokens spread over the slots, each slot's positions in order from 0
        slot = np.arange(c["tokens"]) * c["slots"] // c["tokens"]
        n = np.bincount(slot, minlength=c["slots"])
        pos = np.arange(c["tokens"]) - (np.cumsum(n) - n)[slot]
        need = int(_pages_of(n, c["page"]).sum())
        mp = max(1, int(_pages_of(n, c["page"]).max()))
        s["table"] = _i32(_tables(n, c["page"], rng.permutation(need + 2), mp))
        s["slot"], s["pos"] = _i32(slot), _i32(pos)
        s["pool"] = _pool(c, 1, need + 2, gen)
        kv = (c["tokens"], c["kv_heads"], c["head_dim"])
        s["k"] = torch.randn(kv, device="cuda", generator=gen)
        s["v"] = torch.randn(kv, device="cuda", generator=gen)
    elif op == "fork":
        S, P, mp = c["slots"], c["page"], c["max_pages"]
        parent, grow, length, shared = _fork_plan(c)
        groups = S // c["width"]
        own_pages = _pages_of(length, P) - shared
        used = groups * shared + int(own_pages.sum())
        pages = used + c["spare"]
        numbers = rng.permutation(pages)
        t = np.full((S, mp), -1, np.int64)
        heads = numbers[: groups * shared].reshape(groups, shared)
        t[:, :shared] = heads[np.arange(S) // c["width"]]
        at = np.arange(mp)[None, :]
        t[(at >= shared) & (at < (shared + own_pages)[:, None])] = numbers[groups * shared:used]
        held = np.zeros(pages, np.int64)
        held[numbers[used:used + c["spare"] // 16]] = 1  # pages kept outside the slots
        s |= {"table": _i32(t), "len": _i32(length), "parent": _i32(parent), "grow": _i32(grow),
              "held": _i32(held), "pool": _pool(c, c["layers"], pages, gen)}
        s["out"] = {"table": torch.empty_like(s["table"]), "len": torch.empty_like(s["len"]),
                    "ref": torch.empty_like(s["held"]),
                    "pairs": torch.zeros((S, 2), dtype=torch.int32, device="cuda"),
                    "counts": torch.zeros(4, dtype=torch.int32, device="cuda")}
    else:
        S, P, mp = c["slots"], c["page"], c["max_pages"]
        n = _lengths(c)
        live, pages, moved = _compact_sizes(c)
        numbers = np.concatenate([rng.permutation(live)[: live - moved],
                                  live + rng.permutation(pages - live)[:moved]])
        s["table"] = _i32(_tables(n, P, rng.permutation(numbers), mp))
        s["len"] = _i32(n)
        s["pool"] = _pool(c, c["layers"], pages, gen)
        s["out"] = {"table": torch.empty_like(s["table"]),
                    "ref": torch.empty(pages, dtype=torch.int32, device="cuda"),
                    "map": torch.empty(pages, dtype=torch.int32, device="cuda"),
                    "pairs": torch.zeros((pages, 2), dtype=torch.int32, device="cuda"),
                    "counts": torch.zeros(4, dtype=torch.int32, device="cuda")}
    s["status"] = torch.zeros(4, dtype=torch.int32, device="cuda")
    if own:
        _prepare_own(s)
    return s


def _compact_sizes(c):
    live = int(_pages_of(_lengths(c), c["page"]).sum())
    pages = int(math.ceil(live / c["live"])) + 1
    return live, pages, min(pages - live, int(round(live * (1.0 - live / pages))))


def _prepare_own(s):
    """The descriptor and the workspace that a program keeps between calls."""
    import activation_sparse_decode_rank_gb300 as pi
    c = s["case"]
    s["pi"] = pi
    if c["op"] == "logprobs":
        s["ws"] = pi.logprob_workspace(c["rows"], c["vocab"], c["topk"])
        return
    pool = s["pool"]
    s["desc"] = pi.make_cache_desc(pool.shape[0], pool.shape[1], c["kv_heads"], c["head_dim"],
                                   c["page"], c["dtype"])
    s["ws"] = pi.cache_workspace(s["desc"], c["slots"], c.get("heads", 0))


# ------------------------------------------------------------------ one pass
def run(s):
    return _RUN_OWN[s["case"]["op"]](s) if own else _RUN_PLAIN[s["case"]["op"]](s)


def _own_attend(s):
    pi, c = s["pi"], s["case"]
    y, lse = s["out"]
    pi.check(pi.pi_paged_attention(
        s["desc"], 0, c["slots"], c["heads"], s["table"].shape[1], s["q"], s["k_new"], s["v_new"],
        s["table"], s["len"], s["pool"], c["head_dim"] ** -0.5, c["window"], c["sinks"], y, lse,
        s["status"], s["ws"]), "pi_paged_attention")
    return {"y": y, "lse": lse, "pool": s["pool"] if c["append"] else None}


def _own_append(s):
    pi, c = s["pi"], s["case"]
    pi.check(pi.pi_cache_append(
        s["desc"], 0, c["slots"], s["table"].shape[1], c["tokens"], s["slot"], s["pos"], s["k"],
        s["v"], s["table"], s["pool"], s["status"]), "pi_cache_append")
    return {"pool": s["pool"]}


def _own_fork(s):
    pi, c, o = s["pi"], s["case"], s["out"]
    pi.check(pi.pi_cache_fork(
        s["desc"], c["slots"], c["max_pages"], s["parent"], s["grow"], s["held"], s["table"],
        s["len"], o["table"], o["len"], o["ref"], s["pool"], o["pairs"], o["counts"], s["status"],
        s["ws"]), "pi_cache_fork")
    return dict(o, pool=s["pool"])


def _own_compact(s):
    pi, c, o = s["pi"], s["case"], s["out"]
    pi.check(pi.pi_cache_compact(
        s["desc"], c["slots"], c["max_pages"], None, s["table"], s["len"], o["table"], o["ref"],
        o["map"], s["pool"], o["pairs"], o["counts"], s["status"], s["ws"]), "pi_cache_compact")
    return dict(o, pool=s["pool"])


def _own_logprobs(s):
    pi, c = s["pi"], s["case"]
    lp, ent, idx, top = s["out"]
    pi.check(pi.pi_token_logprobs(
        s["logits"], c["dtype"], c["rows"], c["vocab"], s["logits"].stride(0), s["tokens"],
        c["topk"], lp, ent, idx, top, s["status"], s["ws"]), "pi_token_logprobs")
    return {"logprob": lp, "entropy": ent, "top_idx": idx, "top_logprob": top}


def _plain_attend(s):
    c, table, n = s["case"], s["table"], s["len"].long()
    S, H, Hk, D, P = c["slots"], c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    pool = s["pool"][0]
    if c["append"]:
        live = torch.nonzero(n > 0).flatten()
        at = n[live] - 1
        page = table[live, at // P].long()
        pool[page, 0, :, at % P] = s["k_new"][live].to(pool.dtype)
        pool[page, 1, :, at % P] = s["v_new"][live].to(pool.dtype)
    kv = pool[table.clamp(min=0).long()]                     # [S][pages][2][Hk][P][D]
    T = table.shape[1] * P
    k = kv[:, :, 0].permute(0, 2, 1, 3, 4).reshape(S, Hk, T, D).float()
    v = kv[:, :, 1].permute(0, 2, 1, 3, 4).reshape(S, Hk, T, D).float()
    del kv
    score = torch.matmul(s["q"].view(S, Hk, H // Hk, D), k.transpose(2, 3)) * D ** -0.5
    t = torch.arange(T, device="cuda")
    seen = t[None, :] < n[:, None]
    if c["window"]:
        seen &= (t[None, :] >= n[:, None] - c["window"]) | (t[None, :] < c["sinks"])
    seen = seen[:, None, None, :]
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    y = torch.matmul(e, v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total)).view(S, H)
    return {"y": y.reshape(S, H, D), "lse": lse, "pool": s["pool"] if c["append"] else None}


def _plain_append(s):
    c, pool = s["case"], s["pool"][0]
    pos = s["pos"].long()
    page = s["table"][s["slot"].long(), pos // c["page"]].long()
    pool[page, 0, :, pos % c["page"]] = s["k"].to(pool.dtype)
    pool[page, 1, :, pos % c["page"]] = s["v"].to(pool.dtype)
    return {"pool": s["pool"]}


def _plain_fork(s):
    c, held = s["case"], s["held"].long()
    S, P, mp, pages = c["slots"], c["page"], c["max_pages"], held.numel()
    dev = held.device
    parent = s["parent"].long()
    base = torch.where(parent >= 0, s["len"].long()[parent.clamp(min=0)], torch.zeros_like(parent))
    want = (base + s["grow"].long()).clamp(min=0)
    keep = torch.minimum(base, want)
    whole, some = keep // P, keep % P > 0
    at = torch.arange(mp, device=dev)[None, :]
    src = s["table"].long()[parent.clamp(min=0)]             # the parents' rows
    ones = torch.ones((), dtype=torch.long, device=dev)
    full = src[at < whole[:, None]]
    ref = held.index_add(0, full, ones.expand(full.numel()))
    # the last, partly filled page: its lowest slot keeps it where nobody else has it
    last = torch.where(some, src.gather(1, whole.clamp(max=mp - 1)[:, None])[:, 0],
                       torch.full_like(whole, pages))
    slot = torch.arange(S, device=dev)
    owner = torch.full((pages + 1,), S, device=dev).scatter_reduce(0, last, slot, "amin")
    busy = torch.cat([ref, ones.view(1)])
    stay = some & (owner[last] == slot) & (busy[last] == 0)
    copy = some & ~stay
    ref = torch.cat([ref, ones.view(1) * 0]).index_add(0, torch.where(stay, last, pages), ones.expand(S))[:pages]
    # fresh pages, lowest first, in the order of the slots
    first = whole + stay.long()                               # entries that are kept
    total = (want + P - 1) // P
    need = (total - first).clamp(min=0)
    free = torch.nonzero(ref == 0).flatten()
    before = torch.cumsum(need, 0) - need
    fresh = (at >= first[:, None]) & (at < total[:, None])
    number = free[(before[:, None] + at - first[:, None])[fresh]]
    table = torch.where(at < first[:, None], src, torch.full_like(src, -1))
    table[fresh] = number
    ref[number] = 1
    out = s["out"]
    to = table.gather(1, whole.clamp(max=mp - 1)[:, None])[:, 0][copy]
    frm = last[copy]
    s["pool"][:, to] = s["pool"][:, frm]
    out["pairs"][: frm.numel()] = torch.stack([frm, to], 1).int()
    out["counts"][0] = frm.numel()
    out["counts"][1] = (ref > 0).sum()
    return {"table": table.int(), "len": want.int(), "ref": ref.int(), "pairs": out["pairs"],
            "counts": out["counts"], "pool": s["pool"]}


def _plain_compact(s):
    c, table, n = s["case"], s["table"].long(), s["len"].long()
    pages = s["pool"].shape[1]
    dev = table.device
    used = torch.arange(c["max_pages"], device=dev)[None, :] < ((n + c["page"] - 1) // c["page"])[:, None]
    numbers = table[used]
    ref = torch.zeros(pages, dtype=torch.long, device=dev).index_add(
        0, numbers, torch.ones_like(numbers))
    live = ref > 0
    count = live.sum()
    at = torch.arange(pages, device=dev)
    frm = at[live & (at >= count)]
    to = at[~live & (at < count)]
    where = torch.where(live, at, torch.full_like(at, -1))
    where[frm] = to
    s["pool"][:, to] = s["pool"][:, frm]
    new_ref = torch.zeros_like(ref)
    new_ref[where[live]] = ref[live]
    out = s["out"]
    out["pairs"][: frm.numel()] = torch.stack([frm, to], 1).int()
    out["counts"][0] = frm.numel()
    out["counts"][1] = count
    return {"table": torch.where(used, where[table.clamp(min=0)], torch.full_like(table, -1)).int(),
            "ref": new_ref.int(), "map": where.int(), "pairs": out["pairs"],
            "counts": out["counts"], "pool": s["pool"]}


def _plain_logprobs(s):
    c = s["case"]
    x = s["logits"].float()
    top = x.amax(-1, keepdim=True)
    shift = x - top
    e = torch.exp(shift)
    total = e.sum(-1, keepdim=True)
    log_total = torch.log(total)
    entropy = log_total[:, 0] - (e * torch.where(e > 0, shift, torch.zeros_like(e))).sum(-1) / total[:, 0]
    lp = (shift.gather(1, s["tokens"].long()[:, None]) - log_total)[:, 0]
    # order by value, then by lowest index: one whole-number key for both
    bits = x.view(torch.int32).long()
    del shift, e
    key = torch.where(bits < 0, -(bits & 0x7fffffff), bits) * (1 << 20)
    key -= torch.arange(c["vocab"], device=x.device)
    idx = torch.topk(key, c["topk"], dim=-1).indices
    return {"logprob": lp, "entropy": entropy, "top_idx": idx.int(),
            "top_logprob": x.gather(1, idx) - top - log_total}


_RUN_OWN = {"attend": _own_attend, "append": _own_append, "fork": _own_fork,
            "compact": _own_compact, "logprobs": _own_logprobs}
_RUN_PLAIN = {"attend": _plain_attend, "append": _plain_append, "fork": _plain_fork,
              "compact": _plain_compact, "logprobs": _plain_logprobs}


# ------------------------------------------------------------------ the least work
def work(case):
    """Bytes and operations that one pass cannot do without."""
    c, op = case, case["op"]
    if op == "logprobs":
        size = 4 if c["dtype"] == "f32" else 2
        n = c["rows"] * c["vocab"]
        return {"bytes": n * size + c["rows"] * (12 + 8 * c["topk"]), "flops": 6 * n}
    row = 2 * c["kv_heads"] * c["head_dim"] * 2              # a token's K and V
    if op == "attend":
        n = _lengths(c)
        seen = n
        if c["window"]:
            seen = np.minimum(n, c["window"]) + np.minimum(c["sinks"], np.maximum(0, n - c["window"]))
        seen = int(seen.sum())
        qy = c["slots"] * c["heads"] * c["head_dim"] * 8 + c["slots"] * c["heads"] * 4
        new = c["slots"] * row * 2 if c["append"] else 0
        return {"bytes": seen * row + qy + new + 4 * seen // c["page"],
                "flops": 4 * seen * c["heads"] * c["head_dim"]}
    if op == "append":
        return {"bytes": c["tokens"] * (row * 3 + 8), "flops": 0}
    page = row * c["page"] * c["layers"]                      # a page in every layer
    if op == "fork":
        parent, grow, length, shared = _fork_plan(c)
        P, mp, S = c["page"], c["max_pages"], c["slots"]
        base = np.where(parent >= 0, length[np.maximum(parent, 0)], 0)
        copies = 0
        for p in np.unique(parent[parent >= 0]):
            copies += (int((parent == p).sum()) - 1) * int(length[p] % P > 0)
        used = (S // c["width"]) * shared + int((_pages_of(length, P) - shared).sum())
        read = int(_pages_of(base, P).sum())
        return {"bytes": 2 * copies * page + 4 * (read + S * mp + 4 * S + 2 * (used + c["spare"])),
                "flops": 0}
    live, pages, moved = _compact_sizes(c)
    return {"bytes": 2 * moved * page + 4 * (live + c["slots"] * c["max_pages"] + 2 * pages),
            "flops": 0}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The operators' floating outputs from their definitions in 64 bits."""
    c = dict(case)
    s = prepare(c, seed)
    if c["op"] == "attend":
        return _exact_attend(c, s)
    if c["op"] == "logprobs":
        return _exact_logprobs(c, s)
    if c["op"] == "append":
        return {"pool": _exact_append(c, s["pool"], s["table"], s["slot"], s["pos"], s["k"], s["v"])}
    return None


def _exact_append(c, pool, table, slot, pos, k, v):
    """The pool as 64-bit values, the new rows unrounded: rows by flat offsets."""
    out = pool.double()
    if out.numel() > 2_000_000_000:
        return None
    Hk, P, D = c["kv_heads"], c["page"], c["head_dim"]
    flat = out.view(-1, D)
    for i0 in range(0, slot.numel(), 4096):
        sl, ps = slot[i0:i0 + 4096].long(), pos[i0:i0 + 4096].long()
        page = table.view(-1)[sl * table.shape[1] + ps // P].long()
        for kind, src in ((0, k), (1, v)):
            head = torch.arange(Hk, device="cuda")
            rows = ((page[:, None] * 2 + kind) * Hk + head[None, :]) * P + (ps % P)[:, None]
            flat[rows.reshape(-1)] = src[i0:i0 + 4096].double().reshape(-1, D)
    return out


def _exact_attend(c, s):
    S, H, Hk, D, P = c["slots"], c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    G = H // Hk
    n = s["len"].tolist()
    y = torch.zeros((S, H, D), dtype=torch.float64, device="cuda")
    lse = torch.full((S, H), -math.inf, dtype=torch.float64, device="cuda")
    pool = s["pool"][0]
    if c["append"]:  # the cache holds the new rows in its own type
        for i in range(S):
            if n[i]:
                page = int(s["table"][i, (n[i] - 1) // P])
                pool[page, 0, :, (n[i] - 1) % P] = s["k_new"][i].to(pool.dtype)
                pool[page, 1, :, (n[i] - 1) % P] = s["v_new"][i].to(pool.dtype)
    for i in range(S):
        t = np.arange(n[i])
        if c["window"]:
            t = t[(t >= n[i] - c["window"]) | (t < c["sinks"])]
        if not len(t):
            continue
        t = torch.from_numpy(t).cuda()
        page = s["table"][i].long()[t // P]
        for h in range(Hk):
            k = pool[page, 0, h, t % P].double()
            v = pool[page, 1, h, t % P].double()
            a = (s["q"][i, h * G:(h + 1) * G].double() @ k.T) / math.sqrt(D)
            top = a.max(1, keepdim=True).values
            p = (a - top).exp()
            y[i, h * G:(h + 1) * G] = (p @ v) / p.sum(1, keepdim=True)
            lse[i, h * G:(h + 1) * G] = (top + p.sum(1, keepdim=True).log())[:, 0]
    return {"y": y, "lse": lse, "pool": None}


def _exact_logprobs(c, s):
    got = {"logprob": [], "entropy": [], "top_logprob": []}
    for r in range(0, c["rows"], 256):
        x = s["logits"][r:r + 256].double()
        z = torch.logsumexp(x, 1, keepdim=True)
        p = (x - z).exp()
        got["entropy"].append(-(p * torch.nan_to_num(x - z, neginf=0.0)).sum(1))
        got["logprob"].append((x.gather(1, s["tokens"][r:r + 256].long()[:, None]) - z)[:, 0])
        best = torch.sort(x, 1, descending=True).values[:, : c["topk"]]
        got["top_logprob"].append(best - z)
    return {"logprob": torch.cat(got["logprob"]), "entropy": torch.cat(got["entropy"]),
            "top_idx": None, "top_logprob": torch.cat(got["top_logprob"])}
