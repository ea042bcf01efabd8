"""Beam search with a small decoder: the serving operators around the sparse FFN.

    python examples/beam_decode.py [--beams 4] [--steps 24] [--window 0]

A random-weight decoder (attention, activation-sparse FFN, output layer)
continues a prompt.  Per step and layer the new token's keys and values enter
the paged cache and are attended to (pi_paged_attention), then the FFN runs
(pi_layer_decode); per step the logits are scored (pi_token_logprobs), the
best continuations of all beams are chosen, and the cache follows them
(pi_cache_fork).  The prompt's keys and values are stored by pi_cache_append;
at the end the finished beams' pages are moved together (pi_cache_compact).
Projections are plain torch products.  Needs a GPU and a built libpi.so.
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import activation_sparse_decode_rank_gb300 as pi  # noqa: E402
import synth  # noqa: E402

VOCAB, D_MODEL, NEURONS, RANK = 500, 256, 1024, 16
LAYERS, HEADS, KV_HEADS, HEAD_DIM, PAGE = 3, 8, 2, 32, 16


def _up(a, dev):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).to(dev)


class Decoder:
    """Random weights; the FFN layers are the synthetic sparse layers of the tests."""

    def __init__(self, seed: int = 1, device: str = "cuda"):
        dev = self.device = torch.device(device)
        g = torch.Generator(device=dev).manual_seed(seed)

        def rnd(*shape, scale):
            return torch.randn(shape, generator=g, device=dev) * scale
        self.embed = rnd(VOCAB, D_MODEL, scale=1.0)
        self.out = rnd(VOCAB, D_MODEL, scale=1.0)
        kv = KV_HEADS * HEAD_DIM
        self.wq = [rnd(D_MODEL, HEADS * HEAD_DIM, scale=D_MODEL ** -0.5) for _ in range(LAYERS)]
        self.wk = [rnd(D_MODEL, kv, scale=D_MODEL ** -0.5) for _ in range(LAYERS)]
        self.wv = [rnd(D_MODEL, kv, scale=D_MODEL ** -0.5) for _ in range(LAYERS)]
        self.wo = [rnd(HEADS * HEAD_DIM, D_MODEL, scale=D_MODEL ** -0.5) for _ in range(LAYERS)]
        self.ffn_desc = pi.make_desc(D_MODEL, NEURONS, RANK, "f16")
        self.ffn, self._held = [], []
        for layer in range(LAYERS):
            L = synth.make_layer(D_MODEL, NEURONS, RANK, "f16", alpha=0.8, density=0.1,
                                 seed=seed + layer)
            t = [_up(getattr(L, n), dev) for n in ("A", "Bm", "b1", "W1", "W2", "b2")]
            self._held.append(t)
            self.ffn.append(pi.make_weights(*t))
        self.ffn_ws = pi.workspace(self.ffn_desc, 32, dev)
        self.status = torch.zeros(4, dtype=torch.int32, device=dev)

    def ffn_step(self, layer, x):
        """x + FFN(x) for up to 32 rows."""
        y = torch.empty_like(x)
        pi.check(pi.pi_layer_decode(self.ffn_desc, self.ffn[layer], x, x.shape[0], y, x, None, None,
                                    self.status, self.ffn_ws), "pi_layer_decode")
        return y

    def logits(self, x):
        return (x / x.norm(dim=-1, keepdim=True)) @ self.out.T * 2.0

    def prompt(self, tokens, window: int = 0, sinks: int = 0):
        """Plain forward pass over one sequence: logits [n][vocab] and each
        layer's keys and values [n][kv_heads][head_dim].  As a decode step
        does, attention reads keys and values rounded to the cache's type."""
        n = len(tokens)
        x = self.embed[tokens]
        t = torch.arange(n, device=self.device)
        seen = t[None, :] <= t[:, None]
        if window:
            seen &= (t[None, :] > t[:, None] - window) | (t[None, :] < sinks)
        kept = []
        for layer in range(LAYERS):
            q = (x @ self.wq[layer]).view(n, KV_HEADS, HEADS // KV_HEADS, HEAD_DIM)
            k = (x @ self.wk[layer]).view(n, KV_HEADS, HEAD_DIM)
            v = (x @ self.wv[layer]).view(n, KV_HEADS, HEAD_DIM)
            kept.append((k, v))
            a = torch.einsum("nghd,mgd->nghm", q, k.half().float()) * HEAD_DIM ** -0.5
            p = torch.softmax(a.masked_fill(~seen[:, None, None, :], float("-inf")), -1)
            o = torch.einsum("nghm,mgd->nghd", p, v.half().float()).reshape(n, -1)
            x = x + o @ self.wo[layer]
            x = torch.cat([self.ffn_step(layer, x[i:i + 32].contiguous()) for i in range(0, n, 32)])
        return self.logits(x), kept


class BeamSearch:
    """`beams` continuations of one prompt over a shared paged cache."""

    def __init__(self, model: Decoder, beams: int, longest: int, window: int = 0, sinks: int = 0):
        self.m, self.B, self.window, self.sinks = model, beams, window, sinks
        dev = model.device
        self.max_pages = -(-longest // PAGE)
        pages = beams * self.max_pages + beams
        self.cache = pi.make_cache_desc(LAYERS, pages, KV_HEADS, HEAD_DIM, PAGE, "f16")
        self.pool = torch.empty((LAYERS, pages, 2, KV_HEADS, PAGE, HEAD_DIM), dtype=torch.float16,
                                device=dev)
        self.ws = pi.cache_workspace(self.cache, beams, HEADS, dev)
        self.score_ws = pi.logprob_workspace(beams, VOCAB, beams, dev)

        def ints(*shape, fill=0):
            return torch.full(shape, fill, dtype=torch.int32, device=dev)
        # tables and lengths alternate between two buffers: a fork reads one, writes the other
        self.table = [ints(beams, self.max_pages, fill=-1) for _ in range(2)]
        self.length = [ints(beams) for _ in range(2)]
        self.ref, self.map = ints(pages), ints(pages)
        self.pairs, self.counts = ints(max(beams, pages // 2), 2), ints(4)
        self.status = ints(4)
        self.now = 0

    def fork(self, parent, grow):
        a, b = self.now, 1 - self.now
        pi.check(pi.pi_cache_fork(self.cache, self.B, self.max_pages, parent, grow, None,
                                  self.table[a], self.length[a], self.table[b], self.length[b],
                                  self.ref, self.pool, self.pairs, self.counts, self.status,
                                  self.ws), "pi_cache_fork")
        self.now = b

    def ints(self, values):
        return torch.tensor(values, dtype=torch.int32, device=self.m.device)

    def step(self, tokens):
        """One decode step of every beam: its new token's logits [beams][vocab]."""
        m, B = self.m, self.B
        x = m.embed[tokens]
        y = torch.empty((B, HEADS * HEAD_DIM), device=m.device)
        for layer in range(LAYERS):
            q, k, v = ((x @ w[layer]).contiguous() for w in (m.wq, m.wk, m.wv))
            pi.check(pi.pi_paged_attention(
                self.cache, layer, B, HEADS, self.max_pages, q, k, v, self.table[self.now],
                self.length[self.now], self.pool, HEAD_DIM ** -0.5, self.window, self.sinks, y, None,
                self.status, self.ws), "pi_paged_attention")
            x = m.ffn_step(layer, x + y @ m.wo[layer])
        return m.logits(x)

    def score(self, logits):
        """The beams' best continuations: indices and log probabilities [beams][beams]."""
        R, k = logits.shape[0], self.B
        idx = torch.empty((R, k), dtype=torch.int32, device=logits.device)
        top = torch.empty((R, k), device=logits.device)
        pi.check(pi.pi_token_logprobs(logits, "f32", R, VOCAB, logits.stride(0), None, k, None, None,
                                      idx, top, self.status, self.score_ws), "pi_token_logprobs")
        return idx, top

    def run(self, prompt, steps: int):
        """Token sequences [beams][prompt + steps] and their log probabilities."""
        m, B, dev = self.m, self.B, self.m.device
        prompt = torch.as_tensor(prompt, device=dev)
        n = len(prompt)
        logits, kept = m.prompt(prompt, self.window, self.sinks)
        # slot 0 takes the prompt, the others begin empty
        self.fork(self.ints([-1] * B), self.ints([n] + [0] * (B - 1)))
        where = self.ints([0] * n), self.ints(list(range(n)))
        for layer, (k, v) in enumerate(kept):
            pi.check(pi.pi_cache_append(self.cache, layer, B, self.max_pages, n, *where,
                                        k.contiguous(), v.contiguous(), self.table[self.now],
                                        self.pool, self.status), "pi_cache_append")
        idx, top = self.score(logits[-1:].contiguous())
        score = top[0].clone()
        tokens = torch.cat([prompt.expand(B, n), idx[0, :, None].long()], 1)
        parent = torch.zeros(B, dtype=torch.int32, device=dev)  # all beams continue slot 0
        one = self.ints([1] * B)
        for _ in range(steps - 1):
            self.fork(parent, one)
            idx, top = self.score(self.step(tokens[:, -1]))
            best = torch.topk((score[:, None] + top).flatten(), B)
            parent = (best.indices // B).int()
            score = best.values
            tokens = torch.cat([tokens[parent.long()], idx.flatten()[best.indices][:, None].long()], 1)
        self.fork(parent, self.ints([0] * B))
        return tokens, score

    def compact(self):
        """Moves the pages in use to the front of the pool; returns their number."""
        t = self.table[self.now]
        pi.check(pi.pi_cache_compact(self.cache, self.B, self.max_pages, None, t,
                                     self.length[self.now], t, self.ref, self.map, self.pool,
                                     self.pairs, self.counts, self.status, self.ws),
                 "pi_cache_compact")
        return int(self.counts[1])


def rescore(model, tokens, n, window=0, sinks=0):
    """Log probability of tokens[n:] after tokens[:n] by a pass without a cache."""
    logits, _ = model.prompt(tokens[:-1], window, sinks)
    lp = torch.log_softmax(logits.double(), -1)[n - 1:]
    return float(lp.gather(1, tokens[n:, None]).sum())


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--window", type=int, default=0, help="visible tokens (0: all), plus the first 4")
    a = ap.parse_args()
    model = Decoder()
    prompt = torch.randint(0, VOCAB, (21,), generator=torch.Generator().manual_seed(5))
    sinks = 4 if a.window else 0
    search = BeamSearch(model, a.beams, len(prompt) + a.steps, a.window, sinks)
    tokens, score = search.run(prompt, a.steps)
    live = search.compact()
    assert int(search.status[0]) == 0 and int(model.status[0]) == 0
    print(f"{live} pages hold {a.beams} sequences of {tokens.shape[1] - 1} cached tokens")
    for b in range(a.beams):
        again = rescore(model, tokens[b], len(prompt), a.window, sinks)
        print(f"beam {b}: log p = {float(score[b]):9.4f} (without a cache {again:9.4f}) "
              f"{tokens[b, len(prompt):].tolist()}")


if __name__ == "__main__":
    main()
