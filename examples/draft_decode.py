"""Decoding with drafted tokens: a tree of guesses per sequence, checked in one step.

    python examples/draft_decode.py [--slots 2] [--tokens 40] [--temperature 0.7]

The small random-weight decoder of beam_decode.py continues prompts by sampling.
Each step guesses a few continuations of every sequence (here from the output
layer alone, without attention), lets the slots grow by them (pi_cache_fork), runs
the decoder over all guesses at once (pi_tree_attention, pi_layer_decode), draws
the token that follows each of them (pi_token_sample), and keeps the guesses that
were right (pi_tree_accept).  A token's random number goes by its position, so the
sequences are those that single steps would have drawn.  Needs a GPU and a built
libpi.so.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from beam_decode import (HEAD_DIM, HEADS, KV_HEADS, LAYERS, PAGE, VOCAB, Decoder, pi)  # noqa: E402

PARENT = [-1, 0, 0, 0, 1, 2, 4]  # the root, three children, two grandchildren, one more
DEPTH = [0, 1, 1, 1, 2, 2, 3]
DRAFTS = len(PARENT)


class DraftDecoder:
    """Continues `slots` prompts of one length, for `longest` tokens at most."""

    def __init__(self, model: Decoder, slots: int, longest: int, temperature=0.7, top_k=50, top_p=0.95,
                 seed: int = 7):
        self.m, self.S = model, slots
        dev = model.device
        self.max_pages = -(-(longest + DRAFTS) // PAGE)
        pages = slots * self.max_pages
        self.cache = pi.make_cache_desc(LAYERS, pages, KV_HEADS, HEAD_DIM, PAGE, "f16")
        self.pool = torch.empty((LAYERS, pages, 2, KV_HEADS, PAGE, HEAD_DIM), dtype=torch.float16, device=dev)

        def ints(*shape, fill=0):
            return torch.full(shape, fill, dtype=torch.int32, device=dev)
        # a fork reads one pair of tables and lengths and writes the other; an accept
        # writes the lengths of the pair not in use
        self.table = [ints(slots, self.max_pages, fill=-1) for _ in range(2)]
        self.length, self.kept = ints(slots), ints(slots)
        self.ref, self.pairs, self.counts = ints(pages), ints(slots, 2), ints(4)
        self.path, self.accepted, self.next = ints(slots, DRAFTS), ints(slots), ints(slots)
        self.parent = torch.tensor([PARENT] * slots, dtype=torch.int32, device=dev)
        self.same = torch.arange(slots, dtype=torch.int32, device=dev)
        self.status = ints(4)
        self.now = 0
        self.ws = pi.cache_workspace(self.cache, slots, 0, dev)
        self.tree_ws = pi.tree_workspace(self.cache, slots, HEADS, DRAFTS, dev)
        rows = slots * DRAFTS
        self.sample_ws = pi.sample_workspace(rows, VOCAB, dev)

        def floats(v):
            return torch.full((rows,), v, device=dev)
        self.filters = floats(temperature), ints(rows, fill=top_k), floats(top_p)
        # a random number per slot and position
        g = torch.Generator(device=dev).manual_seed(seed)
        self.u = torch.rand((slots, longest + 2 * DRAFTS), generator=g, device=dev)

    def fork(self, grow, length):
        a, b = self.now, 1 - self.now
        pi.check(pi.pi_cache_fork(self.cache, self.S, self.max_pages, self.same, grow, None, self.table[a],
                                  length, self.table[b], self.length, self.ref, self.pool, self.pairs,
                                  self.counts, self.status, self.ws), "pi_cache_fork")
        self.now = b

    def sample(self, logits, u):
        rows = logits.shape[0]
        token = torch.empty(rows, dtype=torch.int32, device=logits.device)
        t, k, p = (f[:rows] for f in self.filters)
        pi.check(pi.pi_token_sample(logits, "f32", rows, VOCAB, logits.stride(0), t, k, p, None, u, token,
                                    None, self.status, self.sample_ws), "pi_token_sample")
        return token

    def guess(self, root):
        """Trees [slots][DRAFTS] of tokens that may follow the roots."""
        def best(tokens, n):
            return torch.topk(self.m.logits(self.m.embed[tokens.long()]), n).indices.int()
        t = torch.empty((self.S, DRAFTS), dtype=torch.int32, device=root.device)
        t[:, 0], t[:, 1:4] = root, best(root, 3)
        t[:, 4], t[:, 5] = best(t[:, 1], 1)[:, 0], best(t[:, 2], 1)[:, 0]
        t[:, 6] = best(t[:, 4], 1)[:, 0]
        return t

    def step(self, tokens, count):
        """Logits [slots DRAFTS][vocab] of the drafted trees, their keys and values cached.
        Slots without drafts are left alone; their logits mean nothing."""
        m, rows = self.m, self.S * DRAFTS
        x = m.embed[tokens.flatten().long()]
        y = torch.zeros((rows, HEADS * HEAD_DIM), device=m.device)
        for layer in range(LAYERS):
            q, k, v = ((x @ w[layer]).contiguous() for w in (m.wq, m.wk, m.wv))
            pi.check(pi.pi_tree_attention(
                self.cache, layer, self.S, HEADS, self.max_pages, DRAFTS, self.parent, count, q, k, v,
                self.table[self.now], self.length, self.pool, HEAD_DIM ** -0.5, 0, 0, y, None,
                self.status, self.tree_ws), "pi_tree_attention")
            x = m.ffn_step(layer, x + y @ m.wo[layer])
        return m.logits(x)

    def run(self, prompts, new_tokens: int):
        """Sequences as lists, with new_tokens or up to three more tokens each, and the steps taken."""
        m, dev = self.m, self.m.device
        prompts = torch.as_tensor(prompts, device=dev)
        n = prompts.shape[1]
        grow = torch.full((self.S,), n, dtype=torch.int32, device=dev)
        self.fork(grow, torch.zeros_like(grow))
        where = torch.arange(n, dtype=torch.int32, device=dev)
        last = []
        for s in range(self.S):
            logits, kept = m.prompt(prompts[s])
            last.append(logits[-1])
            slot = torch.full((n,), s, dtype=torch.int32, device=dev)
            for layer, (k, v) in enumerate(kept):
                pi.check(pi.pi_cache_append(self.cache, layer, self.S, self.max_pages, n, slot, where,
                                            k.contiguous(), v.contiguous(), self.table[self.now],
                                            self.pool, self.status), "pi_cache_append")
        root = self.sample(torch.stack(last), self.u[:, n].clone())
        out = [prompts[s].tolist() + [int(root[s])] for s in range(self.S)]
        self.kept.copy_(self.length)
        depth = torch.tensor(DEPTH, device=dev)
        steps = 0
        while True:
            # slots that have their tokens draft no more
            more = [len(t) < n + new_tokens for t in out]
            if not any(more):
                return out, steps
            count = torch.tensor([DRAFTS * a for a in more], dtype=torch.int32, device=dev)
            tokens = self.guess(root)
            self.fork(count, self.kept)
            logits = self.step(tokens, count)
            # draft i stands at position base + depth; the token after it at one more
            at = (self.length.long() - count.long())[:, None] + depth + 1
            choice = self.sample(logits, self.u.gather(1, at.clamp(max=self.u.shape[1] - 1)).flatten())
            pi.check(pi.pi_tree_accept(
                self.cache, self.S, self.max_pages, DRAFTS, self.parent, count, tokens, choice,
                self.table[self.now], self.length, self.pool, self.kept, self.path, self.accepted,
                self.next, self.status), "pi_tree_accept")
            root = torch.where(count > 0, self.next, root)
            for s, (path, a) in enumerate(zip(self.path.tolist(), self.accepted.tolist())):
                if a:
                    out[s] += [int(tokens[s, i]) for i in path[1:a]] + [int(root[s])]
            steps += 1


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--slots", type=int, default=2, help="at most 4")
    ap.add_argument("--tokens", type=int, default=40)
    ap.add_argument("--temperature", type=float, default=0.7)
    a = ap.parse_args()
    model = Decoder()
    prompts = torch.randint(0, VOCAB, (a.slots, 21), generator=torch.Generator().manual_seed(5))
    dec = DraftDecoder(model, a.slots, 21 + a.tokens + DRAFTS, a.temperature)
    out, steps = dec.run(prompts, a.tokens)
    assert int(dec.status[0]) == 0 and int(model.status[0]) == 0
    made = sum(len(t) - 21 for t in out)
    print(f"{made} tokens of {a.slots} sequences in {steps} steps")
    for t in out:
        print(t[21:])


if __name__ == "__main__":
    main()
