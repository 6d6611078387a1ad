"""Beam search with a paged key-value cache: every cache operator in the place it has in a serving program.

A one-layer attention model with random weights extends a few prompts of different lengths. The prompts' keys and
values enter the cache at once; each step then forks, drops and grows the beams' rows (cache_select), stores the new
tokens (cache_append) and attends to them (attention_decode); what is elementwise between them, the beams' scores added
to their tokens', is a Command on the same stream. Halfway, requests that are done leave, and the pool is compacted.
Tables, lengths and counts never leave the GPU.

    python examples/beam_search.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tensor_command_execution_gb300 as T  # noqa: E402

VOCABULARY, WIDTH, HEADS, KV_HEADS, DIM, PAGE = 512, 256, 8, 2, 64, 16


class Model:
    """Embedding, one attention layer with rotary positions, and a projection to the vocabulary."""

    def __init__(self, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weights(rows, columns):
            return (torch.randn(rows, columns, generator=gen, device="cuda") * rows ** -0.5).to(dtype)
        self.embedding = torch.randn(VOCABULARY, WIDTH, generator=gen, device="cuda").to(dtype)
        self.q, self.k, self.v = weights(WIDTH, HEADS * DIM), weights(WIDTH, KV_HEADS * DIM), weights(WIDTH, KV_HEADS * DIM)
        self.out = weights(HEADS * DIM, VOCABULARY)
        self.turns = T.rope_turns(DIM, 10000.0)

    def project(self, tokens):
        x = self.embedding[tokens]
        return ((x @ self.q).view(-1, HEADS, DIM), (x @ self.k).view(-1, KV_HEADS, DIM), (x @ self.v).view(-1, KV_HEADS, DIM))


class Scores:
    """Each beam's score added to those of its tokens: a Command over [beams, vocabulary], the beams' scores broadcast."""

    def __init__(self):
        c = T.Command()
        self.tokens, self.beams = c.load_tensor("f32", 2), c.load_tensor("f32", 2)
        self.out = c.store(c.execute([("add", self.tokens, self.beams)])[0], "f32", 2)
        self.kernel = c.compile()

    def __call__(self, tokens, beams):
        out = torch.empty_like(tokens)
        self.kernel.launch({self.tokens: tokens, self.beams: beams[:, None].expand_as(tokens), self.out: out})
        return out


class Cache:
    """The pools and what says who holds which page; `status` collects what the operators could not do."""

    def __init__(self, pages, columns, dtype=torch.bfloat16):
        self.k, self.v = (torch.zeros(pages, PAGE, KV_HEADS, DIM, dtype=dtype, device="cuda") for _ in range(2))
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.tables = torch.empty(0, columns, dtype=torch.int32, device="cuda")
        self.lengths = torch.empty(0, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def select(self, parents, grow):
        """The rows that go on, each with room for `grow` more tokens."""
        self.tables, self.lengths, self.refs = T.cache_select(self.tables, self.lengths, self.refs, parents, [self.k, self.v],
                                                              page_size=PAGE, grow=grow, status=self.status)

    def compact(self):
        self.tables, self.refs, _ = T.cache_compact(self.tables, self.lengths, self.refs, [self.k, self.v], page_size=PAGE,
                                                    status=self.status)

    def attend(self, model, tokens):
        """The last token of every row (whose slot select made): stored and attended with; log-probabilities."""
        q, k, v = model.project(tokens)
        positions = self.lengths - 1
        q = T.cache_append(k, v, self.k, self.v, self.tables, positions, q=q, turns=model.turns, status=self.status)
        x = T.attention_decode(q, self.k, self.v, self.tables, self.lengths, status=self.status)
        return torch.log_softmax((x.flatten(1) @ model.out).float(), -1)


def search(model, prompts, beams=4, steps=40, leave=None):
    """Extends each prompt (a list of token lists) by `steps` tokens, keeping `beams` beams; requests for which `leave`
    says so stop halfway. Returns ({request: [(tokens, score) of each beam]}, cache)."""
    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    longest = max(len(p) for p in prompts) + steps
    columns = -(-longest // PAGE)
    add = Scores()
    cache = Cache(pages=len(prompts) * (columns + beams * (steps // PAGE + 2)), columns=columns)
    # the prompts, but their last tokens, enter the cache; then every request is its beams' first
    cache.select(i32([-1] * len(prompts)), i32([len(p) - 1 for p in prompts]))
    rows = [r for r, p in enumerate(prompts) for _ in p[:-1]]
    if rows:
        _, k, v = model.project(torch.tensor([t for p in prompts for t in p[:-1]], device="cuda"))
        T.cache_append(k, v, cache.k, cache.v, cache.tables, i32([i for p in prompts for i in range(len(p) - 1)]),
                       rows=i32(rows), turns=model.turns, status=cache.status)
    cache.select(i32(range(len(prompts))), i32([1] * len(prompts)))
    scores = cache.attend(model, torch.tensor([p[-1] for p in prompts], device="cuda"))
    best = scores.topk(beams, -1)
    score, token = best.values.flatten(), best.indices.flatten()
    parents = torch.arange(len(prompts), device="cuda").repeat_interleave(beams)
    alive = list(range(len(prompts)))
    history = torch.empty(len(parents), 0, dtype=torch.long, device="cuda")
    done = {}
    one = i32([1] * len(parents))
    for step in range(1, steps):
        cache.select(parents.int(), one[: len(parents)])
        history = torch.cat([history[parents] if step > 1 else history, token[:, None]], 1)
        scores = add(cache.attend(model, token), score)
        best = scores.view(len(alive), -1).topk(beams, -1)  # over a request's beams and the vocabulary
        score, token = best.values.flatten(), (best.indices % VOCABULARY).flatten()
        parents = (best.indices // VOCABULARY + beams * torch.arange(len(alive), device="cuda")[:, None]).flatten()
        if leave is not None and step == steps // 2:
            tokens = torch.cat([history[parents], token[:, None]], 1)
            stay = [i for i, r in enumerate(alive) if not leave(r)]
            for i, r in enumerate(alive):
                if i not in stay:
                    done[r] = [(tokens[b].tolist(), float(score[b])) for b in range(i * beams, (i + 1) * beams)]
            keep = torch.tensor([i * beams + b for i in stay for b in range(beams)], dtype=torch.long, device="cuda")
            alive, parents, token, score = [alive[i] for i in stay], parents[keep], token[keep], score[keep]
            if not alive:
                break
            # the requests that left are freed by not being named, and the pool closes up
            cache.select(parents.int(), torch.zeros_like(one[: len(parents)]))
            cache.compact()
            history, parents = history[parents], torch.arange(len(parents), device="cuda")
    tokens = torch.cat([history[parents], token[:, None]], 1)
    for i, r in enumerate(alive):
        done[r] = [(tokens[b].tolist(), float(score[b])) for b in range(i * beams, (i + 1) * beams)]
    T.cache_status(cache.status)
    add.kernel.sync()
    return done, cache


def main():
    gen = torch.Generator().manual_seed(1)
    prompts = [torch.randint(VOCABULARY, (n,), generator=gen).tolist() for n in (5, 33, 1, 128)]
    done, cache = search(Model(), prompts, leave=lambda r: r == 1)
    for r in sorted(done):
        tokens, score = done[r][0]
        print(f"request {r}: prompt of {len(prompts[r])}, best of {len(done[r])} beams {score:.3f}: {' '.join(map(str, tokens[:10]))} ...")
    used = int((cache.refs > 0).sum())
    print(f"{used} of {len(cache.refs)} pages in use, the last at {int(cache.refs.nonzero().max())}")


if __name__ == "__main__":
    main()
