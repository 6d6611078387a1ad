"""Several tokens to a step, and a cache that stays inside a budget: the operators for drafted tokens and for eviction in the
places they have in a serving program.

A one-layer attention model (beam_search.Model) continues a few prompts, each step choosing its likeliest token. With
drafts, a step guesses a small tree of tokens ahead, stores their keys and values behind each row's, attends to all of
them at once (attention_drafts), walks the tree along the model's own choices (draft_path) and keeps that branch
(cache_accept). With a budget, each step adds up the attention that every cached token gets, and rows that have grown
past the budget give up the tokens that got least (cache_evict). Tables, lengths and counts never leave the GPU.

    python examples/drafting.py
"""
from __future__ import annotations

import torch

from beam_search import DIM, PAGE, VOCABULARY, Cache, Model, T

# a tree of guesses: after the token that is sure, the two likeliest ones, each with its two likeliest, and three more
# behind the best of them
TREE = [-1, 0, 0, 1, 1, 2, 2, 3, 7, 8]
RANK = [0, 0, 1, 0, 1, 0, 1, 0, 0, 0]  # which of its parent's likeliest successors each is


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def _depths(tree):
    out = []
    for p in tree:
        out.append(0 if p < 0 else out[p] + 1)
    return out


class Generation:
    """Rows of a cache that grow in step, and the position that each token had when it was stored."""

    def __init__(self, model, prompts, most):
        self.model, self.rows = model, len(prompts)
        columns = -(-most // PAGE)
        self.cache = Cache(pages=self.rows * (columns + 1), columns=columns)
        self.same = _i32(range(self.rows))
        self.positions = _i32([len(p) - 1 for p in prompts])  # of the tokens that come next
        self.cache.select(_i32([-1] * self.rows), self.positions)
        rows = [r for r, p in enumerate(prompts) for _ in p[:-1]]
        if rows:
            at = _i32([i for p in prompts for i in range(len(p) - 1)])
            _, k, v = model.project(torch.tensor([t for p in prompts for t in p[:-1]], device="cuda"))
            T.cache_append(k, v, self.cache.k, self.cache.v, self.cache.tables, at, rows=_i32(rows), turns=model.turns, status=self.cache.status)
        self.tokens = torch.tensor([p[-1] for p in prompts], device="cuda")

    def attend(self, tokens, depths, parents=None, weights=None):
        """Room for the tokens [rows, n] behind each row's, their keys (at the positions that their depths say) and values
        stored, and what the model would choose after each of them."""
        c, n = self.cache, tokens.shape[1]
        c.select(self.same, torch.full_like(self.positions, n))
        q, k, v = self.model.project(tokens.flatten())
        positions = (self.positions[:, None] + depths).flatten()
        q, k = T.rope(q, k, positions, self.model.turns)
        slots = (c.lengths[:, None] - n + torch.arange(n, dtype=torch.int32, device="cuda")).flatten()
        T.cache_append(k, v, c.k, c.v, c.tables, slots, rows=self.same.repeat_interleave(n), status=c.status)
        x = T.attention_drafts(q.view(self.rows, n, -1, DIM), c.k, c.v, c.tables, c.lengths, parents=parents, weights=weights, status=c.status)
        return (x.flatten(2) @ self.model.out).argmax(-1)


def plain(model, prompts, steps):
    """One token to a step."""
    g = Generation(model, prompts, max(map(len, prompts)) + steps)
    out = []
    for _ in range(steps):
        g.tokens = g.attend(g.tokens[:, None], _i32([0]))[:, 0]
        g.positions = g.positions + 1
        out.append(g.tokens)
    T.cache_status(g.cache.status)
    return torch.stack(out, 1).tolist()


def drafted(model, prompts, steps, tree=TREE, rank=RANK):
    """As many tokens to a step as its guesses hold, and one more: (at least `steps` tokens of each row, tokens that each
    step gave)."""
    parents, depths = _i32(tree).expand(len(prompts), -1), _i32(_depths(tree))
    # what is guessed to follow a token: what the model would choose if it attended to that token alone
    after = (model.embedding @ model.v).view(VOCABULARY, -1, DIM).repeat_interleave(4, 1).flatten(1) @ model.out
    after = after.topk(max(rank) + 1, -1).indices
    g = Generation(model, prompts, max(map(len, prompts)) + (steps + 1) * len(tree))
    out, given = [[] for _ in prompts], []
    while min(map(len, out)) < steps:
        guesses = [g.tokens]
        for p, r in zip(tree[1:], rank[1:]):
            guesses.append(after[guesses[p], r])
        guesses = torch.stack(guesses, 1)
        choices = g.attend(guesses, depths, parents)
        path, counts, last = T.draft_path(guesses.int(), choices.int(), parents=parents, status=g.cache.status)
        c = g.cache
        c.lengths, c.refs = T.cache_accept(c.tables, c.lengths, c.refs, path, counts, [c.k, c.v], status=c.status)
        g.positions, g.tokens = g.positions + counts, last.long()
        for r, (p, n) in enumerate(zip(path.tolist(), counts.tolist())):  # (a server would leave them on the GPU)
            out[r] += guesses[r, p[1:n]].tolist() + [int(last[r])]
        given.append(counts.tolist())
    T.cache_status(g.cache.status)
    return out, given, g


def budgeted(model, prompts, steps, budget, recent):
    """One token to a step, and at most `budget` tokens in the cache before it: (tokens, the generation, weights)."""
    g = Generation(model, prompts, max(max(map(len, prompts)), budget) + steps)
    c = g.cache
    weights = torch.zeros(len(prompts), c.k.shape[2], c.tables.shape[1] * PAGE, device="cuda")
    out = []
    for _ in range(steps):
        g.tokens = g.attend(g.tokens[:, None], _i32([0]), weights=weights)[:, 0]
        g.positions = g.positions + 1
        out.append(g.tokens)
        c.lengths, c.refs = T.cache_evict(c.tables, c.lengths, c.refs, [(c.k, c.v, weights)], budget=budget, recent=recent, status=c.status)
    T.cache_status(c.status)
    return torch.stack(out, 1).tolist(), g, weights


def main():
    gen = torch.Generator().manual_seed(1)
    prompts = [torch.randint(VOCABULARY, (n,), generator=gen).tolist() for n in (5, 33, 1, 128)]
    model = Model()
    out, given, _ = drafted(model, prompts, 40)
    print(f"{sum(map(sum, given)) / len(given) / len(prompts):.2f} tokens to a step: {' '.join(map(str, out[0][:10]))} ...")
    out, g, _ = budgeted(model, prompts, 40, budget=48, recent=16)
    print(f"lengths {g.cache.lengths.tolist()} after 40 tokens: {' '.join(map(str, out[0][:10]))} ...")


if __name__ == "__main__":
    main()
