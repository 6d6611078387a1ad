"""The drafting example: every token that it gives is one that the model, in 64 bits and without a cache, would choose."""
from __future__ import annotations

import os
import sys

import pytest
import torch

import cacheutil as U

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import beam_search as B  # noqa: E402
import drafting as X  # noqa: E402

pytestmark = pytest.mark.gpu


def _prompts():
    gen = torch.Generator().manual_seed(3)
    return [torch.randint(B.VOCABULARY, (n,), generator=gen).tolist() for n in (5, 33, 1, 60)]


def _logits(model, seq):
    """The model's logits after every position, attended to anew, in 64 bits."""
    x = model.embedding[torch.tensor(seq, device="cuda")].double().cpu()
    q, k, v = ((x @ w.double().cpu()).view(len(x), -1, B.DIM) for w in (model.q, model.k, model.v))
    pos = torch.arange(len(x), dtype=torch.int32)
    q, k = (U.rotated(y, pos, model.turns, "half", 1.0) for y in (q, k))
    s = torch.einsum("ihgd,thd->ihgt", q.view(len(x), B.KV_HEADS, -1, B.DIM), k) * B.DIM ** -0.5
    s = s.masked_fill(torch.ones(len(x), len(x)).triu(1).bool()[:, None, None], -torch.inf)
    o = torch.einsum("ihgt,thd->ihgd", torch.softmax(s, -1), v).reshape(len(x), -1)
    return o @ model.out.double().cpu()


def _chosen(model, prompt, tokens):
    """A logit is a product of 512 terms of 16-bit numbers, each off by a few times 2^-9 of about 1 (the beam search
    example's test): the token chosen is within 2 * 2^-6 of the largest."""
    logits = _logits(model, prompt + tokens[:-1])[len(prompt) - 1:]
    off = logits.amax(-1) - logits[torch.arange(len(tokens)), torch.tensor(tokens)]
    assert float(off.max()) < 2 * 2.0 ** -6


def _held(cache):
    held = torch.zeros_like(cache.refs)
    for row, n in zip(cache.tables.tolist(), cache.lengths.tolist()):
        for p in row[: -(-n // B.PAGE)]:
            held[p] += 1
    return held


@pytest.mark.parametrize("tree,rank", [(X.TREE, X.RANK), ([-1, 0, 1, 2], [0, 0, 0, 0]), ([-1], [0]),
                                       ([-1] + [i // 3 for i in range(39)], [0] + [i % 3 for i in range(39)])])
def test_drafted_tokens_are_those_of_the_model(tree, rank):
    model, prompts = B.Model(), _prompts()
    out, given, g = X.drafted(model, prompts, 24, tree, rank)
    for r, p in enumerate(prompts):
        assert len(out[r]) == sum(x[r] for x in given) >= 24
        _chosen(model, p, out[r])
    c = g.cache
    assert torch.equal(_held(c), c.refs)
    assert c.lengths.tolist() == [len(p) - 1 + len(o) for p, o in zip(prompts, out)]
    assert torch.equal(c.lengths, g.positions)


def test_plain_tokens_are_those_of_the_model():
    model, prompts = B.Model(), _prompts()
    for p, o in zip(prompts, X.plain(model, prompts, 24)):
        _chosen(model, p, o)


def test_a_budget_that_is_never_reached_changes_nothing():
    model, prompts = B.Model(), _prompts()
    out, g, weights = X.budgeted(model, prompts, 30, budget=200, recent=10)
    assert out == X.plain(model, prompts, 30)
    # each step's heads give one in all
    for r, n in enumerate(g.cache.lengths.tolist()):
        assert bool(((weights[r].double().sum(-1) - 30 * B.HEADS // B.KV_HEADS).abs() < 30 * 4 * 2.0 ** -18).all())
        assert bool((weights[r, :, n:] == 0).all())


def test_rows_stay_inside_their_budget():
    model, prompts = B.Model(), _prompts()
    out, g, weights = X.budgeted(model, prompts, 40, budget=32, recent=8)
    c = g.cache
    assert c.lengths.tolist() == [32, 32, 32, 32] and torch.equal(_held(c), c.refs)
    assert bool((weights[:, :, 32:] == 0).all()) and all(len(o) == 40 for o in out)
    assert g.positions.tolist() == [len(p) - 1 + 40 for p in prompts]
