"""The beam search example: its scores against the model without a cache, in 64 bits."""
from __future__ import annotations

import os
import sys

import pytest
import torch

import cacheutil as U

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import beam_search as B  # noqa: E402

pytestmark = pytest.mark.gpu


def _score(model, prompt, tokens):
    """log-probability of `tokens` after `prompt`, every position attended to anew."""
    seq = torch.tensor(prompt + tokens, device="cuda")
    x = model.embedding[seq[:-1]].double().cpu()
    q, k, v = ((x @ w.double().cpu()).view(len(x), -1, B.DIM) for w in (model.q, model.k, model.v))
    pos = torch.arange(len(x), dtype=torch.int32)
    q, k = (U.rotated(y, pos, model.turns, "half", 1.0) for y in (q, k))
    group = B.HEADS // B.KV_HEADS
    total = 0.0
    for t in range(len(prompt) - 1, len(x)):
        s = torch.einsum("hgd,thd->hgt", q[t].view(B.KV_HEADS, group, B.DIM), k[: t + 1]) * B.DIM ** -0.5
        o = torch.einsum("hgt,thd->hgd", torch.softmax(s, -1), v[: t + 1]).reshape(1, -1)
        total += float(torch.log_softmax(o @ model.out.double().cpu(), -1)[0, seq[t + 1]])
    return total


def test_beam_search_scores_are_those_of_the_model():
    """The sum of n log-probabilities: each logit is a product of 512 terms of 16-bit numbers, each off by a few times
    2^-9 of about 1, so about 2^-9 * sqrt(512) / sqrt(512) * 4 < 2^-6 each way, and the errors of n steps add up."""
    gen = torch.Generator().manual_seed(1)
    prompts = [torch.randint(B.VOCABULARY, (n,), generator=gen).tolist() for n in (5, 33, 1, 128)]
    steps = 36
    model = B.Model()
    done, cache = B.search(model, prompts, beams=3, steps=steps, leave=lambda r: r == 1)
    assert sorted(done) == [0, 1, 2, 3]
    for r, beams in done.items():
        assert len(beams) == 3 and len({tuple(t) for t, _ in beams}) == 3
        n = steps // 2 + 1 if r == 1 else steps
        for tokens, score in beams:
            assert len(tokens) == n
            assert abs(score - _score(model, prompts[r], tokens)) < n * 2 * 2.0 ** -6
    # the rows that are left hold the pages in use, shared ones counted once for each
    held = torch.zeros_like(cache.refs)
    for row, n in zip(cache.tables.tolist(), cache.lengths.tolist()):
        for p in row[: -(-n // B.PAGE)]:
            held[p] += 1
        assert all(p == -1 for p in row[-(-n // B.PAGE):])
    assert torch.equal(held, cache.refs)
