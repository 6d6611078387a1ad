"""Commands and the cache operators in one program: on one stream, in one graph, each reading what the other wrote."""
from __future__ import annotations

import os
import sys

import pytest
import torch

import cacheutil as U
import tensor_command_execution_gb300 as T

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import beam_search as B  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("beams", [1, 3, 12])
def test_the_examples_command_adds_scores(beams):
    x, s = torch.randn(beams, B.VOCABULARY, device="cuda"), torch.randn(2 * beams, device="cuda")[::2]
    add = B.Scores()
    assert torch.equal(add(x, s), x + s[:, None])
    add.kernel.sync()


def test_a_step_of_commands_and_operators():
    """A gate on the queries and positions from lengths (Commands), append and attention, and a residual on the result (a
    Command): launched, and captured in a graph and replayed on other numbers."""
    c = U.Cache("f32", [33, 16, 5], 2, 64, 16, columns=4)
    gen = torch.Generator(device="cuda").manual_seed(2)
    q, gate, k, v = (torch.randn(3, h, 64, generator=gen, device="cuda") for h in (8, 8, 2, 2))
    turns = T.rope_turns(64)
    before = T.Command()
    a, g = before.load_tensor("f32", 3), before.load_tensor("f32", 3)
    gated = before.store(before.execute([("mul", a, g)])[0], "f32", 3)
    before = before.compile()
    step = T.Command()
    n, one = step.load_tensor("i32", 1), step.load_scalar("i32")
    last = step.store(step.execute([("sub", n, one)])[0], "i32", 1)
    step = step.compile()
    after = T.Command()
    y, z = after.load_tensor("f32", 3), after.load_tensor("f32", 3)
    total = after.store(after.execute([("add", y, z)])[0], "f32", 3)
    after = after.compile()
    x, pos, out = torch.empty_like(q), torch.empty_like(c.lengths), torch.empty_like(q)

    def run():
        before.launch({a: q, g: gate, gated: x})
        step.launch({n: c.lengths, last: pos}, {one: 1})
        turned = T.cache_append(k, v, c.k, c.v, c.tables, pos, q=x, turns=turns)
        after.launch({y: T.attention_decode(turned, c.k, c.v, c.tables, c.lengths), z: q, total: out})
        return out

    def plain():
        turned = T.cache_append(k, v, c.k, c.v, c.tables, c.lengths - 1, q=q * gate, turns=turns)
        return T.attention_decode(turned, c.k, c.v, c.tables, c.lengths) + q
    kc = c.k.clone()
    got = run().clone()
    c.k.copy_(kc)
    assert torch.equal(got, plain())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run()
    for seed in range(3):
        q.copy_(torch.randn(q.shape, generator=gen, device="cuda"))
        c.lengths.copy_(torch.tensor([33 - seed, 16, 1 + seed]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, plain()), seed
    for kernel in (before, step, after):
        kernel.sync()
