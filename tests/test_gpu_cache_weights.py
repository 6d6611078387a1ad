"""Attention over long rows in which one token's score stands far above the others: what is left of small weights."""
from __future__ import annotations

import pytest
import torch

import cacheutil as U
import tensor_command_execution_gb300 as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 100, 33, 256])
@pytest.mark.parametrize("above", [9.0, 15.5, 17.5, 20.0])
def test_small_weights_beside_a_dominant_token(kind, dim, above):
    """The first token takes all but a small part of the softmax and has a value of zero, so the output is what the
    others' weights, e^-above of it each, add up to. 512 rows of the same 8192 tokens: most of a row goes to one warp
    group, whose running maximum is the first token's score.

    The bound is that of arithmetic in 32 bits (cacheutil.attended) and of a weight held as two 16-bit numbers: each
    rounds to the type's digits (2^-22 and 2^-16 of the weight together), and in f16 no finer than half of its smallest
    step of weights lifted by 2^15, 2^-40 of the largest weight."""
    n, rows = 8192, 512
    c = U.Cache(kind, [n], 1, dim, 32)
    gen = torch.Generator(device="cuda").manual_seed(3)
    first = (int(c.tables[0, 0]), 0)
    c.k.copy_(0.05 * torch.randn(c.k.shape, generator=gen, device="cuda"))
    c.v.copy_(64.0 + 64.0 * torch.rand(c.v.shape, generator=gen, device="cuda"))
    c.k[..., 0] = 0
    c.k[first] = 0
    c.k[first + (0, 0)] = above * dim ** 0.5
    c.v[first] = 0
    q = torch.randn(1, 1, dim, generator=gen, device="cuda").to(U.TYPES[kind])
    q[..., 0] = 1
    out, lse = T.attention_decode(q.expand(rows, 1, dim), c.k, c.v, c.tables.expand(rows, -1), c.lengths.expand(rows),
                                  return_lse=True)
    want, want_lse, bound, lse_bound = U.attended(q, c, [n], dim ** -0.5)
    assert float(want.min()) > 1e-4  # (far above f16's smallest numbers)
    k, v = c.rows(0, n)
    split = {"f32": 0.0, "f16": 2.0 ** -22, "bf16": 2.0 ** -16}[kind] * want + {"f16": n * 2.0 ** -40}.get(kind, 0.0) * v.amax()
    bound = bound + split + U.ROUND[kind] * want.abs() * (1 + 2.0 ** -10) + U.TINY[kind]
    off = (out.cpu().double() - want).abs()
    assert bool((off <= bound).all()), f"off by {float((off / want).max()):.3g} of the value, {float((off / bound).max()):.3g} of the bound"
    assert bool(((lse.cpu().double() - want_lse).abs() <= lse_bound).all())
