"""One draft's weights use the workspace that they need, and no more."""
from __future__ import annotations

import pytest
import torch

import cacheutil as U
import tensor_command_execution_gb300 as T
from test_gpu_drafts import _randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,dim,hq,tokens,kept", [("f32", 64, 16, 1 << 18, False), ("bf16", 100, 16, 1 << 18, False), ("bf16", 64, 16, 1 << 18, True),
                                                     ("bf16", 64, 64, 3 << 20, False), ("f16", 33, 16, 1 << 18, False)])
def test_no_room_for_scores_that_are_not_kept(kind, dim, hq, tokens, kept):
    """Tables with room for far more tokens than the rows hold."""
    c = U.Cache(kind, [100, 33], 2, dim, 16, columns=tokens // 16)
    q, lse = _randn(2, 1, hq, dim, kind=kind), torch.empty(2, 1, hq, device="cuda")
    weights, out = torch.zeros(2, 2, tokens, device="cuda"), torch.empty(2, 1, hq, dim, dtype=U.TYPES[kind], device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, weights=weights, out=out, lse=lse, return_lse=True)
    used = torch.cuda.max_memory_allocated() - before
    scores = 2 * hq * tokens * 4
    assert used < 32 << 20 if not kept else scores <= used < scores + (32 << 20)
    # what the same rows give in tables of their own length
    small = torch.zeros(2, 2, 112, device="cuda")
    want, want_lse = T.attention_drafts(q, c.k, c.v, c.tables[:, :7].contiguous(), c.lengths, weights=small, return_lse=True)
    # (split otherwise: sums of 100 terms in 32 bits, values up to 5 and two roundings of the type)
    assert bool(((out.double() - want.double()).abs() <= 5 * (2.0 ** -15 + 2 * U.ROUND[kind])).all())
    assert bool(((lse - want_lse).abs() < 2.0 ** -18).all())
    assert bool(((weights[..., :112] - small).abs() < 2.0 ** -18 * hq).all()) and not weights[..., 112:].any()
