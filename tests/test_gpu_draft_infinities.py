"""Infinite and undefined values of tokens that drafts see, however little they weigh."""
from __future__ import annotations

import math

import pytest
import torch

import cacheutil as U
import tensor_command_execution_gb300 as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("junk", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("drafts,base,columns", [(3, 100, 0), (30, 100, 0), (3, 8, 0), (6, 300, 600), (1, 40, 0)])
def test_a_seen_value_enters_whatever_its_weight(kind, junk, drafts, base, columns):
    """A weight that 32 bits hold as zero is not zero: times infinity it is infinite (NaN, where a part of it is zero). In
    the row's last tile, among the drafts, and in one that all see."""
    for where in (base - 1, 0, base + min(drafts - 1, 1)):
        c = U.Cache(kind, [base + drafts], 2, 64, 16, columns=max(columns, -(-(base + drafts) // 16)))
        q = torch.zeros(1, drafts, 4, 64, device="cuda")
        q[..., 0] = 1.0
        page, slot = int(c.tables[0, where // 16]), where % 16
        c.k[:, :, :, 0] = 0.0
        c.k[page, slot, :, 0] = -8000.0  # a score of -1000: a weight of e^-1000
        c.v[page, slot, 1, 5] = junk
        out = T.attention_drafts(q.to(U.TYPES[kind]), c.k, c.v, c.tables, c.lengths)
        sees = torch.arange(drafts, device="cuda") >= where - base
        enters = ~torch.isfinite(out[0, :, 2:, 5])
        assert torch.equal(enters, sees[:, None].expand(-1, 2))
        rest = out[0].clone()
        rest[:, 2:, 5] = 0.0
        assert bool(torch.isfinite(rest).all())
