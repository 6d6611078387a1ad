"""Tensors without elements as arguments of the cache's operators: given, not absent."""
from __future__ import annotations

import pytest
import torch

import cacheutil as U
import tensor_command_execution_gb300 as T

pytestmark = pytest.mark.gpu


def _cache():
    c = U.Cache("bf16", [20, 33], 2, 64, 16)
    return c, torch.randn(2, 3, 4, 64, device="cuda").bfloat16()


def test_weights_without_room_are_refused():
    c, q = _cache()
    for shape in ((2, 2, 0), (0, 2, 48), (2, 0, 48)):
        with pytest.raises(T.CmdError, match="weights"):
            T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, weights=torch.zeros(shape, device="cuda"))
        with pytest.raises(T.CmdError, match="weights"):
            T.attention_drafts(q[:, :1], c.k, c.v, c.tables, c.lengths, weights=torch.zeros(shape, device="cuda"))


def test_log_sums_without_room_are_refused():
    c, q = _cache()
    for shape in ((0, 3, 4), (2, 3, 0)):
        with pytest.raises(T.CmdError, match="lse"):
            T.attention_drafts(q, c.k, c.v, c.tables, c.lengths, lse=torch.empty(shape, device="cuda"), return_lse=True)
    for shape in ((0, 4), (2, 0)):
        with pytest.raises(T.CmdError, match="lse"):
            T.attention_decode(q[:, 0], c.k, c.v, c.tables, c.lengths, lse=torch.empty(shape, device="cuda"))


def test_rows_and_growth_of_nobody_are_refused():
    c, q = _cache()
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    k = torch.randn(2, 2, 64, device="cuda").bfloat16()
    with pytest.raises(T.CmdError, match="rows"):
        T.cache_append(k, k, c.k, c.v, c.tables, c.lengths - 1, rows=none)
    refs = torch.ones(c.pages, dtype=torch.int32, device="cuda")
    with pytest.raises(T.CmdError, match="grow"):
        T.cache_select(c.tables, c.lengths, refs, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), [c.k, c.v], page_size=16, grow=none)


def test_calls_of_nobody_go_through():
    c, q = _cache()
    out, lse = T.attention_drafts(q[:0], c.k, c.v, c.tables[:0], c.lengths[:0], weights=torch.zeros(0, 2, 48, device="cuda"),
                                  lse=torch.empty(0, 3, 4, device="cuda"), return_lse=True)
    assert out.shape == (0, 3, 4, 64) and lse.shape == (0, 3, 4)
    out, lse = T.attention_decode(q[:0, 0], c.k, c.v, c.tables[:0], c.lengths[:0], lse=torch.empty(0, 4, device="cuda"), return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    # tables without a column: rows of no token
    for drafts in (1, 3):
        out = T.attention_drafts(q[:, :drafts], c.k, c.v, c.tables[:, :0], c.lengths * 0, weights=torch.zeros(2, 2, 0, device="cuda"))
        assert bool((out == 0).all())
    k = torch.randn(0, 2, 64, device="cuda").bfloat16()
    T.cache_append(k, k, c.k, c.v, c.tables, c.lengths[:0], rows=c.lengths[:0])
