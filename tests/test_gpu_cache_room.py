"""Selections from a pool that runs out."""
from __future__ import annotations

import pytest
import torch

import tensor_command_execution_gb300 as T

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_a_row_without_room_keeps_its_place_in_the_order():
    """Two free pages; row 0 asks for three and gets none, and row 1, whose page would be the fourth in order, is
    dropped with it. A row that needs no new page goes on."""
    refs, pool = _i32([0, 0, 1]), torch.zeros(3, 4, device="cuda")
    tables, lengths = _i32([[2, -1, -1, -1]]), _i32([3])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, n, r = T.cache_select(tables, lengths, refs, _i32([-1, -1, 0]), [pool], page_size=4, grow=_i32([12, 1, 1]), status=status)
    assert n.tolist() == [0, 0, 4] and t.tolist() == [[-1] * 4, [-1] * 4, [2, -1, -1, -1]] and r.tolist() == [0, 0, 1]
    with pytest.raises(T.CmdError, match="free page"):
        T.cache_status(status)
    t, n, r = T.cache_select(tables, lengths, refs, _i32([-1, -1, 0]), [pool], page_size=4, grow=_i32([1, 12, 1]))
    assert n.tolist() == [1, 0, 4] and r.tolist() == [1, 0, 1]
