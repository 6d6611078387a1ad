"""The workspace that a call of the attention of drafts really needs; no GPU (the pointers are never read)."""
from __future__ import annotations

import ctypes

import pytest

import tensor_command_execution_gb300 as T
from tensor_command_execution_gb300 import cache as C
from test_cache_refusals import i32, op, refuses

F32, F16, BF16 = 0, 1, 2
ROWS, HEADS, KV, PAGE = 3, 8, 2, 16


def _args(dtype, dim, columns, drafts=1, weights=True, pad=0, **kw):
    wide = dim + pad
    k, v = (op(9, PAGE, KV, dim, dtype=dtype, strides=(PAGE * KV * wide, KV * wide, wide, 1)) for _ in range(2))
    return C.cmd_drafts_args(q=op(ROWS, drafts, HEADS, dim, dtype=dtype), out=op(ROWS, drafts, HEADS, dim, dtype=dtype), k_cache=k, v_cache=v,
                             tables=i32(ROWS, columns), lengths=i32(ROWS), scale=0.25,
                             weights=op(ROWS, KV, columns * PAGE) if weights else C.cmd_operand(), **kw)


def _need(a):
    n = ctypes.c_int64()
    status = C.entry("cmd_attention_drafts_workspace")(ctypes.byref(a), ctypes.byref(n))
    assert status == 0
    return n.value


def _most(dim, columns, drafts=1):
    return C.cmd_drafts_workspace(ROWS, drafts, HEADS, KV, dim, columns * PAGE)


def _scores(columns):
    return 4 * ROWS * HEADS * columns * PAGE


def test_scores_that_are_kept_have_room():
    for dtype, dim in ((BF16, 64), (F16, 128), (BF16, 256)):
        assert _need(_args(dtype, dim, 40)) == _most(dim, 40)


@pytest.mark.parametrize("dtype,dim,pad", [(F32, 64, 0), (BF16, 33, 0), (F16, 100, 0), (BF16, 64, 1), (F16, 64, 2)])
def test_scores_that_are_not_kept_have_none(dtype, dim, pad):
    """32 bits, and rows that are no whole 16-byte vectors."""
    assert _need(_args(dtype, dim, 40, pad=pad)) == _most(dim, 40) - _scores(40)


def test_scores_above_a_gib_have_none():
    columns = (1 << 30) // (4 * ROWS * HEADS * PAGE)
    assert _need(_args(BF16, 64, columns)) == _most(64, columns) == _most(64, 1) - _scores(1) + (_scores(columns) + 15) // 16 * 16
    assert _need(_args(BF16, 64, columns + 1)) == _most(64, 1) - _scores(1) < 1 << 24


def test_without_weights_and_of_several_drafts_it_is_what_the_sizes_say():
    for dtype in (F32, BF16):
        assert _need(_args(dtype, 64, 40, weights=False)) == C.cmd_drafts_workspace(ROWS, 1, HEADS, KV, 64, 0)
        assert _need(_args(dtype, 64, 40, drafts=7)) == _most(64, 40, 7)
        assert _need(_args(dtype, 64, 40, drafts=7, weights=False)) == C.cmd_drafts_workspace(ROWS, 7, HEADS, KV, 64, 0)


def test_a_call_asks_for_as_much():
    """One byte less is refused."""
    for a in (_args(F32, 64, 40), _args(BF16, 64, 40), _args(F16, 100, 40), _args(BF16, 64, 1 << 20)):
        a.workspace, a.workspace_bytes = 1 << 62, _need(a) - 1
        refuses("cmd_attention_drafts", (ctypes.byref(a), None), "CMD_ERR_LIMIT", f"workspace has {a.workspace_bytes} bytes, not {a.workspace_bytes + 1}")


def test_what_a_call_refuses():
    n = ctypes.c_int64()
    a = _args(BF16, 64, 40)
    a.scale = 0.0
    refuses("cmd_attention_drafts_workspace", (ctypes.byref(a), ctypes.byref(n)), "CMD_ERR_ARG", "scale")
    refuses("cmd_attention_drafts_workspace", (ctypes.byref(_args(BF16, 64, 40)), None), "CMD_ERR_NULL", "bytes")
    refuses("cmd_attention_drafts_workspace", (None, ctypes.byref(n)), "CMD_ERR_NULL", "args")
    with pytest.raises(T.CmdError):
        C.cmd_drafts_workspace(1, 0, 1, 1, 1)
