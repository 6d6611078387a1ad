"""What the cache operators' C entry points check before anything is read or launched; no GPU (the pointers are never
read)."""
from __future__ import annotations

import ctypes
import re

import pytest

import tensor_command_execution_gb300 as T
from tensor_command_execution_gb300 import cache as C

F32, I32 = 0, 3
_at = iter(range(1 << 40, 1 << 60, 1 << 36))


def op(*sizes, dtype=F32, strides=None, ptr=None):
    if strides is None:
        strides, n = [], 1
        for s in reversed(sizes):
            strides.insert(0, n)
            n *= max(s, 1)
    o = C.cmd_operand(next(_at) if ptr is None else ptr, dtype, len(sizes))
    for d, (s, t) in enumerate(zip(sizes, strides)):
        o.sizes[d], o.strides[d] = s, t
    return o


def i32(*sizes, **kw):
    return op(*sizes, dtype=I32, **kw)


def refuses(name, args, status, words=""):
    s = C.entry(name)(*args)
    msg = T.lib().cmd_last_error().decode()
    assert T.STATUS[s] == status and re.search(words, msg), (T.STATUS[s], msg)


def _spec():
    return C.cmd_rope_spec(next(_at), 4, 0, 1.0, 0)


def _append(**kw):
    a = C.cmd_append_args(k=op(6, 2, 16), v=op(6, 2, 16), k_cache=op(9, 4, 2, 16), v_cache=op(9, 4, 2, 16), tables=i32(3, 5),
                          positions=i32(6), rows=i32(6), q=op(6, 4, 16), q_out=op(6, 4, 16), rope=_spec())
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_a_rank_is_checked_before_the_sizes_are_walked():
    """An operand whose rank is past its arrays is refused for that, not read beyond them. (What lies behind it here is
    another operand; its pointer, taken for a stride, would make the two ranges meet.)"""
    pair = (C.cmd_operand * 2)(i32(5, ptr=1 << 39), i32(5))
    pair[0].rank = 8
    for d in range(4):
        pair[0].sizes[d], pair[0].strides[d] = 2, 2
    q, out, spec = op(5, 2, 8), op(5, 2, 8), _spec()
    refuses("cmd_rope", (ctypes.byref(q), ctypes.byref(out), None, None, ctypes.byref(pair[0]), ctypes.byref(spec), None),
            "CMD_ERR_SHAPE", "positions has rank 8")
    a = _append()
    a.q.rank, a.q.ptr = 8, 1 << 39  # (q_out lies behind q)
    for d in range(4):
        a.q.sizes[d], a.q.strides[d] = 2, 2
    refuses("cmd_cache_append", (ctypes.byref(a), None), "CMD_ERR_SHAPE", "q has rank 8")
    a = _append()
    a.q_out.rank = 8
    refuses("cmd_cache_append", (ctypes.byref(a), None), "CMD_ERR_SHAPE", "q_out has rank 8")
