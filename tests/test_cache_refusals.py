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


def _attention(**kw):
    a = C.cmd_attention_args(q=op(3, 4, 16), out=op(3, 4, 16), k_cache=op(9, 4, 2, 16), v_cache=op(9, 4, 2, 16), tables=i32(3, 5),
                             lengths=i32(3), scale=0.25, workspace=next(_at), workspace_bytes=1 << 30)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _pooled(kind, rows=4, **kw):
    common = dict(tables=i32(rows, 0), lengths=i32(rows), refs=i32(20), refs_out=i32(20), page_size=8, workspace=next(_at), workspace_bytes=1 << 40)
    if kind == "select":
        a = C.cmd_select_args(parents=i32(5), tables_out=i32(5, 0), lengths_out=i32(5), **common)
    else:
        a = C.cmd_compact_args(tables_out=i32(rows, 0), page_map_out=i32(20), **common)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("name,make", [
    ("cmd_cache_append", _append), ("cmd_attention_decode", _attention), ("cmd_cache_select", lambda **kw: _pooled("select", **kw)),
    ("cmd_cache_compact", lambda **kw: _pooled("compact", **kw))])
def test_a_status_word_off_its_alignment_is_refused(name, make):
    """(The kernels set its bits with 4-byte atomics.)"""
    refuses(name, (ctypes.byref(make(status=(1 << 39) + 2)), None), "CMD_ERR_ALIGN", "status")
    refuses("cmd_cache_status", ((1 << 39) + 2, None, None), "CMD_ERR_ALIGN", "status")


@pytest.mark.parametrize("kind", ["select", "compact"])
def test_rows_that_pass_the_kernels_counters_are_refused(kind):
    """The kernels step through rows in 32 bits, thousands at a time; a table of no columns may have any number."""
    many, rows = (1 << 30) + 1, "rows"
    refuses(f"cmd_cache_{kind}", (ctypes.byref(_pooled(kind, rows=many)), None), "CMD_ERR_LIMIT", rows)
    if kind == "select":
        a = _pooled(kind, parents=i32(many), tables_out=i32(many, 0), lengths_out=i32(many))
        refuses("cmd_cache_select", (ctypes.byref(a), None), "CMD_ERR_LIMIT", rows)


def test_a_workspace_serves_what_the_header_says():
    """Any call with at most as many query heads to a kv head, and at most the dim."""
    for q, kv, dim in ((32, 8, 128), (32, 32, 64), (16, 1, 256), (48, 3, 80)):
        mine = C.cmd_attention_workspace(q, kv, dim)
        for q2, kv2, dim2 in ((64, 64, 16), (64, 16, 64), (32, 1, 200), (7, 7, 256), (4096, 512, 1), (16, 1, 80)):
            if q2 * kv <= q * kv2 and dim2 <= dim:
                assert C.cmd_attention_workspace(q2, kv2, dim2) <= mine


def test_tensors_without_elements_have_any_strides():
    """Empty views come with the strides of whatever they were cut from: nothing is read through them. (No token, row or
    page: no launch, and so no GPU needed.)"""
    q, positions, spec = op(0, 2, 8, strides=(16, 8, 2)), i32(0), _spec()
    assert C.entry("cmd_rope")(ctypes.byref(q), ctypes.byref(op(0, 2, 8)), None, None, ctypes.byref(positions), ctypes.byref(spec), None) == 0
    a = _append(k=op(0, 2, 16, strides=(64, 32, 2)), v=op(0, 2, 16, strides=(0, 0, 0)), positions=i32(0), rows=i32(0), q=op(0, 4, 16), q_out=op(0, 4, 16))
    assert C.entry("cmd_cache_append")(ctypes.byref(a), None) == 0
    a = _pooled("compact", rows=0, tables=i32(0, 5, strides=(0, 3)), tables_out=i32(0, 5, strides=(1, 2)), refs=i32(0, strides=(2,)), refs_out=i32(0),
                page_map_out=i32(0))
    assert C.entry("cmd_cache_compact")(ctypes.byref(a), None) == 0
    refuses("cmd_cache_compact", (ctypes.byref(_pooled("compact", tables=i32(4, 5, strides=(10, 2)), tables_out=i32(4, 5))), None), "CMD_ERR_SHAPE", "unit stride")
