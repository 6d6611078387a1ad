"""What the entry points for drafted tokens and budgets check before anything is read or launched; no GPU (the pointers are
never read)."""
from __future__ import annotations

import ctypes
import os
import re
import shutil
import subprocess

import pytest

import tensor_command_execution_gb300 as T
from tensor_command_execution_gb300 import cache as C
from test_cache_refusals import F32, i32, op, refuses

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = 2
_at = iter(range(1 << 50, 1 << 60, 1 << 36))


def _drafts(**kw):
    a = C.cmd_drafts_args(q=op(3, 5, 4, 16), out=op(3, 5, 4, 16), lse=op(3, 5, 4), k_cache=op(9, 4, 2, 16), v_cache=op(9, 4, 2, 16),
                          tables=i32(3, 6), lengths=i32(3), parents=i32(3, 5), weights=op(3, 2, 24), scale=0.25,
                          workspace=next(_at), workspace_bytes=1 << 30)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _path(**kw):
    a = C.cmd_path_args(tokens=i32(3, 5), choices=i32(3, 5), parents=i32(3, 5), path=i32(3, 5), counts=i32(3), last=i32(3))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _accept(pools=None, **kw):
    pools = [op(9, 4, 2, 16) for _ in range(2)] if pools is None else pools
    a = C.cmd_accept_args(tables=i32(3, 6), lengths=i32(3), refs=i32(9), path=i32(3, 5), counts=i32(3), lengths_out=i32(3),
                          refs_out=i32(9), pools=(C.cmd_operand * max(1, len(pools)))(*pools), n_pools=len(pools))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _evict(ks=None, vs=None, ws=None, **kw):
    ks = [op(9, 4, 2, 16)] if ks is None else ks
    vs = [op(9, 4, 2, 16) for _ in ks] if vs is None else vs
    ws = [op(3, 2, 24) for _ in ks] if ws is None else ws
    arrays = [(C.cmd_operand * max(1, len(x)))(*x) for x in (ks, vs, ws)]
    a = C.cmd_evict_args(tables=i32(3, 6), lengths=i32(3), refs=i32(9), lengths_out=i32(3), refs_out=i32(9), k_caches=arrays[0],
                         v_caches=arrays[1], weights=arrays[2], n_layers=len(ks), budget=10, recent=3, workspace=next(_at),
                         workspace_bytes=1 << 30)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_structures_match_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no gcc")
    names = ["cmd_drafts_args", "cmd_path_args", "cmd_accept_args", "cmd_evict_args"]
    src = '#include <stddef.h>\n#include <stdio.h>\n#include "cmd_cache.h"\nint main(void) {\n'
    for n in names:
        src += f'  printf("{n} %zu\\n", sizeof({n}));\n'
        for f, _ in getattr(C, n)._fields_:
            src += f'  printf("{n}.{f} %zu\\n", offsetof({n}, {f}));\n'
    src += '  printf("limits %d %d %d\\n", CMD_CACHE_MAX_DRAFTS, CMD_CACHE_MAX_LAYERS, CMD_CACHE_SHARED_PAGE);\n'
    (tmp_path / "s.c").write_text(src + "  return 0;\n}\n")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(tmp_path / "s.c"), "-o",
                    str(tmp_path / "s")], check=True)
    out = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout
    lines = out.splitlines()
    assert lines.pop() == f"limits {C.CMD_CACHE_MAX_DRAFTS} {C.CMD_CACHE_MAX_LAYERS} {C.SHARED_PAGE}"
    for line in lines:
        name, value = line.split()
        n, _, f = name.partition(".")
        s = getattr(C, n)
        assert (getattr(s, f).offset if f else ctypes.sizeof(s)) == int(value), name


@pytest.mark.parametrize("change,status,words", [
    (dict(q=op(3, 4, 16)), "SHAPE", "rank"), (dict(out=op(3, 5, 4, 17)), "SHAPE", "out"), (dict(out=op(3, 5, 4, 16, dtype=BF16)), "TYPE", "out"),
    (dict(q=op(3, 5, 4, 16, strides=(640, 128, 32, 2))), "SHAPE", "unit stride"), (dict(q=op(3, 5, 3, 16), out=op(3, 5, 3, 16)), "SHAPE", "divide"),
    (dict(q=op(3, 0, 4, 16), out=op(3, 0, 4, 16)), "LIMIT", "1 to 256"), (dict(q=op(3, 257, 4, 16), out=op(3, 257, 4, 16)), "LIMIT", "1 to 256"),
    (dict(q=op(3, 256, 8192, 16), out=op(3, 256, 8192, 16)), "LIMIT", "2.20"),
    (dict(tables=i32(2, 6)), "SHAPE", "rows"), (dict(lengths=i32(4)), "SHAPE", "lengths"), (dict(lengths=op(3)), "TYPE", "lengths"),
    (dict(parents=i32(3, 4)), "SHAPE", "parents"), (dict(parents=op(3, 5)), "TYPE", "parents"), (dict(lse=op(3, 5, 3)), "SHAPE", "lse"),
    (dict(lse=op(3, 5, 4, dtype=BF16)), "TYPE", "lse"), (dict(weights=op(3, 2, 23)), "SHAPE", "fewer tokens"), (dict(weights=op(3, 1, 24)), "SHAPE", "heads"),
    (dict(weights=op(3, 2, 24, dtype=BF16)), "TYPE", "weights"), (dict(weights=op(3, 2, 24, strides=(48, 24, 2))), "SHAPE", "unit stride"),
    (dict(weights=op(3, 2, 24, strides=(0, 24, 1))), "ALIAS", "weights"), (dict(out=op(3, 5, 4, 16, strides=(0, 64, 16, 1))), "ALIAS", "out"),
    (dict(scale=0.0), "ARG", "scale"), (dict(scale=float("nan")), "ARG", "scale"), (dict(softcap=-1.0), "ARG", "softcap"), (dict(window=-1), "ARG", "window"),
    (dict(reserved=1), "ARG", "reserved"), (dict(status=(1 << 39) + 2), "ALIGN", "status"), (dict(workspace=None), "NULL", "workspace"),
    (dict(workspace=(1 << 39) + 8), "ALIGN", "workspace"), (dict(workspace_bytes=64), "LIMIT", "workspace"), (dict(q=op(3, 5, 4, 0), out=op(3, 5, 4, 0), k_cache=op(9, 4, 2, 0), v_cache=op(9, 4, 2, 0)), "SHAPE", "no elements"),
    (dict(tables=i32(3, 1 << 30)), "LIMIT", "2.31"), (dict(k_cache=op(9, 4, 2, 264), v_cache=op(9, 4, 2, 264)), "LIMIT", "256"),
])
def test_attention(change, status, words):
    refuses("cmd_attention_drafts", (ctypes.byref(_drafts(**change)), None), "CMD_ERR_" + status, words)


def test_attention_overlaps():
    a = _drafts()
    for name in ("q", "k_cache", "v_cache", "tables", "lengths", "parents"):
        refuses("cmd_attention_drafts", (ctypes.byref(_drafts(out=op(3, 5, 4, 16, ptr=getattr(a, name).ptr), **{name: getattr(a, name)})), None), "CMD_ERR_ALIAS", name)
        refuses("cmd_attention_drafts", (ctypes.byref(_drafts(weights=op(3, 2, 24, ptr=getattr(a, name).ptr), **{name: getattr(a, name)})), None), "CMD_ERR_ALIAS", name)
    refuses("cmd_attention_drafts", (ctypes.byref(_drafts(lse=a.lse, weights=op(3, 2, 24, ptr=a.lse.ptr))), None), "CMD_ERR_ALIAS", "lse")
    refuses("cmd_attention_drafts", (None, None), "CMD_ERR_NULL")


def test_a_rank_is_checked_before_the_sizes_are_walked():
    for name in ("q", "out", "lse", "k_cache", "v_cache", "tables", "lengths", "parents", "weights"):
        a = _drafts()
        getattr(a, name).rank = 8
        refuses("cmd_attention_drafts", (ctypes.byref(a), None), "CMD_ERR_SHAPE", f"{name} has rank 8")
    for name in ("tokens", "choices", "parents", "path", "counts", "last"):
        a = _path()
        getattr(a, name).rank = 8
        refuses("cmd_draft_path", (ctypes.byref(a), None), "CMD_ERR_SHAPE", f"{name} has rank 8")
    for make, entry in ((_accept, "cmd_cache_accept"), (_evict, "cmd_cache_evict")):
        for name in ("tables", "lengths", "refs", "lengths_out", "refs_out") + (("path", "counts") if make is _accept else ()):
            a = make()
            getattr(a, name).rank = 8
            refuses(entry, (ctypes.byref(a), None), "CMD_ERR_SHAPE", f"{name} has rank 8")
    bad = op(9, 4, 2, 16)
    bad.rank = 8
    refuses("cmd_cache_accept", (ctypes.byref(_accept([op(9, 4, 2, 16), bad])), None), "CMD_ERR_SHAPE", "pool 1 has rank 8")
    refuses("cmd_cache_evict", (ctypes.byref(_evict(vs=[bad])), None), "CMD_ERR_SHAPE", "v_cache 0 has rank 8")
    w = op(3, 2, 24)
    w.rank = 8
    refuses("cmd_cache_evict", (ctypes.byref(_evict(ws=[w])), None), "CMD_ERR_SHAPE", "weights 0 has rank 8")


@pytest.mark.parametrize("change,status,words", [
    (dict(tokens=op(3, 5)), "TYPE", "tokens"), (dict(choices=i32(3, 4)), "SHAPE", "choices"), (dict(parents=i32(2, 5)), "SHAPE", "parents"),
    (dict(path=i32(3, 6)), "SHAPE", "path"), (dict(path=i32(3, 5, strides=(0, 1))), "ALIAS", "path"), (dict(counts=i32(5)), "SHAPE", "counts"),
    (dict(last=i32(3, strides=(0,))), "ALIAS", "last"), (dict(status=(1 << 39) + 2), "ALIGN", "status"),
    (dict(tokens=i32(3, 257), choices=i32(3, 257), parents=i32(3, 257), path=i32(3, 257)), "LIMIT", "256"),
    (dict(tokens=i32(3, 0), choices=i32(3, 0), parents=i32(3, 0), path=i32(3, 0)), "LIMIT", "256"),
])
def test_path(change, status, words):
    refuses("cmd_draft_path", (ctypes.byref(_path(**change)), None), "CMD_ERR_" + status, words)
    a = _path()
    refuses("cmd_draft_path", (ctypes.byref(_path(path=i32(3, 5, ptr=a.tokens.ptr), tokens=a.tokens)), None), "CMD_ERR_ALIAS", "tokens")
    refuses("cmd_draft_path", (None, None), "CMD_ERR_NULL")


def _common(make):
    return [
        (dict(lengths=i32(2)), "SHAPE", "lengths"), (dict(lengths=i32(3, strides=(2,))), "SHAPE", "unit stride"), (dict(refs=op(9)), "TYPE", "refs"),
        (dict(refs=i32(8)), "SHAPE", "pages"), (dict(refs_out=i32(8)), "SHAPE", "refs_out"), (dict(lengths_out=i32(4)), "SHAPE", "lengths_out"),
        (dict(tables=i32(3, 6, strides=(12, 2))), "SHAPE", "unit stride"), (dict(reserved=1), "ARG", "reserved"), (dict(status=(1 << 39) + 2), "ALIGN", "status"),
        (dict(tables=i32(3, 1 << 30)), "LIMIT", "2.31|fewer"),
    ]


@pytest.mark.parametrize("change,status,words", _common(_accept) + [
    (dict(pools=[]), "LIMIT", "1 to 64"), (dict(pools=[op(9, 4, 2, 16) for _ in range(65)]), "LIMIT", "1 to 64"), (dict(n_pools=-1), "LIMIT", "1 to 64"),
    (dict(pools=[op(9, 4, 2, 16), op(9, 4, 2, 17)]), "SHAPE", "pool 1"), (dict(pools=[op(9, 4, 2, 16), op(9, 4, 2, 16, dtype=BF16)]), "TYPE", "pool 1"),
    (dict(pools=[i32(9, 4, 2, 16)]), "TYPE", "no float"), (dict(pools=[op(9, 0, 2, 16)]), "SHAPE", "no token"), (dict(pools=[op(9, 4, 0, 16)]), "SHAPE", "no elements"),
    (dict(pools=[op(9, 4, 2, 300)]), "LIMIT", "256"), (dict(pools=[op(9, 4, 2, 16, strides=(0, 32, 16, 1))]), "ALIAS", "pool 0"),
    (dict(pools=[op(9, 4, 2, 16, ptr=1 << 38), op(9, 4, 2, 16, ptr=(1 << 38) + 64)]), "ALIAS", "pool"), (dict(path=i32(2, 5)), "SHAPE", "path"),
    (dict(path=i32(3, 257)), "LIMIT", "256"), (dict(path=i32(3, 0)), "LIMIT", "256"), (dict(counts=i32(2)), "SHAPE", "counts"), (dict(path=op(3, 5)), "TYPE", "path"),
])
def test_accept(change, status, words):
    refuses("cmd_cache_accept", (ctypes.byref(_accept(**change)), None), "CMD_ERR_" + status, words)


@pytest.mark.parametrize("change,status,words", _common(_evict) + [
    (dict(ks=[]), "LIMIT", "1 to 32"), (dict(ks=[op(9, 4, 2, 16) for _ in range(33)]), "LIMIT", "1 to 32"), (dict(budget=2), "ARG", "recent"),
    (dict(recent=-1), "ARG", "recent"), (dict(ws=[op(3, 2, 23)]), "SHAPE", "fewer"), (dict(ws=[op(3, 3, 24)]), "SHAPE", "heads"),
    (dict(ws=[op(3, 2, 24, dtype=BF16)]), "TYPE", "weights 0"), (dict(ws=[op(3, 2, 24, strides=(48, 24, 2))]), "SHAPE", "unit stride"),
    (dict(ws=[op(3, 2, 24, strides=(24, 24, 1))]), "ALIAS", "weights 0"), (dict(vs=[op(9, 4, 2, 8)]), "SHAPE", "v_cache 0"),
    (dict(workspace=None), "NULL", "workspace"), (dict(workspace_bytes=32), "LIMIT", "workspace"), (dict(workspace=(1 << 39) + 8), "ALIGN", "workspace"),
])
def test_evict(change, status, words):
    refuses("cmd_cache_evict", (ctypes.byref(_evict(**change)), None), "CMD_ERR_" + status, words)


def test_keep_overlaps():
    pool = op(9, 4, 2, 16)
    for make, entry in ((lambda **kw: _accept([pool], **kw), "cmd_cache_accept"), (lambda **kw: _evict([pool], **kw), "cmd_cache_evict")):
        for name, sizes in (("tables", (3, 6)), ("lengths", (3,)), ("refs", (9,)), ("lengths_out", (3,)), ("refs_out", (9,))):
            refuses(entry, (ctypes.byref(make(**{name: i32(*sizes, ptr=pool.ptr)})), None), "CMD_ERR_ALIAS", name)
        a = make()
        refuses(entry, (ctypes.byref(make(lengths=a.lengths, lengths_out=i32(3, ptr=a.lengths.ptr))), None), "CMD_ERR_ALIAS", "lengths")
        refuses(entry, (ctypes.byref(make(refs=a.refs, refs_out=i32(9, ptr=a.refs.ptr))), None), "CMD_ERR_ALIAS", "refs")
        refuses(entry, (None, None), "CMD_ERR_NULL")
    refuses("cmd_cache_accept", (ctypes.byref(_accept([pool], path=i32(3, 5, ptr=pool.ptr))), None), "CMD_ERR_ALIAS", "path")
    refuses("cmd_cache_evict", (ctypes.byref(_evict([pool], ws=[op(3, 2, 24, ptr=pool.ptr)])), None), "CMD_ERR_ALIAS", "weights 0")
    refuses("cmd_cache_evict", (ctypes.byref(_evict([pool], vs=[pool])), None), "CMD_ERR_ALIAS", "v_cache 0")


def test_no_rows():
    """No row, no launch."""
    a = _drafts(q=op(0, 5, 4, 16), out=op(0, 5, 4, 16), lse=op(0, 5, 4), tables=i32(0, 6), lengths=i32(0), parents=i32(0, 5), weights=op(0, 2, 24))
    assert C.entry("cmd_attention_drafts")(ctypes.byref(a), None) == 0
    a = _path(tokens=i32(0, 5), choices=i32(0, 5), parents=i32(0, 5), path=i32(0, 5), counts=i32(0), last=i32(0))
    assert C.entry("cmd_draft_path")(ctypes.byref(a), None) == 0


def test_workspaces():
    for args, status, words in (((3, 0, 4, 2, 64, 0), "LIMIT", "1 to 256"), ((3, 257, 4, 2, 64, 0), "LIMIT", "1 to 256"), ((3, 5, 4, 3, 64, 0), "SHAPE", "divide"),
                                ((-1, 5, 4, 2, 64, 0), "SHAPE", "negative"), ((3, 5, 4, 2, 257, 0), "LIMIT", "256"), ((3, 256, 8192, 2, 64, 0), "LIMIT", "2.20")):
        with pytest.raises(T.CmdError, match=words):
            C.cmd_drafts_workspace(*args)
    with pytest.raises(T.CmdError, match="negative"):
        C.cmd_evict_workspace(-1, 1, 1, 1)
    with pytest.raises(T.CmdError, match="2.31"):
        C.cmd_evict_workspace(1 << 20, 32, 64, 1)
    # any call of as many drafts with at most as many rows and heads, query heads to a kv head, tokens, and at most the dim
    for rows, d, q, kv, dim, t in ((4, 24, 32, 8, 128, 900), (1, 256, 8, 8, 64, 0), (700, 1, 16, 1, 256, 64)):
        mine = C.cmd_drafts_workspace(rows, d, q, kv, dim, t)
        for rows2, q2, kv2, dim2, t2 in ((1, 32, 8, 128, 900), (1, 8, 8, 64, 1), (4, 8, 2, 20, 0), (700, 4, 1, 1, 64), (2, 16, 4, 64, 2)):
            if rows2 <= rows and q2 <= q and q2 * kv <= q * kv2 and dim2 <= dim and t2 <= t:
                assert C.cmd_drafts_workspace(rows2, d, q2, kv2, dim2, t2) <= mine
    assert C.cmd_drafts_workspace(512, 1, 64, 8, 128, 1 << 30) < C.cmd_drafts_workspace(512, 1, 64, 8, 128, 0) + (1 << 30) + (1 << 20)


def test_the_module_refuses():
    """Arguments of the Python functions that never reach a GPU."""
    import torch
    x = torch.zeros(1, 2, 3, 4)
    for call in (lambda: T.attention_drafts(x, x, x, x, x), lambda: T.draft_path(x, x), lambda: T.cache_accept(x, x, x, x, x, [x]),
                 lambda: T.cache_evict(x, x, x, [(x, x, x)], budget=1)):
        with pytest.raises(ValueError, match="not on a GPU"):
            call()


def test_the_header_names_the_entry_points():
    with open(os.path.join(ROOT, "include", "cmd_cache.h")) as f:
        text = f.read()
    for name in ("cmd_attention_drafts", "cmd_draft_path", "cmd_cache_accept", "cmd_cache_evict"):
        assert re.search(rf"\*   {name} ", text) and hasattr(C, "SIGNATURES") and name in C.SIGNATURES
