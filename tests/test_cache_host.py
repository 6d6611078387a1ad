"""The cache operators' C ABI without a GPU: declarations, structures, frequencies and refusals."""
from __future__ import annotations

import ctypes
import math
import os
import re
import shutil
import subprocess
from decimal import Decimal, getcontext

import pytest

import tensor_command_execution_gb300 as T
from tensor_command_execution_gb300 import cache as C

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def test_every_declaration_is_bound():
    with open(os.path.join(ROOT, "include", "cmd_cache.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = re.findall(r"\b(cmd_\w+)\(", text)
    assert set(names) == set(C.SIGNATURES)
    for n in names:
        assert C.entry(n) is not None


def test_structures_match_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no gcc")
    names = ["cmd_operand", "cmd_rope_spec", "cmd_append_args", "cmd_attention_args", "cmd_pool", "cmd_select_args",
             "cmd_compact_args"]
    src = '#include <stddef.h>\n#include <stdio.h>\n#include "cmd_cache.h"\nint main(void) {\n'
    for n in names:
        src += f'  printf("{n} %zu\\n", sizeof({n}));\n'
        for f, _ in getattr(C, n)._fields_:
            src += f'  printf("{n}.{f} %zu\\n", offsetof({n}, {f}));\n'
    (tmp_path / "s.c").write_text(src + "  return 0;\n}\n")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(tmp_path / "s.c"), "-o",
                    str(tmp_path / "s")], check=True)
    out = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout
    for line in out.splitlines():
        name, value = line.split()
        n, _, f = name.partition(".")
        s = getattr(C, n)
        assert (getattr(s, f).offset if f else ctypes.sizeof(s)) == int(value), name


# ---- frequencies ---------------------------------------------------------------------------------------------------

def _turns(n, base, f=lambda i, x: x):
    """2^64 base^(-i / n) / (2 pi), with f applied to the frequency, in 60 digits."""
    return [f(i, (-(Decimal(base).ln() * i / n)).exp()) / (2 * PI) * 2 ** 64 for i in range(n)]


def _close(got, want):
    # binary64: a power (1 ulp), a division and a product, 2^-53 each, and the integer's rounding
    assert len(got) == len(want)
    for g, w in zip(got, want):
        assert abs(Decimal(g) - w) <= w * Decimal(2) ** -50 + 1


@pytest.mark.parametrize("n,base", [(1, 10000.0), (5, 500000.0), (32, 10000.0), (64, 1e6), (128, 2.5)])
def test_turns(n, base):
    _close(C.cmd_rope_turns(n, base, 0, 0, 0, 0, 0), _turns(n, base))
    _close(C.cmd_rope_turns(n, base, 1, 8.0, 0, 0, 0), _turns(n, base, lambda i, x: x / 8))
    if n > 1:
        scaled = Decimal(base) * (Decimal(4).ln() * n / (n - 1)).exp()
        got = C.cmd_rope_turns(n, base, 2, 4.0, 0, 0, 0)
        # (the base is itself rounded: its relative error enters up to once)
        for g, w in zip(got, _turns(n, scaled)):
            assert abs(Decimal(g) - w) <= w * Decimal(2) ** -48 + 1
        plain = _turns(n, base)
        assert abs(Decimal(got[-1]) - plain[-1] / 4) <= plain[-1] * Decimal(2) ** -48 + 1  # the slowest, divided by the factor
        assert got[0] == C.cmd_rope_turns(n, base, 0, 0, 0, 0, 0)[0]            # the fastest, kept


def test_turns_by_parts():
    """Pairs that turn often over the original length are kept, slow ones divided, with a ramp between."""
    n, base, factor, length, fast, slow = 64, 10000.0, 16.0, 4096.0, 32.0, 1.0
    got = C.cmd_rope_turns(n, base, 3, factor, length, fast, slow)
    plain = C.cmd_rope_turns(n, base, 0, 0, 0, 0, 0)
    pair = lambda beta: n * math.log(length / (beta * 2 * math.pi)) / math.log(base)  # noqa: E731
    lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), n - 1)
    assert 0 < lo < hi < n - 1
    for i in range(n):
        r = min(max((i - lo) / (hi - lo), 0.0), 1.0)
        want = plain[i] * (1 - r) + plain[i] / factor * r
        assert abs(got[i] - want) <= want * 2.0 ** -48 + 1
    assert got[0] == plain[0] and got[lo] == plain[lo]
    # one pair whose ramp has no width, and a factor of one
    assert C.cmd_rope_turns(1, 1.5, 3, 2.0, 1.0, 2.0, 1.0)
    _close(C.cmd_rope_turns(n, base, 3, 1.0, length, fast, slow), _turns(n, base))


@pytest.mark.parametrize("args,status", [
    ((-1, 1e4, 0, 0, 0, 0, 0), "CMD_ERR_SHAPE"), ((4, 1.0, 0, 0, 0, 0, 0), "CMD_ERR_ARG"), ((4, math.inf, 0, 0, 0, 0, 0), "CMD_ERR_ARG"),
    ((4, math.nan, 0, 0, 0, 0, 0), "CMD_ERR_ARG"), ((4, 1e4, 4, 1, 0, 0, 0), "CMD_ERR_ARG"), ((4, 1e4, 1, 0.5, 0, 0, 0), "CMD_ERR_ARG"),
    ((4, 1e4, 2, math.nan, 0, 0, 0), "CMD_ERR_ARG"), ((4, 1e4, 3, 2, 0, 32, 1), "CMD_ERR_ARG"), ((4, 1e4, 3, 2, 4096, 1, 32), "CMD_ERR_ARG"),
    ((4, 1e4, 3, 2, 4096, 32, 0), "CMD_ERR_ARG"),
])
def test_turns_refusals(args, status):
    with pytest.raises(T.CmdError) as e:
        C.cmd_rope_turns(*args)
    assert e.value.name == status


def test_turns_in_python():
    t = T.rope_turns(8, 1000.0, device="cpu")
    assert [x % (1 << 64) for x in t.tolist()] == C.cmd_rope_turns(4, 1000.0, 0, 0, 0, 0, 0)
    for bad in (lambda: T.rope_turns(7, device="cpu"), lambda: T.rope_turns(8, scaling="other", device="cpu")):
        with pytest.raises(ValueError):
            bad()


# ---- refusals (every check comes before anything is launched; the pointers are never read) ----------------------------

F32, F16, BF16, I32, B1 = 0, 1, 2, 3, 4
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


def refuses(name, args, status, words=""):
    s = C.entry(name)(*args)
    msg = T.lib().cmd_last_error().decode()
    assert T.STATUS[s] == status and re.search(words, msg), (T.STATUS[s], msg)


def _spec(**kw):
    s = C.cmd_rope_spec(next(_at), 4, 0, 1.0, 0)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def test_rope_refusals():
    ok = dict(q=op(5, 2, 8), q_out=op(5, 2, 8), k=op(5, 1, 8), k_out=op(5, 1, 8), positions=op(5, dtype=I32), spec=_spec())

    def bad(status, words="", **kw):
        a = {**ok, **kw}
        ref = [ctypes.byref(a[n]) if a[n] is not None else None for n in ("q", "q_out", "k", "k_out", "positions", "spec")]
        refuses("cmd_rope", (*ref, None), status, words)
    bad("CMD_ERR_NULL", positions=None)
    bad("CMD_ERR_NULL", spec=None)
    bad("CMD_ERR_NULL", "absent", q=None, k=None)
    bad("CMD_ERR_NULL", "q_out", q_out=None)
    bad("CMD_ERR_NULL", "q is NULL", q=op(5, 2, 8, ptr=0))
    bad("CMD_ERR_TYPE", "q_out", q_out=op(5, 2, 8, dtype=BF16))
    bad("CMD_ERR_TYPE", "k", k=op(5, 1, 8, dtype=F16), k_out=op(5, 1, 8, dtype=F16))
    bad("CMD_ERR_TYPE", "float", q=op(5, 2, 8, dtype=I32))
    bad("CMD_ERR_TYPE", "positions", positions=op(5, dtype=F32))
    bad("CMD_ERR_SHAPE", "rank", q=op(5, 8))
    bad("CMD_ERR_SHAPE", "rank", positions=op(1, 5, dtype=I32))
    bad("CMD_ERR_SHAPE", "size", positions=op(4, dtype=I32))
    bad("CMD_ERR_SHAPE", "size", q_out=op(5, 2, 6))
    bad("CMD_ERR_SHAPE", "tokens or dim", k=op(6, 1, 8), k_out=op(6, 1, 8))
    bad("CMD_ERR_SHAPE", "unit stride", q=op(5, 2, 8, strides=(32, 16, 2)))
    bad("CMD_ERR_SHAPE", "negative stride", q=op(5, 2, 8, strides=(-16, 8, 1)))
    bad("CMD_ERR_SHAPE", "negative size", q=op(-5, 2, 8))
    bad("CMD_ERR_SHAPE", "rotated", spec=_spec(n_pairs=5))
    bad("CMD_ERR_SHAPE", "rotated", spec=_spec(n_pairs=-1))
    bad("CMD_ERR_NULL", "turns", spec=_spec(turns=0))
    bad("CMD_ERR_ALIGN", "turns", spec=_spec(turns=12))
    bad("CMD_ERR_ARG", "layout", spec=_spec(layout=2))
    bad("CMD_ERR_ARG", "scale", spec=_spec(scale=math.inf))
    bad("CMD_ERR_ALIGN", "q ", q=op(5, 2, 8, ptr=(1 << 40) + 2))
    bad("CMD_ERR_ALIAS", "overlaps itself", q_out=op(5, 2, 8, strides=(0, 8, 1)))
    bad("CMD_ERR_ALIAS", "overlaps itself", q_out=op(5, 2, 8, strides=(16, 4, 1)))
    bad("CMD_ERR_ALIAS", "q_out overlaps q", q_out=op(5, 2, 8, ptr=ok["q"].ptr + 4))
    bad("CMD_ERR_ALIAS", "k_out overlaps q", k_out=op(5, 1, 8, ptr=ok["q"].ptr))
    bad("CMD_ERR_ALIAS", "positions", q_out=op(5, 2, 8, ptr=ok["positions"].ptr))
    wide = [op(2, 1, 257), op(2, 1, 257)]
    bad("CMD_ERR_LIMIT", "256", q=wide[0], q_out=wide[1], k=None, positions=op(2, dtype=I32))


def test_append_refusals():
    def make(**kw):
        a = C.cmd_append_args(k=op(6, 2, 16), v=op(6, 2, 16), k_cache=op(9, 4, 2, 16), v_cache=op(9, 4, 2, 16),
                              tables=op(3, 5, dtype=I32), positions=op(6, dtype=I32), rows=op(6, dtype=I32), q=op(6, 4, 16),
                              q_out=op(6, 4, 16), rope=_spec())
        for k, v in kw.items():
            setattr(a, k, v)
        return a

    def bad(status, words="", **kw):
        refuses("cmd_cache_append", (ctypes.byref(make(**kw)), None), status, words)
    refuses("cmd_cache_append", (None, None), "CMD_ERR_NULL")
    bad("CMD_ERR_TYPE", "v_cache", v_cache=op(9, 4, 2, 16, dtype=F16))
    bad("CMD_ERR_TYPE", "k ", k=op(6, 2, 16, dtype=F16))
    bad("CMD_ERR_SHAPE", "heads or dim", k=op(6, 3, 16), v=op(6, 3, 16))
    bad("CMD_ERR_SHAPE", "size", v_cache=op(9, 4, 2, 8))
    bad("CMD_ERR_SHAPE", "no token", k_cache=op(9, 0, 2, 16), v_cache=op(9, 0, 2, 16))
    bad("CMD_ERR_SHAPE", "rows may be absent", rows=C.cmd_operand())
    bad("CMD_ERR_SHAPE", "size", positions=op(5, dtype=I32))
    bad("CMD_ERR_SHAPE", "unit stride", k_cache=op(9, 4, 2, 16, strides=(256, 64, 32, 2)))
    bad("CMD_ERR_ARG", "nothing rotates", rope=_spec(n_pairs=0))
    bad("CMD_ERR_SHAPE", "tokens or dim", q=op(5, 4, 16), q_out=op(5, 4, 16))
    bad("CMD_ERR_ALIAS", "overlaps itself", k_cache=op(9, 4, 2, 16, strides=(0, 32, 16, 1)))
    both = make().k_cache
    bad("CMD_ERR_ALIAS", "v_cache", k_cache=both, v_cache=both)
    bad("CMD_ERR_ALIAS", "k_cache overlaps tables", k_cache=both, tables=op(3, 5, dtype=I32, ptr=both.ptr + 64))
    bad("CMD_ERR_ALIAS", "q_out overlaps k", q_out=op(6, 4, 16, ptr=both.ptr), k_cache=both)
    bad("CMD_ERR_LIMIT", "2.31", tables=op(3, 1 << 30, dtype=I32))
    bad("CMD_ERR_LIMIT", "256", **{n: op(*s, 264) for n, s in (("k", (6, 2)), ("v", (6, 2)), ("k_cache", (9, 4, 2)), ("v_cache", (9, 4, 2)))})


def test_attention_refusals():
    ws = next(_at)
    need = C.cmd_attention_workspace(4, 2, 16)

    def make(**kw):
        a = C.cmd_attention_args(q=op(3, 4, 16), out=op(3, 4, 16), lse=op(3, 4), k_cache=op(9, 4, 2, 16), v_cache=op(9, 4, 2, 16),
                                 tables=op(3, 5, dtype=I32), lengths=op(3, dtype=I32), scale=0.25, workspace=ws,
                                 workspace_bytes=need)
        for k, v in kw.items():
            setattr(a, k, v)
        return a

    def bad(status, words="", **kw):
        refuses("cmd_attention_decode", (ctypes.byref(make(**kw)), None), status, words)
    refuses("cmd_attention_decode", (None, None), "CMD_ERR_NULL")
    bad("CMD_ERR_SHAPE", "heads must divide", q=op(3, 5, 16), out=op(3, 5, 16))
    bad("CMD_ERR_SHAPE", "dim", q=op(3, 4, 8), out=op(3, 4, 8))
    bad("CMD_ERR_SHAPE", "no elements", **{n: op(*s) for n, s in (("q", (3, 4, 0)), ("out", (3, 4, 0)), ("k_cache", (9, 4, 2, 0)), ("v_cache", (9, 4, 2, 0)))})
    bad("CMD_ERR_SHAPE", "rows", tables=op(4, 5, dtype=I32))
    bad("CMD_ERR_SHAPE", "lengths", lengths=op(2, dtype=I32))
    bad("CMD_ERR_TYPE", "lse", lse=op(3, 4, dtype=F16))
    bad("CMD_ERR_TYPE", "q ", q=op(3, 4, 16, dtype=BF16))
    bad("CMD_ERR_TYPE", "tables", tables=op(3, 5))
    bad("CMD_ERR_ARG", "scale", scale=0.0)
    bad("CMD_ERR_ARG", "scale", scale=math.nan)
    bad("CMD_ERR_ARG", "softcap", softcap=-1.0)
    bad("CMD_ERR_ARG", "window", window=-1)
    bad("CMD_ERR_ARG", "reserved", reserved=1)
    bad("CMD_ERR_NULL", "workspace", workspace=0)
    bad("CMD_ERR_ALIGN", "workspace", workspace=ws + 8)
    bad("CMD_ERR_LIMIT", "workspace", workspace_bytes=need - 1)
    a = make()
    bad("CMD_ERR_ALIAS", "out overlaps q", out=op(3, 4, 16, ptr=a.q.ptr), q=a.q)
    bad("CMD_ERR_ALIAS", "lse overlaps out", lse=op(3, 4, ptr=a.out.ptr), out=a.out)
    bad("CMD_ERR_ALIAS", "out .*overlaps itself", out=op(3, 4, 16, strides=(64, 0, 1)))
    bad("CMD_ERR_LIMIT", "2.31 tiles", **{n: op(1, 1 << 28, 4096, 1, strides=(0, 0, 0, 1)) for n in ("k_cache", "v_cache")}, q=op(3, 4096, 1),
        out=op(3, 4096, 1), lse=C.cmd_operand(), workspace_bytes=1 << 40)
    for args, status in (((0, 1, 8), "CMD_ERR_SHAPE"), ((5, 2, 8), "CMD_ERR_SHAPE"), ((4, 0, 8), "CMD_ERR_SHAPE"),
                         ((4, 2, 257), "CMD_ERR_LIMIT"), ((1 << 20, 1, 8), "CMD_ERR_LIMIT")):
        with pytest.raises(T.CmdError) as e:
            C.cmd_attention_workspace(*args)
        assert e.value.name == status
    # nothing to do: no launch, and so no GPU needed
    empty = C.cmd_attention_args(q=op(0, 4, 16), out=op(0, 4, 16), k_cache=op(9, 4, 2, 16), v_cache=op(9, 4, 2, 16),
                                 tables=op(0, 5, dtype=I32), lengths=op(0, dtype=I32), scale=1.0)
    assert C.entry("cmd_attention_decode")(ctypes.byref(empty), None) == 0


def _pool(n_bytes=1024, stride=1024, ptr=None):
    return C.cmd_pool(next(_at) if ptr is None else ptr, n_bytes, stride)


def test_select_and_compact_refusals():
    ws = next(_at)

    def i32(*s, **kw):
        return op(*s, dtype=I32, **kw)

    def select(**kw):
        a = C.cmd_select_args(tables=i32(4, 6), lengths=i32(4), refs=i32(20), parents=i32(5), grow=i32(5), tables_out=i32(5, 6),
                              lengths_out=i32(5), refs_out=i32(20), page_size=8, workspace=ws, workspace_bytes=1 << 20)
        a.pools, a.n_pools = (C.cmd_pool * 2)(_pool(), _pool()), 2
        for k, v in kw.items():
            setattr(a, k, v)
        return a

    def compact(**kw):
        a = C.cmd_compact_args(tables=i32(4, 6), lengths=i32(4), refs=i32(20), tables_out=i32(4, 6), refs_out=i32(20),
                               page_map_out=i32(20), page_size=8, workspace=ws, workspace_bytes=1 << 20)
        a.pools, a.n_pools = (C.cmd_pool * 2)(_pool(), _pool()), 2
        for k, v in kw.items():
            setattr(a, k, v)
        return a
    for name, make in (("cmd_cache_select", select), ("cmd_cache_compact", compact)):
        def bad(status, words="", **kw):
            refuses(name, (ctypes.byref(make(**kw)), None), status, words)
        refuses(name, (None, None), "CMD_ERR_NULL")
        bad("CMD_ERR_TYPE", "tables", tables=op(4, 6))
        bad("CMD_ERR_SHAPE", "lengths", lengths=i32(3))
        bad("CMD_ERR_SHAPE", "refs_out", refs_out=i32(19))
        bad("CMD_ERR_SHAPE", "unit stride", tables=i32(4, 6, strides=(12, 2)))
        bad("CMD_ERR_SHAPE", "no token", page_size=0)
        bad("CMD_ERR_NULL", "workspace", workspace=0)
        bad("CMD_ERR_ALIGN", "workspace", workspace=ws + 4)
        bad("CMD_ERR_LIMIT", "workspace", workspace_bytes=64)
        bad("CMD_ERR_LIMIT", "pools", n_pools=65)
        bad("CMD_ERR_LIMIT", "pools", n_pools=-1)
        bad("CMD_ERR_LIMIT", "2.31", page_size=1 << 30)
        bad("CMD_ERR_SHAPE", "overlap", pools=(C.cmd_pool * 2)(_pool(stride=512), _pool()))
        bad("CMD_ERR_NULL", "pool", pools=(C.cmd_pool * 2)(_pool(ptr=0), _pool()))
        bad("CMD_ERR_LIMIT", "address space", pools=(C.cmd_pool * 2)(_pool(stride=1 << 60), _pool()))
        p = _pool()
        bad("CMD_ERR_ALIAS", "two pools", pools=(C.cmd_pool * 2)(p, p))
        bad("CMD_ERR_ALIAS", "two pools", pools=(C.cmd_pool * 2)(p, _pool(stride=2048, ptr=p.ptr + 1024)))
        refs = i32(20)
        bad("CMD_ERR_ALIAS", "refs_out overlaps refs", refs=refs, refs_out=refs)
        bad("CMD_ERR_ALIAS", "refs overlaps a pool", refs=refs, pools=(C.cmd_pool * 2)(_pool(ptr=refs.ptr), _pool()))
        out = i32(5 if name == "cmd_cache_select" else 4, 6, strides=(3, 1))
        bad("CMD_ERR_ALIAS", "overlaps itself", tables_out=out)
    refuses("cmd_cache_select", (ctypes.byref(select(tables_out=i32(5, 7))), None), "CMD_ERR_SHAPE", "columns")
    refuses("cmd_cache_select", (ctypes.byref(select(grow=i32(4))), None), "CMD_ERR_SHAPE", "grow")
    refuses("cmd_cache_select", (ctypes.byref(select(refs=i32((1 << 30) + 1), refs_out=i32((1 << 30) + 1))), None), "CMD_ERR_LIMIT", "2.30")
    refuses("cmd_cache_compact", (ctypes.byref(compact(page_map_out=i32(21))), None), "CMD_ERR_SHAPE", "page_map_out")
    for f, a in ((C.cmd_select_workspace, (-1, 1, 1)), (C.cmd_compact_workspace, (1 << 31,))):
        with pytest.raises(T.CmdError) as e:
            f(*a)
        assert e.value.name == "CMD_ERR_SHAPE"
    assert C.cmd_select_workspace(0, 0, 0) > 0 and C.cmd_compact_workspace(1000) >= 8000


def test_views_that_interleave_are_apart():
    """Keys and values in one tensor, and slices of a fused projection, share their ranges and no element; shifted by
    one element they do."""
    def call(shift):
        kv = next(_at)
        strides = (2 * 4 * 2 * 16, 2 * 16, 16, 1)
        a = C.cmd_append_args(k=op(0, 2, 16), v=op(0, 2, 16), k_cache=op(9, 4, 2, 16, strides=strides, ptr=kv),
                              v_cache=op(9, 4, 2, 16, strides=strides, ptr=kv + 4 * (4 * 2 * 16 + shift)),
                              tables=op(3, 5, dtype=I32), positions=op(0, dtype=I32), rows=op(0, dtype=I32), rope=_spec())
        return C.entry("cmd_cache_append")(ctypes.byref(a), None)
    assert call(0) == 0
    assert T.STATUS[call(-1)] == "CMD_ERR_ALIAS" and T.STATUS[call(1)] == "CMD_ERR_ALIAS"

    def fused(heads, shift):
        x = next(_at)
        strides = (8 * 16, 16, 1)
        q = op(0, 5, 16, strides=strides, ptr=x)
        k = op(0, heads, 16, strides=strides, ptr=x + 4 * (5 * 16 + shift))
        for o in (q, k):
            o.sizes[0] = 3
        return C.entry("cmd_rope")(ctypes.byref(q), ctypes.byref(q), ctypes.byref(k), ctypes.byref(k),
                                   ctypes.byref(op(4, dtype=I32)), ctypes.byref(_spec()), None)
    # (the positions are too long: what is refused shows which check was met first)
    assert T.STATUS[fused(3, 0)] == "CMD_ERR_SHAPE"
    assert T.STATUS[fused(4, 0)] == "CMD_ERR_ALIAS" and T.STATUS[fused(3, -16)] == "CMD_ERR_ALIAS"


def test_tensors_must_be_on_a_gpu():
    torch = pytest.importorskip("torch")
    x, i = torch.zeros(2, 1, 8), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        T.rope(x, None, i, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="absent"):
        T.rope(None, None, i, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="layout"):
        T.rope(x, None, i, torch.zeros(4, dtype=torch.int64), layout="other")
    with pytest.raises(TypeError, match="tensor"):
        T.cache_append([1.0], x, x, x, i, i)
    with pytest.raises(ValueError, match="GPU"):
        T.attention_decode(x, x, x, i, i)
    with pytest.raises(ValueError, match="GPU"):
        T.cache_select(i, i, i, i, [x], page_size=1)
    with pytest.raises(ValueError, match="GPU"):
        T.cache_compact(i, i, i, [x], page_size=1)
    with pytest.raises(ValueError, match="GPU"):
        T.cache_status(i)
